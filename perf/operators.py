"""The language-model operators of this library as a set of measured cases.

Five operators, each in two forms: with ``own`` false in elementary torch
operations (computed in 32 bits, rounded once at the end), with ``own`` true
through the public entry points of post_weight_quantization_accumulate_amd.

  int4      Y = X Wq^T from an int4 or NF4 pack (codes, per-(row, group) scales),
            for one layer or for the experts of a mixture
  fp8q      a matrix to e4m3 codes with one scale per 1 x 128 or 128 x 128 block
  fp8       Y = Xq Wq^T from two such packs, for one layer or for experts
  dispatch  rows ordered by expert: the stable sort of the router's choices and
            the gather of the activations
  combine   rows brought back with the router's weights, and the gradient
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}

# The NF4 levels: standard normal quantiles at evenly spaced probabilities, 7
# below zero and 8 above, scaled to [-1, 1], as fp32.
NF4 = [float.fromhex(v) for v in (
    "-0x1p+0", "-0x1.647362p-1", "-0x1.0cd65cp-1", "-0x1.94653cp-2", "-0x1.234496p-2", "-0x1.7a6a7ap-3",
    "-0x1.74f0d2p-4", "0x0p+0", "0x1.45f602p-4", "0x1.4995bep-3", "0x1.f809b4p-3", "0x1.5a066cp-2",
    "0x1.c3496ap-2", "0x1.200f52p-1", "0x1.722760p-1", "0x1p+0")]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through an attention projection packed to int4: the decoding step, bound by the pack's bytes
        {"name": "int4 decode", "op": "int4", "M": 1, "N": 10240, "K": 5120, "group": 128, "nf4": False,
         "x": "bf16", "y": "bf16", "E": 0},
        # a prompt through an MLP down-projection packed to int4: bound by the matrix cores
        {"name": "int4 prompt", "op": "int4", "M": 4096, "N": 5120, "K": 17408, "group": 128, "nf4": False,
         "x": "bf16", "y": "bf16", "E": 0},
        # checking an NF4-packed mixture layer in fp32: ragged expert batches, a smaller group
        {"name": "int4 experts nf4", "op": "int4", "M": 1021, "N": 1000, "K": 1024, "group": 64, "nf4": True,
         "x": "fp32", "y": "fp32", "E": 16},
        # packing a weight matrix to 8 bits, 128 x 128 blocks
        {"name": "fp8 pack weights", "op": "fp8q", "M": 5120, "K": 17408, "rows": 128, "x": "fp32"},
        # packing one prompt's activations, 1 x 128 blocks; a width that ends inside a block
        {"name": "fp8 pack activations", "op": "fp8q", "M": 777, "K": 5000, "rows": 1, "x": "bf16"},
        # one token through an 8-bit MLP down-projection
        {"name": "fp8 decode", "op": "fp8", "M": 1, "N": 5120, "K": 17408, "y": "bf16", "E": 0},
        # a long prompt through an 8-bit attention projection
        {"name": "fp8 prompt", "op": "fp8", "M": 8192, "N": 10240, "K": 5120, "y": "bf16", "E": 0},
        # a mixture layer's 8-bit experts over one prompt's sorted rows
        {"name": "fp8 experts", "op": "fp8", "M": 4000, "N": 1024, "K": 5120, "y": "bf16", "E": 64},
        # one decoding batch's rows to their experts: latency counts
        {"name": "dispatch decode", "op": "dispatch", "T": 4, "k": 8, "E": 128, "D": 5120, "x": "bf16", "drop": 0.0},
        # a long prompt's rows to their experts, some choices dropped
        {"name": "dispatch prompt", "op": "dispatch", "T": 8192, "k": 8, "E": 128, "D": 5120, "x": "bf16",
         "drop": 0.02},
        # router tuning on a small fp32 batch of odd width
        {"name": "combine small", "op": "combine", "T": 33, "k": 2, "D": 1001, "x": "fp32", "drop": 0.1},
        # router tuning on a whole prompt
        {"name": "combine prompt", "op": "combine", "T": 8192, "k": 8, "D": 5120, "x": "bf16", "drop": 0.02},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["int4", "int4", "fp8q", "fp8", "fp8", "dispatch", "combine"])
    if op == "int4":
        experts = rng.random() < 0.4
        group = rng.choice([32, 64, 128])
        x = rng.choice(["bf16", "bf16", "fp32"])
        return {"op": op, "M": _log(rng, 1, 2048 if experts else 4096), "N": _log(rng, 16, 1024 if experts else 10240),
                "K": group * _log(rng, 2, (2048 if experts else 16384) // group), "group": group,
                "nf4": rng.random() < 0.4, "x": x, "y": x if rng.random() < 0.7 else "fp32",
                "E": _log(rng, 2, 64) if experts else 0}
    if op == "fp8q":
        return {"op": op, "M": _log(rng, 1, 8192), "K": _log(rng, 100, 17408), "rows": rng.choice([1, 128]),
                "x": rng.choice(["bf16", "fp32"])}
    if op == "fp8":
        experts = rng.random() < 0.4
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 16, 1024 if experts else 10240),
                "K": _log(rng, 100, 2048 if experts else 8192) if rng.random() < 0.5
                else BLOCK * _log(rng, 1, 16 if experts else 64),
                "y": rng.choice(["bf16", "bf16", "fp32"]), "E": _log(rng, 2, 64) if experts else 0}
    T, D = _log(rng, 1, 8192), _log(rng, 64, 5120)
    if op == "dispatch":
        return {"op": op, "T": T, "k": rng.randint(1, 8), "E": _log(rng, 8, 256), "D": D,
                "x": rng.choice(["bf16", "fp32"]), "drop": rng.choice([0.0, 0.05])}
    return {"op": op, "T": T, "k": rng.randint(1, 8), "D": D, "x": rng.choice(["bf16", "fp32"]),
            "drop": rng.choice([0.0, 0.05])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(g, rows, cols, dtype):
    """Normal rows under per-channel scales, log-normal with sigma 1 as hidden states have them."""
    x = torch.randn(rows, cols, generator=g, device=DEV)
    x *= torch.randn(cols, generator=g, device=DEV).exp()
    return x.to(DTYPES[dtype])


def _weights(g, rows, cols):
    """N(0, 0.02^2) with a few outliers."""
    w = torch.randn(rows, cols, generator=g, device=DEV) * 0.02
    w[torch.rand(rows, cols, generator=g, device=DEV) < 0.001] *= 20.0
    return w


def _pack_int4(w, group, nf4):
    """Round to nearest: codes (rows x K/2 bytes, even column in the low nibble) and scales."""
    rows, K = w.shape
    v = w.view(rows, K // group, group)
    s = v.abs().amax(2) / (1.0 if nf4 else 7.0)
    u = (v / s.clamp_min(1e-30).unsqueeze(2)).view(rows, K)
    if nf4:
        lv = torch.tensor(NF4, device=DEV)
        c = torch.bucketize(u, (lv[1:] + lv[:-1]) / 2).to(torch.uint8)
    else:
        c = (u.round().clamp(-8, 7).to(torch.int8) & 15).view(torch.uint8)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous(), s.contiguous()


def _blocks(x, rows):
    """x, zero-padded to whole rows x 128 blocks, as (row block, row, column block, column)."""
    R, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % BLOCK, 0, -R % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // BLOCK, BLOCK)


def _pack_fp8(x, rows):
    R, K = x.shape
    b = _blocks(x.float(), rows)
    s = b.abs().amax((1, 3)) / torch.full((), E4M3_MAX, device=DEV)     # by a tensor: an IEEE division
    q = (b / s.view(s.shape[0], 1, s.shape[1], 1)).clamp(-E4M3_MAX, E4M3_MAX)
    q = torch.where((s > 0).view(s.shape[0], 1, s.shape[1], 1), q, torch.zeros_like(q))
    q = q.view(b.shape[0] * rows, -1)[:R, :K].to(torch.float8_e4m3fn)
    return q.contiguous(), s


def _offsets(g, rows, E):
    """Expert batches as a router makes them: uneven, some empty."""
    p = torch.randn(E, generator=g, device=DEV).mul(1.0).exp()
    e = torch.multinomial(p, rows, replacement=True, generator=g)
    n = torch.bincount(e, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    off[1:] = n.cumsum(0)
    return off, int(n.max())


def _choices(g, T, k, E, drop):
    """The router's k experts of each token, distinct; a dropped choice is -1."""
    logits = torch.randn(T, E, generator=g, device=DEV) + torch.randn(E, generator=g, device=DEV)
    ids = logits.topk(k, dim=1).indices
    ids[torch.rand(T, k, generator=g, device=DEV) < drop] = -1
    return ids.to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case, "op": op}
    if op == "int4":
        M, N, K, E, G = case["M"], case["N"], case["K"], case["E"], case["group"]
        st["x"] = _activations(g, M, K, case["x"])
        st["codes"], st["scales"] = _pack_int4(_weights(g, max(E, 1) * N, K), G, case["nf4"])
        st["y"] = torch.zeros(M, N, dtype=DTYPES[case["y"]], device=DEV)
        if E:
            st["codes"], st["scales"] = st["codes"].view(E, N, K // 2), st["scales"].view(E, N, K // G)
            st["offsets"], st["most"] = _offsets(g, M, E)
    elif op == "fp8q":
        M, K = case["M"], case["K"]
        st["x"] = _activations(g, M, K, case["x"]) if case["rows"] == 1 else _weights(g, M, K).to(DTYPES[case["x"]])
        st["codes"] = torch.zeros(M, K, dtype=torch.float8_e4m3fn, device=DEV)
        st["scales"] = torch.zeros(-(-M // case["rows"]), -(-K // BLOCK), device=DEV)
    elif op == "fp8":
        M, N, K, E = case["M"], case["N"], case["K"], case["E"]
        st["xq"], st["xs"] = _pack_fp8(_activations(g, M, K, "fp32"), 1)
        if E:
            Np = -(-N // BLOCK) * BLOCK
            q, s = _pack_fp8(_weights(g, E * Np, K), BLOCK)
            st["wq"], st["ws"] = q.view(E, Np, K)[:, :N].contiguous(), s.view(E, Np // BLOCK, -1)
            st["offsets"], st["most"] = _offsets(g, M, E)
        else:
            st["wq"], st["ws"] = _pack_fp8(_weights(g, N, K), BLOCK)
        st["y"] = torch.zeros(M, N, dtype=DTYPES[case["y"]], device=DEV)
    elif op == "dispatch":
        T, k, E, D = case["T"], case["k"], case["E"], case["D"]
        st["x"] = _activations(g, T, D, case["x"])
        st["ids"] = _choices(g, T, k, E, case["drop"])
        st["offsets"] = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        st["order"] = torch.zeros(T * k, dtype=torch.int32, device=DEV)
        st["pos"] = torch.zeros(T, k, dtype=torch.int32, device=DEV)
        st["xs"] = torch.zeros(T * k, D, dtype=DTYPES[case["x"]], device=DEV)
        st["scratch"] = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)
    else:
        T, k, D = case["T"], case["k"], case["D"]
        dt = DTYPES[case["x"]]
        st["y"] = _activations(g, T * k, D, case["x"])
        kept = torch.rand(T * k, generator=g, device=DEV) >= case["drop"]
        perm = torch.randperm(T * k, generator=g, device=DEV)
        rank = torch.empty_like(perm)
        rank[perm[kept[perm]]] = torch.arange(int(kept.sum()), device=DEV)
        st["pos"] = torch.where(kept, rank, -1).to(torch.int32).view(T, k).contiguous()
        st["w"] = torch.softmax(torch.randn(T, k, generator=g, device=DEV), 1)
        st["dout"] = torch.randn(T, D, generator=g, device=DEV).to(dt)
        st["out"] = torch.zeros(T, D, dtype=dt, device=DEV)
        st["dy"] = torch.zeros(T * k, D, dtype=dt, device=DEV)
        st["dw"] = torch.zeros(T, k, device=DEV)
    return st


# ------------------------------------------------------------------ the passes
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import post_weight_quantization_accumulate_amd as gq
    op, c = st["op"], st["case"]
    if op == "int4":
        flags = gq.GQ_NF4 if c["nf4"] else 0
        if c["E"]:
            gq.int4_matmul_experts(st["y"], st["x"], st["codes"], st["scales"], st["offsets"], c["group"], flags)
        else:
            gq.int4_matmul(st["y"], st["x"], st["codes"], st["scales"], c["group"], flags)
        return st["y"]
    if op == "fp8q":
        gq.fp8_quantize(st["codes"], st["scales"], st["x"], c["rows"])
        return {"codes": st["codes"], "scales": st["scales"]}
    if op == "fp8":
        if c["E"]:
            gq.fp8_matmul_experts(st["y"], st["xq"], st["xs"], st["wq"], st["ws"], st["offsets"])
        else:
            gq.fp8_matmul(st["y"], st["xq"], st["xs"], st["wq"], st["ws"])
        return st["y"]
    if op == "dispatch":
        gq.experts_sort(st["offsets"], st["order"], st["pos"], st["ids"], st["scratch"])
        gq.experts_gather(st["xs"], st["x"], st["pos"])
        return {"offsets": st["offsets"], "order": st["order"], "pos": st["pos"], "xs": st["xs"]}
    gq.experts_combine(st["out"], st["y"], st["pos"], st["w"])
    gq.experts_combine_backward(st["dy"], st["dw"], st["dout"], st["y"], st["pos"], st["w"])
    return {"out": st["out"], "dy": st["dy"], "dw": st["dw"]}


def _product(x, w, st):
    """x w^T in fp32; with experts, each batch's rows against their expert's w, batches padded to the longest."""
    if not st["case"]["E"]:
        return x @ w.t()
    off, M = st["offsets"].long(), x.shape[0]
    row = off[:-1, None] + torch.arange(st["most"], device=DEV)
    live = row < off[1:, None]
    y = torch.bmm(x[row.clamp_max(M - 1)], w.transpose(1, 2).contiguous())
    out = torch.empty(M, w.shape[1], dtype=y.dtype, device=DEV)
    out[row[live]] = y[live]
    return out


def _run_plain(st):
    op, c = st["op"], st["case"]
    if op == "int4":
        codes, scales, G = st["codes"], st["scales"], c["group"]
        c4 = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        if c["nf4"]:
            v = torch.tensor(NF4, device=DEV)[c4.int()]
        else:
            v = ((c4 ^ 8).to(torch.int8) - 8).float()
        w = (v.unflatten(-1, (-1, G)) * scales.unsqueeze(-1)).flatten(-2)
        return _product(st["x"].float(), w, st).to(DTYPES[c["y"]])
    if op == "fp8q":
        q, s = _pack_fp8(st["x"], c["rows"])
        return {"codes": q, "scales": s}
    if op == "fp8":
        x, w, N, K = st["xq"].float(), st["wq"].float(), c["N"], c["K"]
        x = x * st["xs"].repeat_interleave(BLOCK, 1)[:, :K]
        w = w * st["ws"].repeat_interleave(BLOCK, -1).repeat_interleave(BLOCK, -2)[..., :N, :K]
        return _product(x, w, st).to(DTYPES[c["y"]])
    if op == "dispatch":
        ids, x, k, E = st["ids"].reshape(-1), st["x"], c["k"], c["E"]
        live = ids >= 0
        order = torch.sort(torch.where(live, ids, E), stable=True).indices
        n = torch.bincount(torch.where(live, ids, E), minlength=E + 1).cumsum(0)
        offsets = torch.nn.functional.pad(n[:E], (1, 0)).to(torch.int32)
        at = torch.arange(ids.numel(), device=DEV)
        pos = torch.empty_like(order)
        pos[order] = at
        pos = torch.where(live, pos, -1).to(torch.int32).view(-1, k)
        used = at < offsets[E]
        xs = torch.where(used[:, None], x[order // k], torch.zeros((), dtype=x.dtype, device=DEV))
        return {"offsets": offsets, "order": torch.where(used, order, -1).to(torch.int32), "pos": pos, "xs": xs}
    y, pos, w, dout = st["y"], st["pos"].long(), st["w"], st["dout"].float()
    live = pos >= 0
    rows = y[pos.clamp_min(0)].float()
    w = torch.where(live, w, 0.0)
    out = (rows * w.unsqueeze(2)).sum(1).to(y.dtype)
    dw = torch.where(live, (rows * dout.unsqueeze(1)).sum(2), 0.0)
    dy = torch.zeros_like(y)
    dy[pos[live]] = (w.unsqueeze(2) * dout.unsqueeze(1))[live].to(y.dtype)
    return {"out": out, "dy": dy, "dw": dw}


# ------------------------------------------------------------------ work and definition
def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "int4":
        M, N, K, n = case["M"], case["N"], case["K"], max(1, min(case["E"], case["M"]))
        return {"bytes": M * K * size[case["x"]] + n * N * (K // 2 + 4 * (K // case["group"])) + M * N * size[case["y"]],
                "flops": 2.0 * M * N * K}
    if op == "fp8q":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (size[case["x"]] + 1) + 4 * -(-M // case["rows"]) * -(-K // BLOCK), "flops": 2.0 * M * K}
    if op == "fp8":
        M, N, K, n = case["M"], case["N"], case["K"], max(1, min(case["E"], case["M"]))
        kb = -(-K // BLOCK)
        return {"bytes": M * (K + 4 * kb) + n * (N * K + 4 * kb * -(-N // BLOCK)) + M * N * size[case["y"]],
                "flops": 2.0 * M * N * K}
    T, k, D, b = case["T"], case["k"], case["D"], size[case["x"]]
    if op == "dispatch":
        return {"bytes": T * D * b + T * k * (D * b + 12) + 4 * (case["E"] + 1), "flops": 0.0}
    return {"bytes": 2 * T * D * b + 2 * T * k * D * b + 12 * T * k, "flops": 5.0 * T * k * D}


def exact(case, seed):
    """The definitions in 64 bits, expert by expert and block by block."""
    st = prepare(case, seed)
    op = case["op"]
    if op == "int4":
        N, K, G, E = case["N"], case["K"], case["group"], max(1, case["E"])
        codes, scales = st["codes"].view(E, N, K // 2), st["scales"].view(E, N, K // G)
        value = torch.tensor(NF4 if case["nf4"] else list(range(8)) + list(range(-8, 0)), dtype=torch.float64, device=DEV)
        edge = st["offsets"].tolist() if case["E"] else [0, case["M"]]
        out = torch.zeros(case["M"], N, dtype=torch.float64, device=DEV)
        for e in range(E):
            if edge[e + 1] > edge[e]:
                w = torch.empty(N, K, dtype=torch.float64, device=DEV)
                w[:, 0::2] = value[(codes[e] % 16).long()]
                w[:, 1::2] = value[(codes[e] // 16).long()]
                w.view(N, K // G, G).mul_(scales[e].double().view(N, K // G, 1))
                out[edge[e]:edge[e + 1]] = torch.mm(st["x"][edge[e]:edge[e + 1]].double(), w.t())
        return out
    if op == "fp8q":
        x, r = st["x"].double(), case["rows"]
        R, K = x.shape
        s = torch.zeros(st["scales"].shape, dtype=torch.float64, device=DEV)
        a = torch.zeros(s.shape[0] * r, K, dtype=torch.float64, device=DEV)
        a[:R] = x.abs()
        for b in range(s.shape[1]):
            s[:, b] = a[:, b * BLOCK:(b + 1) * BLOCK].reshape(s.shape[0], -1).max(1).values / E4M3_MAX
        col = torch.arange(K, device=DEV) // BLOCK
        for i in range(0, R, 1024):
            sc = s[torch.arange(i, min(R, i + 1024), device=DEV) // r][:, col]
            v = torch.where(sc > 0, x[i:i + 1024] / sc, 0.0)
            m = v.abs().clamp_min(2.0 ** -6)
            step = torch.exp2(torch.floor(torch.log2(m)) - 3)
            x[i:i + 1024] = (v / step).round() * step
        return {"codes": x.clamp(-E4M3_MAX, E4M3_MAX), "scales": s}
    if op == "fp8":
        M, N, K, E = case["M"], case["N"], case["K"], max(1, case["E"])
        edge = st["offsets"].tolist() if case["E"] else [0, M]
        wq, ws = st["wq"].view(E, N, K), st["ws"].view(E, -(-N // BLOCK), -(-K // BLOCK)).double()
        out = torch.zeros(M, N, dtype=torch.float64, device=DEV)
        col = torch.arange(K, device=DEV) // BLOCK
        for e in range(E):
            a, z = edge[e], edge[e + 1]
            if z > a:
                xd = st["xq"][a:z].double() * st["xs"].double()[a:z][:, col]
                for n in range(0, N, BLOCK):
                    wd = wq[e, n:n + BLOCK].double() * ws[e, n // BLOCK][col]
                    out[a:z, n:n + BLOCK] = torch.mm(xd, wd.t())
        return out
    if op == "dispatch":
        ids = st["ids"].reshape(-1).tolist()
        rows = [i for _, i in sorted((e, i) for i, e in enumerate(ids) if e >= 0)]
        xs = torch.zeros(len(ids), case["D"], dtype=torch.float64, device=DEV)
        xs[:len(rows)] = st["x"].double()[torch.tensor(rows, dtype=torch.long, device=DEV) // case["k"]]
        return {"offsets": None, "order": None, "pos": None, "xs": xs}
    T, k = case["T"], case["k"]
    y, dout, w = st["y"], st["dout"].double(), st["w"].double()
    pos = st["pos"].long()
    out = torch.zeros(T, case["D"], dtype=torch.float64, device=DEV)
    dw = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    dy = torch.zeros(y.shape, dtype=torch.float64, device=DEV)
    for j in range(k):
        t = (pos[:, j] >= 0).nonzero()[:, 0]
        p = pos[t, j]
        r = y[p].double()
        out[t] += w[t, j:j + 1] * r
        dw[t, j] = torch.linalg.vecdot(r, dout[t])
        dy[p] = w[t, j:j + 1] * dout[t]
    return {"out": out, "dy": dy, "dw": dw}

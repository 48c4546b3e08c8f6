"""GPU parity of the pack products (int4_matmul, fp8_matmul and their expert
forms) and the 8-bit pack (fp8_quantize) against their formulas in 64 bits.

Tolerances.  A sum of K products in fp32, in any order, is off by at most
(K + 8) 2^-23 sum |x w| when every addition is off by a whole step (the matrix
cores may truncate), the 8 covering the scale products and the parts left out
(below 2^-24 of a product); as a random walk the whole matrix is off by about
sqrt(K) 2^-24, held here to four times that plus two steps.  A bf16 output is
rounded once more, half a step: 2^-8 relative at most, 2^-8 / sqrt(3) or less in
the norm.  An fp8 product with a bf16 output may use the fp8 matrix instructions,
which add 8 products at a time with everything below 2^-13 of the largest cut
off: at most 8 2^-13 = 2^-10 of the sum of their magnitudes.  Codes and scales of the 8-bit pack are equal bit for bit: one IEEE
division each, rounding to nearest even."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gq():
    import post_weight_quantization_accumulate_amd as m
    assert torch.cuda.is_available()
    m.lib()
    return m


def _check(y, ref, mag, K, what="", cut=0.0):
    """y against the 64-bit ref; mag = sum |x w| of each entry, cut what of it may be cut off."""
    bf = y.dtype == torch.bfloat16
    y = y.double().cpu().numpy()
    half = 2.0 ** -8 if bf else 0.0
    tol = ((K + 8) * 2.0 ** -23 + cut) * mag * (1 + half) + half * np.abs(ref)
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4], y[bad][:4], ref[bad][:4])
    rel = np.linalg.norm(y - ref) / max(np.linalg.norm(ref), 1e-300)
    assert rel <= 4 * np.sqrt(K) * 2.0 ** -24 + 2.0 ** -23 + half / np.sqrt(3) + cut * np.linalg.norm(mag) / max(np.linalg.norm(ref), 1e-300), (what, rel)


def _x(rng, M, K, dt):
    return torch.from_numpy((rng.standard_normal((M, K)) * np.exp(rng.standard_normal(K))).astype(np.float32)).to(dt)


def _pack4(rng, N, K, G):
    codes = rng.integers(0, 256, (N, K // 2)).astype(np.uint8)
    scales = np.exp(rng.standard_normal((N, K // G)) * 0.5 - 4).astype(np.float32)
    return codes, scales


def _deq4(gq, codes, scales, G, nf4):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    v = gq.nf4_levels().numpy().astype(np.float64)[c] if nf4 else ((c ^ 8).astype(np.float64) - 8)
    return v * np.repeat(scales.astype(np.float64), G, 1)


def _int4(gq, M, N, K, G, nf4, xd, yd, seed, padx=0, pady=0):
    rng = np.random.default_rng(seed)
    x = _x(rng, M, K + padx, DT[xd])
    codes, scales = _pack4(rng, N, K, G)
    y = torch.full((M, N + pady), 7.0, dtype=DT[yd], device=DEV)
    xg = x.to(DEV)
    gq.int4_matmul(y[:, :N], xg[:, :K], torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), G,
                   gq.GQ_NF4 if nf4 else 0)
    w = _deq4(gq, codes, scales, G, nf4)
    xd64 = x[:, :K].double().numpy()
    _check(y[:, :N], xd64 @ w.T, np.abs(xd64) @ np.abs(w).T, K, (M, N, K, G, nf4, xd, yd))
    assert (y[:, N:] == 7.0).all()


@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M,N,K,G", [(1, 64, 128, 32), (1, 10, 6, 2), (3, 33, 96, 32), (17, 100, 130, 1),
                                     (16, 48, 640, 128), (64, 256, 1024, 128), (65, 300, 192, 64), (130, 257, 256, 16),
                                     (300, 130, 512, 128), (257, 515, 2176, 128), (5, 16, 2, 1), (2, 1000, 5120, 128),
                                     (33, 272, 1152, 128), (600, 520, 384, 128), (100, 70, 160, 32), (129, 65, 32, 32),
                                     (200, 129, 320, 64), (20, 40, 224, 32), (50, 40, 320, 64), (1, 20, 17408, 128),
                                     (1, 24, 33280, 128), (2, 16, 20608, 64), (1, 40, 96, 32), (20, 70, 64, 16)])
def test_int4_matmul(gq, M, N, K, G, nf4, xd, yd):
    _int4(gq, M, N, K, G, nf4, xd, yd, M * 31 + N + K)


@pytest.mark.parametrize("xd,nf4,G", [("bf16", False, 128), ("bf16", False, 64), ("bf16", False, 32), ("bf16", True, 128),
                                      ("fp32", False, 128), ("fp32", True, 32)])
@pytest.mark.parametrize("M,N", [(4000, 4090), (2040, 4090), (1000, 5000), (250, 10200)])
def test_int4_matmul_every_tile(gq, M, N, xd, nf4, G):
    """Sizes at which each shape of the many-row kernel is chosen, with ragged edges."""
    _int4(gq, M, N, 256, G, nf4, xd, xd, M + G)


@pytest.mark.parametrize("M,N,K,G,padx,pady", [(5, 64, 256, 128, 3, 5), (70, 128, 256, 64, 8, 8), (2, 64, 256, 128, 3, 5), (300, 256, 256, 128, 1, 0),
                                               (300, 256, 256, 128, 8, 1)])
@pytest.mark.parametrize("xd", ["bf16", "fp32"])
def test_int4_matmul_strides(gq, M, N, K, G, padx, pady, xd):
    _int4(gq, M, N, K, G, False, xd, xd, 5, padx, pady)


@pytest.mark.parametrize("M", [1, 20, 100])
@pytest.mark.parametrize("xoff", [0, 1])
def test_int4_matmul_unaligned_bases(gq, M, xoff):
    """Pointers that are only element aligned: X two bytes, the codes one byte off."""
    rng = np.random.default_rng(1)
    N, K, G = 48, 256, 128
    x = _x(rng, M, K, torch.bfloat16)
    codes, scales = _pack4(rng, N, K, G)
    xb = torch.zeros(M * K + xoff, dtype=torch.bfloat16, device=DEV)
    xb[xoff:] = x.to(DEV).reshape(-1)
    cb = torch.zeros(N * K // 2 + 1, dtype=torch.uint8, device=DEV)
    cb[1:] = torch.from_numpy(codes).to(DEV).reshape(-1)
    sb = torch.zeros(N * K // G + 1, device=DEV)
    sb[1:] = torch.from_numpy(scales).to(DEV).reshape(-1)
    yb = torch.zeros(M * N + 1, device=DEV)
    gq.int4_matmul(yb[1:].view(M, N), xb[xoff:].view(M, K), cb[1:].view(N, K // 2), sb[1:].view(N, K // G), G)
    w = _deq4(gq, codes, scales, G, False)
    x64 = x.double().numpy()
    _check(yb[1:].view(M, N), x64 @ w.T, np.abs(x64) @ np.abs(w).T, K)


@pytest.mark.parametrize("xd", ["bf16", "fp32"])
@pytest.mark.parametrize("M", [2, 4, 20, 300])
def test_int4_matmul_special_values(gq, xd, M):
    """NaN and infinity spread along their own row only; huge and tiny values survive the split into parts."""
    rng = np.random.default_rng(2)
    N, K, G = 64, 256, 128
    x = _x(rng, M, K, DT[xd])
    x[0, 5] = float("inf")
    x[1, 7] = float("nan")
    codes, scales = _pack4(rng, N, K, G)
    codes[:, 2] = 0x33                                      # column 5: code 3, so inf * 3
    y = torch.zeros(M, N, dtype=DT[xd], device=DEV)
    gq.int4_matmul(y, x.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), G)
    y = y.float().cpu()
    assert torch.isposinf(y[0]).all() and torch.isnan(y[1]).all() and torch.isfinite(y[2:]).all()
    for big in (1e30, 1e-30):
        x = _x(rng, M, K, torch.float32) * np.float32(big)
        x = x.to(DT[xd])
        y = torch.zeros(M, N, dtype=torch.float32, device=DEV)
        gq.int4_matmul(y, x.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), G)
        w, x64 = _deq4(gq, codes, scales, G, False), x.double().numpy()
        _check(y, x64 @ w.T, np.abs(x64) @ np.abs(w).T, K, big)


@pytest.mark.parametrize("xd,yd", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("M,K,G", [(1, 256, 64), (2, 256, 128), (20, 256, 128), (20, 224, 32), (300, 256, 64), (300, 320, 64), (40, 256, 16)])
def test_int4_matmul_infinity_times_every_code(gq, M, K, G, nf4, xd, yd):
    """An infinite x gives each column the infinity of its weight's sign (NaN for a weight of 0)."""
    N = 64
    rng = np.random.default_rng(M + K)
    x = _x(rng, M, K, DT[xd])
    x[0, 5] = float("inf")
    codes, scales = _pack4(rng, N, K, G)
    codes[:, 2] = ((np.arange(N) % 16) << 4) | 3             # column 5: every code
    y = torch.empty((M, N), dtype=DT[yd], device=DEV)
    gq.int4_matmul(y, x.to(DEV), torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), G, gq.GQ_NF4 if nf4 else 0)
    w = _deq4(gq, codes, scales, G, nf4)[:, 5]
    want = np.where(w == 0, np.nan, np.sign(w) * np.inf)
    np.testing.assert_array_equal(y[0].double().cpu().numpy(), want)
    assert torch.isfinite(y[1:]).all()


@pytest.mark.parametrize("counts,M", [([0, 5, 0, 17, 1, 40], 63), ([3], 3), ([0, 0, 0], 4), ([16] * 8, 128),
                                      ([1] * 70, 70), ([300, 0, 2, 257], 560), ([0, 700], 700), ([513, 31, 64], 608)])
@pytest.mark.parametrize("nf4,xd,G", [(False, "bf16", 128), (True, "fp32", 64), (False, "fp32", 32), (True, "bf16", 128),
                                      (False, "bf16", 16)])
def test_int4_matmul_experts(gq, counts, M, nf4, xd, G):
    """Ragged and empty experts; rows behind the last are left as they were."""
    rng = np.random.default_rng(M)
    E, N, K = len(counts), 136, 256
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x = _x(rng, M, K, DT[xd])
    codes, scales = _pack4(rng, E * N, K, G)
    y = torch.full((M, N), 7.0, dtype=DT[xd], device=DEV)
    gq.int4_matmul_experts(y, x.to(DEV), torch.from_numpy(codes).view(E, N, -1).to(DEV),
                           torch.from_numpy(scales).view(E, N, -1).to(DEV), torch.from_numpy(off).to(DEV), G,
                           gq.GQ_NF4 if nf4 else 0)
    w = _deq4(gq, codes, scales, G, nf4).reshape(E, N, K)
    x64 = x.double().numpy()
    for e in range(E):
        a, z = off[e], off[e + 1]
        if z > a:
            _check(y[a:z], x64[a:z] @ w[e].T, np.abs(x64[a:z]) @ np.abs(w[e]).T, K, e)
    assert (y[off[-1]:] == 7.0).all()


def test_experts_offsets_are_clamped(gq):
    """Offsets outside the rows or out of order lead nowhere outside X and Y: the rows they do name are right."""
    rng = np.random.default_rng(3)
    E, N, K, M = 4, 32, 128, 20
    x = _x(rng, M, K, torch.float32)
    codes, scales = _pack4(rng, E * N, K, 128)
    buf = torch.full((M + 2, N), 7.0, device=DEV)
    off = torch.tensor([-5, 8, 3, 12, 1000], dtype=torch.int32, device=DEV)      # expert 1 is empty
    gq.int4_matmul_experts(buf[1:-1], x.to(DEV), torch.from_numpy(codes).view(E, N, -1).to(DEV),
                           torch.from_numpy(scales).view(E, N, -1).to(DEV), off, 128)
    assert (buf[0] == 7.0).all() and (buf[-1] == 7.0).all()
    w = _deq4(gq, codes, scales, 128, False).reshape(E, N, K)
    x64 = x.double().numpy()
    for e, a, z in [(0, 0, 3), (2, 8, 12), (3, 12, 20)]:                         # rows 3 .. 7 are named twice
        _check(buf[1 + a:1 + z], x64[a:z] @ w[e].T, np.abs(x64[a:z]) @ np.abs(w[e]).T, K, e)


# ------------------------------------------------------------------ 8-bit
def _pack8_ref(x, br):
    """fp8_quantize in numpy fp32 (IEEE divisions) and torch's host conversion to e4m3."""
    x = x.float().numpy()
    R, K = x.shape
    kb = -(-K // 128)
    codes = np.zeros((R, K), np.uint8)
    scales = np.zeros((-(-R // br), kb), np.float32)
    with np.errstate(all="ignore"):
        for i in range(scales.shape[0]):
            for j in range(kb):
                b = x[i * br:(i + 1) * br, j * 128:(j + 1) * 128]
                s = np.float32(np.abs(b).max()) / np.float32(448)
                q = np.clip(b / s, -448, 448).astype(np.float32)
                if s == 0:
                    q = np.zeros_like(b)
                scales[i, j] = s
                codes[i * br:(i + 1) * br, j * 128:(j + 1) * 128] = (
                    torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    return codes, scales


def _pack8(gq, x, br, pad=0):
    R, K = x.shape
    codes = torch.zeros(R, K, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.zeros(-(-R // br), -(-K // 128), device=DEV)
    full = torch.zeros(R, K + pad, dtype=x.dtype, device=DEV)
    full[:, :K] = x.to(DEV)
    gq.fp8_quantize(codes, scales, full[:, :K], br)
    return codes, scales


@pytest.mark.parametrize("br", [1, 128])
@pytest.mark.parametrize("R,K,pad", [(1, 1, 0), (1, 128, 0), (3, 100, 0), (128, 128, 0), (129, 257, 0), (77, 5000, 0),
                                     (200, 1024, 8), (5, 130, 3), (256, 640, 0), (1000, 384, 0)])
@pytest.mark.parametrize("xd", ["bf16", "fp32"])
def test_fp8_quantize(gq, R, K, pad, xd, br):
    x = _x(np.random.default_rng(R + K), R, K, DT[xd])
    if R > 2:
        x[1] = 0.0                                   # empty blocks (of one row)
    codes, scales = _pack8(gq, x, br, pad)
    rc, rs = _pack8_ref(x, br)
    assert np.array_equal(scales.cpu().numpy().view(np.uint32), rs.view(np.uint32))
    assert np.array_equal(codes.cpu().view(torch.uint8).numpy(), rc)


@pytest.mark.parametrize("br", [1, 128])
def test_fp8_quantize_special_values(gq, br):
    """Zeros, values whose scale is subnormal or rounds to 0, halfway cases, infinity and NaN."""
    x = torch.zeros(6 * 128, 256)
    x[128] = 1e-40
    x[256] = 1e-44                                   # 1e-44 / 448 rounds to 0: codes 0
    x[384, :128] = torch.arange(128) * 0.5           # many values halfway between two codes
    x[384, 127] = 448.0
    x[512, 3] = float("inf")
    x[640, 130] = float("nan")
    x[641, 131] = -1.0
    for dt in (torch.float32, torch.bfloat16):
        xx = x.to(dt)
        codes, scales = _pack8(gq, xx, br)
        finite = slice(0, 512)
        rc, rs = _pack8_ref(xx[finite], br)
        nb = 512 // br
        assert np.array_equal(scales[:nb].cpu().numpy().view(np.uint32), rs.view(np.uint32))
        assert np.array_equal(codes[finite].cpu().view(torch.uint8).numpy(), rc)
        s = scales.repeat_interleave(br, 0).repeat_interleave(128, 1).cpu()
        v = codes.float().cpu()
        assert torch.isposinf(s[512, 0]) and torch.isnan(v[512, 3]) and v[512, 4] == 0 and torch.isnan((v * s)[512, :128]).all()
        assert torch.isnan(s[640, 128]) and torch.isnan(v[640, 128:]).all() and (v[640, :128] == 0).all()
        assert torch.isnan(v[641, 131]) == (br == 128)


def _deq8(codes, scales, br):
    v = codes.double().cpu().numpy()
    s = scales.double().cpu().numpy().repeat(br, 0).repeat(128, 1)[:v.shape[0], :v.shape[1]]
    return v * s


@pytest.mark.parametrize("yd", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(1, 16, 128), (1, 1, 1), (3, 200, 100), (16, 128, 256), (33, 130, 1000),
                                   (64, 300, 1024), (65, 257, 129), (130, 256, 640), (300, 384, 512), (257, 515, 2176),
                                   (513, 260, 136), (2, 1024, 5120), (600, 512, 384), (40, 1000, 4100),
                                   (33, 130, 1008), (5, 64, 144), (17, 40, 16), (1, 30, 17408), (1, 20, 33280), (2, 24, 20608),
                                   (1, 40, 96), (1, 33, 33), (2, 70, 5001), (1, 4100, 1000), (1, 9, 31), (2, 20, 161),
                                   (3, 50, 640), (4200, 260, 256), (700, 2050, 128)])
def test_fp8_matmul(gq, M, N, K, yd):
    rng = np.random.default_rng(M + N + K)
    xq, xs = _pack8(gq, _x(rng, M, K, torch.float32), 1)
    wq, ws = _pack8(gq, _x(rng, N, K, torch.float32) * 0.02, 128)
    y = torch.full((M, N + 3), 7.0, dtype=DT[yd], device=DEV)
    gq.fp8_matmul(y[:, :N], xq, xs, wq, ws)
    x, w = _deq8(xq, xs, 1), _deq8(wq, ws, 128)
    _check(y[:, :N], x @ w.T, np.abs(x) @ np.abs(w).T, K, cut=2.0 ** -10 if yd == "bf16" else 0.0)
    assert (y[:, N:] == 7.0).all()


@pytest.mark.parametrize("yd", ["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(4090, 2810, 384), (4090, 2810, 128), (4090, 2810, 200)])
def test_fp8_matmul_large_tile(gq, M, N, K, yd):
    """Enough rows and columns for 256 x 256 tiles (whole blocks of k, bf16), with ragged edges."""
    test_fp8_matmul(gq, M, N, K, yd)


def test_fp8_matmul_experts_large_tile(gq):
    rng = np.random.default_rng(8)
    counts, N, K = [2500, 0, 1700], 2816, 256
    M, off = 4210, np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xq, xs = _pack8(gq, _x(rng, M, K, torch.float32), 1)
    packs = [_pack8(gq, _x(rng, N, K, torch.float32) * 0.02, 128) for _ in counts]
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    gq.fp8_matmul_experts(y, xq, xs, torch.stack([p[0].view(torch.uint8) for p in packs]).view(torch.float8_e4m3fn),
                          torch.stack([p[1] for p in packs]), torch.from_numpy(off).to(DEV))
    x = _deq8(xq, xs, 1)
    for e in (0, 2):
        a, z, w = off[e], off[e + 1], _deq8(*packs[e], 128)
        _check(y[a:z], x[a:z] @ w.T, np.abs(x[a:z]) @ np.abs(w).T, K, e, 2.0 ** -10)
    assert (y[off[-1]:] == 7.0).all()


@pytest.mark.parametrize("yd", ["bf16", "fp32"])
@pytest.mark.parametrize("counts,M", [([0, 5, 0, 17, 1, 40], 63), ([0, 0, 0], 4), ([1] * 70, 70),
                                      ([300, 0, 2, 257], 560), ([0, 700], 700), ([513, 31, 64], 608)])
@pytest.mark.parametrize("N,K", [(136, 256), (300, 200)])
def test_fp8_matmul_experts(gq, counts, M, N, K, yd):
    rng = np.random.default_rng(M)
    E = len(counts)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    xq, xs = _pack8(gq, _x(rng, M, K, torch.float32), 1)
    packs = [_pack8(gq, _x(rng, N, K, torch.float32) * 0.02, 128) for _ in range(E)]
    y = torch.full((M, N), 7.0, dtype=DT[yd], device=DEV)
    gq.fp8_matmul_experts(y, xq, xs, torch.stack([p[0].view(torch.uint8) for p in packs]).view(torch.float8_e4m3fn),
                          torch.stack([p[1] for p in packs]), torch.from_numpy(off).to(DEV))
    x = _deq8(xq, xs, 1)
    for e in range(E):
        a, z = off[e], off[e + 1]
        if z > a:
            w = _deq8(*packs[e], 128)
            _check(y[a:z], x[a:z] @ w.T, np.abs(x[a:z]) @ np.abs(w).T, K, e, 2.0 ** -10 if yd == "bf16" else 0.0)
    assert (y[off[-1]:] == 7.0).all()


@pytest.mark.parametrize("K", [256, 250])
@pytest.mark.parametrize("M", [2, 20, 300])
def test_fp8_matmul_nan_stays_in_its_row(gq, M, K):
    rng = np.random.default_rng(4)
    x = _x(rng, M, K, torch.float32)
    x[1, 200] = float("nan")
    xq, xs = _pack8(gq, x, 1)
    wq, ws = _pack8(gq, _x(rng, 256, K, torch.float32), 128)
    y = torch.zeros(M, 256, device=DEV)
    gq.fp8_matmul(y, xq, xs, wq, ws)
    assert torch.isnan(y[1]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


# ------------------------------------------------------------------ streams, graphs, refusals with device tensors
def test_products_follow_the_packs_and_the_current_stream(gq):
    """gptq's and rtn's own packs (int4 and NF4) through the product on a side stream, twice: the same bits."""
    rng = np.random.default_rng(6)
    N, K, G, M = 256, 512, 128, 40
    W = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32) * 0.02).to(DEV)
    x = _x(rng, M, K, torch.bfloat16).to(DEV)
    for flags in (0, gq.GQ_NF4):
        codes = torch.empty(N, K // 2, dtype=torch.uint8, device=DEV)
        scales = torch.empty(N, K // G, device=DEV)
        gq.rtn_quantize_ex(codes, scales, W, None, G, flags, gq.workspace(gq.rtn_quantize_workspace_size(N, K, G), DEV))
        torch.cuda.synchronize()
        ys = [torch.empty(M, N, device=DEV) for _ in range(2)]
        s = torch.cuda.Stream()
        for y in ys:
            with torch.cuda.stream(s):
                gq.int4_matmul(y, x, codes, scales, G, flags)
        s.synchronize()
        assert torch.equal(ys[0], ys[1])
        w = _deq4(gq, codes.cpu().numpy(), scales.cpu().numpy(), G, flags != 0)
        x64 = x.double().cpu().numpy()
        _check(ys[0], x64 @ w.T, np.abs(x64) @ np.abs(w).T, K)
        # the pack is an approximation of W: half a step of the int4 grid, or of NF4's widest gap, at most
        err = np.abs(w - W.cpu().numpy().astype(np.float64))
        step = np.repeat(scales.cpu().numpy().astype(np.float64), G, 1) * (0.152 if flags else 0.5)
        assert (err <= step * (1 + 1e-5)).all()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_products_in_a_graph(gq, M):
    """Captured once, replayed several times on new inputs with eager work between: each replay equals the eager call."""
    rng = np.random.default_rng(7)
    N, K, G = 300, 512, 128
    codes, scales = (torch.from_numpy(a).to(DEV) for a in _pack4(rng, N, K, G))
    wq, ws = _pack8(gq, _x(rng, N, K, torch.float32), 128)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV)
    xq, xs = torch.zeros(M, K, dtype=torch.float8_e4m3fn, device=DEV), torch.zeros(M, K // 128, device=DEV)
    y4, y8 = torch.zeros(M, N, device=DEV), torch.zeros(M, N, device=DEV)

    def calls():
        gq.int4_matmul(y4, x, codes, scales, G)
        gq.fp8_quantize(xq, xs, x, 1)
        gq.fp8_matmul(y8, xq, xs, wq, ws)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for i in range(4):
        x.copy_(_x(rng, M, K, torch.bfloat16))
        calls()
        torch.cuda.synchronize()
        want = y4.clone(), y8.clone()
        y4.zero_()
        y8.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y4, want[0]) and torch.equal(y8, want[1]), i


def test_binding_refuses_wrong_shapes(gq):
    z = lambda *s, dt=torch.float32: torch.zeros(*s, device=DEV).to(dt)       # noqa: E731
    u8, f8, i32 = torch.uint8, torch.float8_e4m3fn, torch.int32
    bad = [
        lambda: gq.int4_matmul(z(2, 8), z(3, 64), z(8, 32, dt=u8), z(8, 2), 32),
        lambda: gq.int4_matmul(z(2, 8), z(2, 64), z(8, 31, dt=u8), z(8, 2), 32),
        lambda: gq.int4_matmul(z(2, 8), z(2, 64), z(8, 32, dt=u8), z(8, 1), 32),
        lambda: gq.int4_matmul(z(2, 8), z(2, 64, dt=torch.float16), z(8, 32, dt=u8), z(8, 2), 32),
        lambda: gq.int4_matmul(z(8, 2).t(), z(2, 64), z(8, 32, dt=u8), z(8, 2), 32),
        lambda: gq.int4_matmul(z(2, 8), z(1, 64).expand(2, 64), z(8, 32, dt=u8), z(8, 2), 32),
        lambda: gq.int4_matmul(z(2, 8), z(2, 64), z(8, 32, dt=u8), z(8, 2), 0),
        lambda: gq.int4_matmul_experts(z(2, 8), z(2, 64), z(3, 8, 32, dt=u8), z(3, 8, 2), z(3, dt=i32), 32),
        lambda: gq.fp8_quantize(z(4, 64, dt=f8), z(4, 2), z(4, 64), 1),
        lambda: gq.fp8_quantize(z(4, 64, dt=f8), z(1, 1), z(4, 64), 64),
        lambda: gq.fp8_quantize(z(4, 64, dt=u8), z(4, 1), z(4, 64), 1),
        lambda: gq.fp8_matmul(z(2, 8), z(2, 64, dt=f8), z(2, 1), z(8, 63, dt=f8), z(1, 1)),
        lambda: gq.fp8_matmul(z(2, 8), z(2, 64, dt=f8), z(1, 1), z(8, 64, dt=f8), z(1, 1)),
        lambda: gq.fp8_matmul_experts(z(2, 8), z(2, 64, dt=f8), z(2, 1), z(3, 8, 64, dt=f8), z(2, 1, 1), z(4, dt=i32)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, gq.GQError)):
            call()
            pytest.fail(f"call {i} was accepted")

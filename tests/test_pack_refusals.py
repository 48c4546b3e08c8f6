"""Refusals of the pack products and the expert rows (int4_matmul, fp8_quantize,
fp8_matmul, experts_*): every bad argument is turned down before anything is
launched, so these run without a GPU.  The device pointers are never followed."""
import os

import pytest
import torch

import post_weight_quantization_accumulate_amd as gq

pytestmark = pytest.mark.skipif(not os.path.exists(gq.LIB_PATH), reason="libgq.so not built")

P = 4096            # stands for a device pointer
BAD = gq.GQ_ERR_INVALID_ARG

INT4 = dict(Y=P, yd=gq.GQ_BF16, ldy=64, X=P, xd=gq.GQ_BF16, ldx=128, codes=P, scales=P, M=4, N=64, K=128, group=32,
            flags=0)
INT4E = dict(Y=P, yd=gq.GQ_BF16, ldy=64, X=P, xd=gq.GQ_BF16, ldx=128, codes=P, scales=P, offsets=P, E=4, M=4, N=64,
             K=128, group=32, flags=0)
PACK = dict(codes=P, scales=P, X=P, xd=gq.GQ_F32, ldx=100, rows=7, K=100, block_rows=128)
FP8 = dict(Y=P, yd=gq.GQ_BF16, ldy=64, Xq=P, xs=P, Wq=P, ws=P, M=4, N=64, K=100)
FP8E = dict(Y=P, yd=gq.GQ_BF16, ldy=64, Xq=P, xs=P, Wq=P, ws=P, offsets=P, E=4, M=4, N=64, K=100)
SORT = dict(offsets=P, order=P, pos=P, ids=P, id_bytes=4, n=1 << 16, E=8, ws=P, ws_bytes=1 << 20)
GATHER = dict(Xs=P, ldxs=16, X=P, ldx=16, dtype=gq.GQ_F32, pos=P, rows=8, T=4, k=2, D=16)
COMBINE = dict(out=P, ldo=16, Y=P, ldy=16, dtype=gq.GQ_F32, pos=P, weights=P, rows=8, T=4, k=2, D=16)
BACK = dict(dY=P, lddy=16, dw=P, dout=P, ldo=16, Y=P, ldy=16, dtype=gq.GQ_F32, pos=P, weights=P, rows=8, T=4, k=2,
            D=16)

ROWS = [dict(dtype=2), dict(dtype=-1), dict(T=-1), dict(k=0), dict(rows=-1), dict(D=0), dict(ldy=15, ldx=15),
        dict(pos=None), dict(T=1 << 30, k=4), dict(k=1 << 33), dict(rows=1 << 32)]
CASES = [
    ("int4_matmul", INT4, [dict(flags=8), dict(yd=2), dict(xd=-1), dict(M=-1), dict(N=0), dict(K=127), dict(K=0),
                           dict(group=0), dict(group=3), dict(group=256), dict(K=96, group=64), dict(ldx=127),
                           dict(ldy=63), dict(Y=None), dict(X=None), dict(codes=None), dict(scales=None),
                           dict(M=1 << 32), dict(N=1 << 30, ldy=1 << 30), dict(K=1 << 30, ldx=1 << 30)]),
    ("int4_matmul_experts", INT4E, [dict(E=0), dict(E=gq.GQ_MAX_EXPERTS + 1), dict(offsets=None), dict(ldx=127),
                                    dict(X=None), dict(group=256)]),
    ("fp8_quantize", PACK, [dict(xd=2), dict(block_rows=64), dict(block_rows=0), dict(rows=-1), dict(K=0),
                            dict(ldx=99), dict(codes=None), dict(scales=None), dict(X=None), dict(rows=1 << 32),
                            dict(K=1 << 30, ldx=1 << 30)]),
    ("fp8_matmul", FP8, [dict(yd=7), dict(M=-1), dict(N=0), dict(K=0), dict(ldy=63), dict(Y=None), dict(Xq=None),
                         dict(xs=None), dict(Wq=None), dict(ws=None), dict(M=1 << 32), dict(N=1 << 30, ldy=1 << 30),
                         dict(K=1 << 30)]),
    ("fp8_matmul_experts", FP8E, [dict(E=0), dict(E=gq.GQ_MAX_EXPERTS + 1), dict(offsets=None), dict(Xq=None)]),
    ("experts_sort", SORT, [dict(id_bytes=2), dict(n=-1), dict(n=1 << 31), dict(E=0), dict(E=gq.GQ_MAX_EXPERTS + 1),
                            dict(offsets=None), dict(order=None), dict(pos=None), dict(ids=None), dict(ws=None),
                            dict(ws_bytes=4)]),
    ("experts_gather", GATHER, ROWS + [dict(ldxs=15), dict(Xs=None), dict(X=None)]),
    ("experts_combine", COMBINE, [r for r in ROWS if "ldx" not in r] + [dict(ldo=15), dict(ldy=15), dict(out=None), dict(Y=None)]),
    ("experts_combine_backward", BACK, [r for r in ROWS if "ldx" not in r] + [dict(lddy=15), dict(ldo=15), dict(ldy=15), dict(dY=None),
                                               dict(dw=None), dict(dout=None), dict(Y=None), dict(weights=None)]),
]


@pytest.mark.parametrize("name,base,bad", [(n, b, x) for n, b, xs in CASES for x in xs])
def test_bad_arguments_are_refused(name, base, bad):
    args = {**base, **{k: v for k, v in bad.items() if k in base}}
    assert getattr(gq.lib(), name)(*args.values(), None) == BAD
    assert gq.lib().gq_last_error() != b""


@pytest.mark.parametrize("name,base,empty", [
    ("int4_matmul", INT4, dict(M=0, X=None, Y=None)), ("int4_matmul_experts", INT4E, dict(M=0, X=None, Y=None)),
    ("fp8_quantize", PACK, dict(rows=0, X=None)), ("fp8_matmul", FP8, dict(M=0, Y=None)),
    ("experts_gather", GATHER, dict(T=0, pos=None)), ("experts_gather", GATHER, dict(rows=0, Xs=None)),
    ("experts_combine", COMBINE, dict(T=0, out=None)), ("experts_combine_backward", BACK, dict(T=0, dout=None))])
def test_nothing_to_do_is_ok(name, base, empty):
    assert getattr(gq.lib(), name)(*{**base, **empty}.values(), None) == gq.GQ_OK
    assert gq.lib().gq_last_error() == b""


def test_sort_workspace_size():
    for n, E in [(0, 1), (1, 1), (64, 8), (1 << 20, 1024)]:
        assert 0 <= gq.experts_sort_workspace_size(n, E) <= 4 * (E + 1) * (n // 1024 + 2)
    assert gq.experts_sort_workspace_size(5, 0) == gq.experts_sort_workspace_size(-1, 4) == 0


def _t(*shape, dtype=torch.float32):
    return torch.zeros(*shape).to(dtype)


def test_binding_refuses_host_tensors():
    f8, i32 = torch.float8_e4m3fn, torch.int32
    calls = [
        lambda: gq.int4_matmul(_t(2, 8), _t(2, 64), _t(8, 32, dtype=torch.uint8), _t(8, 2), 32),
        lambda: gq.int4_matmul_experts(_t(2, 8), _t(2, 64), _t(3, 8, 32, dtype=torch.uint8), _t(3, 8, 2),
                                       _t(4, dtype=i32), 32),
        lambda: gq.fp8_quantize(_t(2, 8, dtype=f8), _t(2, 1), _t(2, 8), 1),
        lambda: gq.fp8_matmul(_t(2, 8), _t(2, 8, dtype=f8), _t(2, 1), _t(8, 8, dtype=f8), _t(1, 1)),
        lambda: gq.fp8_matmul_experts(_t(2, 8), _t(2, 8, dtype=f8), _t(2, 1), _t(3, 8, 8, dtype=f8), _t(3, 1, 1),
                                      _t(4, dtype=i32)),
        lambda: gq.experts_sort(_t(4, dtype=i32), _t(6, dtype=i32), _t(2, 3, dtype=i32), _t(2, 3, dtype=i32),
                                _t(4096, dtype=torch.uint8)),
        lambda: gq.experts_gather(_t(6, 8), _t(2, 8), _t(2, 3, dtype=i32)),
        lambda: gq.experts_combine(_t(2, 8), _t(6, 8), _t(2, 3, dtype=i32)),
        lambda: gq.experts_combine_backward(_t(6, 8), _t(2, 3), _t(2, 8), _t(6, 8), _t(2, 3, dtype=i32), _t(2, 3)),
    ]
    for call in calls:
        with pytest.raises(ValueError, match="must be a CUDA"):
            call()

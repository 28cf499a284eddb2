"""Refusals of the norms' and the 8-bit operators' entry points, on the host and before any launch."""
import ctypes

import pytest

from mixture_experts_routed_04_b200 import binding as b
from mixture_experts_routed_04_b200.build import build

INVALID, TOO_SMALL, UNSUPPORTED, MISALIGNED = 1, 2, 3, 5
P = ctypes.c_void_p(4096)  # an aligned address that no call here may reach


@pytest.fixture(scope="module")
def lib():
    build()
    return b.lib()


def norm(lib, p, x=P, y=P, q8=None, s8=None):
    return lib.moe_norm_forward(ctypes.byref(p), x, None, None, y, q8, s8, None, None, None)


@pytest.mark.parametrize("over,status", [
    (dict(T=-1), INVALID), (dict(d=0), INVALID), (dict(d=b.NORM_MAX_D + 1), UNSUPPORTED), (dict(kind=3), INVALID),
    (dict(kind=b.NORM_NONE), INVALID), (dict(next_kind=b.NORM_RMS), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(alpha=float("inf")), INVALID), (dict(stream_dtype=b.DT_E4M3), INVALID),
    (dict(block_dtype=-1), INVALID), (dict(param_dtype=4), INVALID), (dict(gate_kind=b.GATE_TOKEN), INVALID),
    (dict(ld_stream=63), INVALID), (dict(ld_block=1), INVALID)])
def test_norm_params(lib, over, status):
    kw = dict(T=4, d=64)
    kw.update(over)
    p = b.norm_params(**kw)
    assert norm(lib, p) == status
    if "kind" not in over and "next_kind" not in over and "gate_kind" not in over:
        assert lib.moe_norm_workspace_size(ctypes.byref(p)) == 0


def test_norm_buffers(lib):
    p = b.norm_params(4, 64)
    assert norm(lib, p, x=None) == INVALID
    assert norm(lib, p, y=None) == INVALID                       # neither y nor q8
    assert norm(lib, p, q8=P) == INVALID                         # q8 without its scales
    assert norm(lib, b.norm_params(4, 64, block_dtype=b.DT_BF16)) == INVALID  # in place over rows of another type
    assert norm(lib, b.norm_params(4, 64, block_dtype=b.DT_F32, ld_block=72)) == INVALID  # or of another stride
    assert norm(lib, p, x=ctypes.c_void_p(4098)) == MISALIGNED   # fp32 at an odd half word
    assert norm(lib, p, q8=ctypes.c_void_p(4100), s8=P) == MISALIGNED
    assert norm(lib, b.norm_params(4, 24), q8=P, s8=P) == INVALID
    assert norm(lib, b.norm_params(4, 64, ld_stream=65), q8=P, s8=P) == MISALIGNED  # rows off 16 bytes
    back = lambda p, g, ws=P, n=1 << 30, mean=P, w=P: lib.moe_norm_backward(  # noqa: E731
        ctypes.byref(p), P, w, P, None, mean, P, P, ctypes.byref(g), ws, n, None)
    dw = b.NormGrads(4096, None, None)
    assert back(p, b.NormGrads(None, None, 4096)) == INVALID     # no gate before the block
    assert back(p, dw, ws=None) == INVALID
    assert back(p, dw, n=256) == TOO_SMALL
    assert back(p, dw, ws=ctypes.c_void_p(4112)) == MISALIGNED
    assert back(p, dw, w=None) == INVALID                        # a weight's gradient without a weight
    assert back(b.norm_params(4, 64, kind=b.NORM_LAYER), dw, mean=None) == INVALID


def test_norm_residual_buffers(lib):
    def fwd(p, w=None, gate=None, nw=None, xn=None, m=None):
        return lib.moe_norm_residual_forward(ctypes.byref(p), P, P, w, None, gate, None, m, None, nw, None, xn, None,
                                             None, None, None, None)
    assert fwd(b.norm_params(4, 64)) == INVALID                                         # no out
    assert fwd(b.norm_params(4, 64, kind=b.NORM_NONE), w=P) == INVALID                  # a weight without a norm
    assert fwd(b.norm_params(4, 64, kind=b.NORM_NONE), m=P) == INVALID
    assert fwd(b.norm_params(4, 64), xn=P) == INVALID                                   # a result without its norm
    assert fwd(b.norm_params(4, 64), gate=P) == INVALID
    assert fwd(b.norm_params(4, 64, gate_kind=b.GATE_TOKEN)) == INVALID
    back = lambda p, g, bias=None, gate=None, w=P: lib.moe_norm_residual_backward(  # noqa: E731
        ctypes.byref(p), P, w, bias, gate, P, P, P, None, P, ctypes.byref(g), P, 1 << 30, None)
    assert back(b.norm_params(4, 64), b.NormGrads(None, 4096, None)) == INVALID         # dbias without a bias
    assert back(b.norm_params(4, 64), b.NormGrads(None, None, 4096)) == INVALID         # dgate without a gate
    assert back(b.norm_params(4, 64, gate_kind=b.GATE_TOKEN), b.NormGrads(None, None, 4096)) == INVALID
    assert back(b.norm_params(4, 64, kind=b.NORM_NONE), b.NormGrads(4096, None, None), w=None) == INVALID


def test_empty_batches_need_no_buffers(lib):
    p = b.norm_params(0, 64)
    assert norm(lib, p, x=None, y=None) == 0
    assert lib.moe_norm_workspace_size(ctypes.byref(p)) >= 256
    q = b.f8_params(0, 64, 64)
    assert lib.moe_matmul_f8(ctypes.byref(q), None, None, None, None, None, None, None, None, P, 256, None) == 0
    assert lib.moe_quantize_f8(0, 64, None, b.DT_F32, 0, 0, None, None, None, None, P, 256, None) == 0


@pytest.mark.parametrize("over", [dict(rows=-1), dict(rows=1 << 31), dict(K=8), dict(K=24), dict(N=4), dict(N=12), dict(E=0),
                                  dict(E=257), dict(out_dtype=4), dict(variant=3), dict(swiglu_limit=float("nan")),
                                  dict(N=1 << 24, E=256), dict(N=(1 << 31) - 8)])
def test_f8_params(lib, over):
    kw = dict(rows=4, K=64, N=64)
    kw.update(over)
    p = b.f8_params(**kw)
    assert lib.moe_f8_workspace_size(ctypes.byref(p)) == 0
    assert lib.moe_matmul_f8(ctypes.byref(p), P, P, P, P, P, None, None, P, P, 256, None) == INVALID
    assert lib.moe_gated_f8(ctypes.byref(p), P, P, P, P, P, P, P, P, None, P, 256, None) == INVALID


def test_f8_buffers(lib):
    odd = ctypes.c_void_p(4104)

    def mm(p, a=P, off=None, w=P, sw=P, sp=None, tw=None, out=P, ws=P, n=256):
        return lib.moe_matmul_f8(ctypes.byref(p), a, P, off, w, sw, sp, tw, out, ws, n, None)
    p = b.f8_params(4, 64, 64)
    assert mm(b.f8_params(4, 64, 64, out_dtype=b.DT_E4M3)) == UNSUPPORTED
    assert mm(p, a=None) == INVALID and mm(p, w=None) == INVALID and mm(p, sw=None) == INVALID and mm(p, out=None) == INVALID
    assert mm(p, a=odd) == MISALIGNED and mm(p, w=odd) == MISALIGNED and mm(p, out=odd) == MISALIGNED
    assert mm(p, ws=None) == INVALID and mm(p, ws=odd) == MISALIGNED and mm(p, n=128) == TOO_SMALL
    assert mm(p, sp=P) == INVALID and mm(p, tw=P) == INVALID                 # one without the other
    assert mm(b.f8_params(4, 64, 64, E=2)) == INVALID                        # experts without offsets

    def gt(p, hs=None, h=P):
        return lib.moe_gated_f8(ctypes.byref(p), P, P, None, P, P, P, P, h, hs, P, 256, None)
    assert gt(p, hs=P) == INVALID                                            # scales of a 16-bit result
    assert gt(b.f8_params(4, 64, 64, out_dtype=b.DT_E4M3)) == INVALID        # an e4m3 result without scales
    assert gt(b.f8_params(4, 64, 72, out_dtype=b.DT_E4M3), hs=P) == INVALID  # rows of 72 bytes

    def rows(rows=4, K=64, x=P, dt=b.DT_BF16, ld=0, src=4, q=P, s=P, ws=P, n=256, idx=None):
        return lib.moe_quantize_f8(rows, K, x, dt, ld, src, idx, None, q, s, ws, n, None)
    assert rows(rows=-1) == INVALID and rows(K=24) == INVALID and rows(dt=b.DT_E4M3) == INVALID and rows(ld=63) == INVALID
    assert rows(src=3) == INVALID and rows(x=None) == INVALID and rows(q=None) == INVALID and rows(s=None) == INVALID
    assert rows(q=odd) == MISALIGNED and rows(x=ctypes.c_void_p(4097)) == MISALIGNED
    assert rows(ws=None) == INVALID and rows(n=4) == TOO_SMALL

    def weights(E=1, N=64, K=64, w=P, dt=b.DT_BF16, t=0, q=P):
        return lib.moe_quantize_f8_weights(E, N, K, w, dt, t, q, P, None)
    assert weights(E=0) == INVALID and weights(N=12) == INVALID and weights(K=24) == INVALID and weights(t=2) == INVALID
    assert weights(N=(1 << 31) - 8) == INVALID
    assert weights(w=None) == INVALID and weights(q=odd) == MISALIGNED and weights(dt=3) == INVALID


def test_f8_selftest_arguments(lib):
    def run(gated=0, blocks=3, limit=1000, ws=P, n=b.F8_SELFTEST_BYTES):
        return lib.moe_f8_wait_selftest(gated, blocks, limit, ws, n, None)
    assert run(blocks=-1) == INVALID and run(blocks=8) == INVALID and run(limit=0) == INVALID and run(limit=10 ** 11) == INVALID
    assert run(ws=None) == INVALID and run(ws=ctypes.c_void_p(4112)) == MISALIGNED and run(n=1 << 19) == TOO_SMALL

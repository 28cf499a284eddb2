"""Thin Python binding of the C ABI in ``include/moe.h`` (ctypes).

Argument marshalling only: every step of the layer runs in the CUDA kernels of
``libmoe_b200.so``. PyTorch supplies device memory and the current stream. If
the library has not been built, loading it raises ``MoeError``; there is no
fallback of any kind.

Tensors are passed by ``data_ptr()``: x and bf16 weights as ``torch.bfloat16``
(or int16 bit patterns), y_rows as ``torch.float16``, the layer output as
``torch.float32`` (default) or ``torch.bfloat16`` (out_dtype=OUT_BF16). Calls are asynchronous on
``torch.cuda.current_stream()`` unless a stream is given.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_b200.so")

MOE_OK = 0
MOE_ERR_DEVICE = 6  # moe_get_error: the device error word is set
STATUS = {0: "ok", 1: "invalid argument", 2: "workspace too small", 3: "unsupported configuration",
          4: "CUDA error", 5: "misaligned pointer", 6: "device error word set"}
DEVERR_TIMEOUT, DEVERR_BOUNDS, DEVERR_RANGE = 0x1, 0x2, 0x4
OUT_F32, OUT_BF16 = 0, 1
DOWN_BF16, DOWN_F16 = 0, 1
WEIGHTS_BF16, WEIGHTS_Q4G32 = 0, 1
VARIANT_AUTO, VARIANT_TENSOR, VARIANT_STREAM = 0, 1, 2
TILE_AUTO, TILE_ONE, TILE_PAIR = 0, 1, 2
DT_F32, DT_BF16, DT_F16, DT_E4M3 = range(4)
NORM_NONE, NORM_RMS, NORM_LAYER = range(3)
GATE_NONE, GATE_CHANNEL, GATE_TOKEN = range(3)
NORM_MAX_D = 8192  # MOE_NORM_MAX_D
F8_SELFTEST_BYTES = 1 << 20  # MOE_F8_SELFTEST_BYTES
WS_ROUTE, WS_PERMUTE, WS_EXPERT_FFN, WS_COMBINE, WS_FORWARD, WS_FORWARD_HOST, WS_ROUTE_STATS, WS_BACKWARD = range(8)

# every entry point declared in include/moe.h
EXPORTS = ("moe_version", "moe_status_string", "moe_capacity", "moe_max_rows", "moe_workspace_size",
           "moe_route", "moe_permute", "moe_expert_ffn", "moe_combine", "moe_forward", "moe_forward_host",
           "moe_get_error", "moe_clear_error", "moe_set_wait_limit_ns", "moe_launch_count",
           "moe_profile_enable", "moe_profile_collect", "moe_convert_bf16_to_f16",
           "moe_permute_noalloc", "moe_forward_host_async", "moe_wait_selftest", "moe_tile_ctas",
           "moe_route_stats", "moe_expert_ffn_backward", "moe_variant_table",
           "moe_norm_workspace_size", "moe_norm_forward", "moe_norm_backward", "moe_norm_residual_forward",
           "moe_norm_residual_backward", "moe_quantize_f8", "moe_quantize_f8_weights", "moe_f8_workspace_size",
           "moe_matmul_f8", "moe_gated_f8", "moe_f8_wait_selftest")
NOALLOC_MAX_PAIRS = 262144  # MOE_NOALLOC_MAX_PAIRS

# kernel ids (MOE_K_*), in order
KERNELS = ("route", "perm_count", "perm_scan", "perm_scatter", "schedule", "gather", "tc_gateup", "tc_down",
           "stream_gateup", "stream_reduce", "stream_down", "combine", "convert", "front", "route_stats",
           "bwd_gemm", "bwd_small", "norm", "norm_bwd", "quant_f8", "tc_f8", "stream_f8")


class MoeError(RuntimeError):
    pass


class Params(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("E", ctypes.c_int32), ("k", ctypes.c_int32), ("capacity_factor", ctypes.c_float),
                ("swiglu_limit", ctypes.c_float), ("weight_format", ctypes.c_int32),
                ("has_shared", ctypes.c_int32), ("d_ff_shared", ctypes.c_int32),
                ("variant", ctypes.c_int32), ("stream_max_rows", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("down_dtype", ctypes.c_int32), ("tile_ctas", ctypes.c_int32)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
                                               "shared_gate", "shared_up", "shared_down")]


class Grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dx", "dw_gate", "dw_up", "dw_down", "d_topk_w", "dlogits",
                                               "dshared_gate", "dshared_up", "dshared_down")]


class NormParams(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("kind", ctypes.c_int32), ("next_kind", ctypes.c_int32),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float), ("stream_dtype", ctypes.c_int32),
                ("block_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32), ("gate_kind", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("ld_stream", ctypes.c_int64),
                ("ld_block", ctypes.c_int64)]


class NormGrads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("dweight", "dbias", "dgate")]


class F8Params(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("E", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("swiglu_limit", ctypes.c_float), ("variant", ctypes.c_int32)]


_lib = None
_P, _V, _S = ctypes.POINTER(Params), ctypes.c_void_p, ctypes.c_size_t


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MoeError(f"{LIB_PATH} is not built; run `python -m mixture_experts_routed_04_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "moe_version": ([], ctypes.c_int),
            "moe_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "moe_capacity": ([_P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
            "moe_max_rows": ([_P, ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
            "moe_tile_ctas": ([_P, ctypes.POINTER(ctypes.c_int32)], ctypes.c_int),
            "moe_workspace_size": ([_P, ctypes.c_int], _S),
            "moe_route": ([_P, _V, _V, _V, _V, _S, _V], ctypes.c_int),
            "moe_route_stats": ([_P, _V, _V, _V, ctypes.c_float, _V, _V, _V, _V, _V, _S, _V], ctypes.c_int),
            "moe_permute": ([_P, _V, _V, _V, _V, _V, _V, _V, _V, _S, _V], ctypes.c_int),
            "moe_expert_ffn": ([_P, _V, _V, _V, _V, _V, ctypes.POINTER(Weights), _V, _V, _S, _V], ctypes.c_int),
            "moe_combine": ([_P, _V, _V, _V, _V, _V, _S, _V], ctypes.c_int),
            "moe_forward": ([_P, _V, _V, ctypes.POINTER(Weights), _V, _V, _V, _S, _V], ctypes.c_int),
            "moe_forward_host": ([_P, _V, _V, ctypes.POINTER(Weights), _V, _V, _S, _V], ctypes.c_int),
            "moe_forward_host_async": ([_P, _V, _V, ctypes.POINTER(Weights), _V, _V, _S, _V], ctypes.c_int),
            "moe_wait_selftest": ([_V, ctypes.c_uint64, _V], ctypes.c_int),
            "moe_get_error": ([_V, ctypes.POINTER(ctypes.c_uint32), _V], ctypes.c_int),
            "moe_clear_error": ([_V, _V], ctypes.c_int),
            "moe_set_wait_limit_ns": ([ctypes.c_uint64], ctypes.c_int),
            "moe_launch_count": ([_P, ctypes.c_int, ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
            "moe_profile_enable": ([ctypes.c_int], ctypes.c_int),
            "moe_profile_collect": ([ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
            "moe_convert_bf16_to_f16": ([_V, _V, ctypes.c_int64, _V, _V], ctypes.c_int),
            "moe_permute_noalloc": ([_P, _V, _V, _V, _V, _V, _V, _V, _V, _V], ctypes.c_int),
            "moe_variant_table": ([ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int32), ctypes.c_int],
                                  ctypes.c_int),
            "moe_expert_ffn_backward": ([_P, _V, _V, _V, _V, _V, _V, _V, ctypes.POINTER(Weights), _V,
                                         ctypes.POINTER(Grads), _V, _S, _V], ctypes.c_int),
        }
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        N, G, F = ctypes.POINTER(NormParams), ctypes.POINTER(NormGrads), ctypes.POINTER(F8Params)
        sig.update({
            "moe_norm_workspace_size": ([N], _S),
            "moe_norm_forward": ([N] + [_V] * 9, ctypes.c_int),
            "moe_norm_backward": ([N] + [_V] * 7 + [G, _V, _S, _V], ctypes.c_int),
            "moe_norm_residual_forward": ([N] + [_V] * 16, ctypes.c_int),
            "moe_norm_residual_backward": ([N] + [_V] * 9 + [G, _V, _S, _V], ctypes.c_int),
            "moe_quantize_f8": ([i64, i32, _V, i32, i64, i64, _V, _V, _V, _V, _V, _S, _V], ctypes.c_int),
            "moe_quantize_f8_weights": ([i32, i32, i32, _V, i32, i32, _V, _V, _V], ctypes.c_int),
            "moe_f8_workspace_size": ([F], _S),
            "moe_matmul_f8": ([F] + [_V] * 9 + [_S, _V], ctypes.c_int),
            "moe_gated_f8": ([F] + [_V] * 10 + [_S, _V], ctypes.c_int),
            "moe_f8_wait_selftest": ([i32, i32, ctypes.c_uint64, _V, _S, _V], ctypes.c_int),
        })
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _lib = L
    return _lib


def params(T, d_model, d_ff, E, k, capacity_factor=0.0, swiglu_limit=7.0, weight_format=WEIGHTS_BF16,
           has_shared=0, d_ff_shared=0, variant=VARIANT_AUTO, stream_max_rows=-1, out_dtype=OUT_F32,
           down_dtype=DOWN_BF16, tile_ctas=TILE_AUTO) -> Params:
    return Params(T, d_model, d_ff, E, k, capacity_factor, swiglu_limit, weight_format, int(has_shared),
                  d_ff_shared if has_shared else 0, variant, stream_max_rows, out_dtype, down_dtype, tile_ctas)


def params_for(cfg, **over) -> Params:
    """Params of a ``synth.LayerConfig``-like object (fields T, d, f, E, k, ...)."""
    kw = dict(T=cfg.T, d_model=cfg.d, d_ff=cfg.f, E=cfg.E, k=cfg.k, capacity_factor=cfg.capacity_factor,
              swiglu_limit=cfg.swiglu_limit,
              weight_format=WEIGHTS_Q4G32 if cfg.weight_format == "q4g32" else WEIGHTS_BF16,
              has_shared=int(cfg.has_shared), d_ff_shared=cfg.f_shared)
    kw.update(over)
    return params(**kw)


def check(status: int, what: str = "") -> None:
    if status != MOE_OK:
        raise MoeError(f"{what}: {STATUS.get(status, status)}")


def _p(t):
    return None if t is None else t.data_ptr()  # the prototypes make it a void*


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    import torch
    # the raw handle: building the Stream object of torch.cuda.current_stream() takes longer than a launch
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def capacity(p: Params):
    v = ctypes.c_int32()
    check(lib().moe_capacity(ctypes.byref(p), ctypes.byref(v)), "moe_capacity")
    return None if v.value < 0 else v.value


def tile_ctas(p: Params) -> int:
    """SMs per tcgen05 tile these params use (TILE_ONE or TILE_PAIR)."""
    v = ctypes.c_int32()
    check(lib().moe_tile_ctas(ctypes.byref(p), ctypes.byref(v)), "moe_tile_ctas")
    return v.value


def max_rows(p: Params) -> int:
    v = ctypes.c_int64()
    check(lib().moe_max_rows(ctypes.byref(p), ctypes.byref(v)), "moe_max_rows")
    return v.value


def workspace_size(p: Params, which: int) -> int:
    return int(lib().moe_workspace_size(ctypes.byref(p), which))


def workspace(p: Params, which: int, device="cuda"):
    """A zeroed device workspace of the size `which` needs (256-byte aligned)."""
    import torch
    n = workspace_size(p, which)
    if n == 0:
        raise MoeError("invalid parameters")
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def weights(w_gate, w_up, w_down, s_gate=None, s_up=None, s_down=None, shared=None) -> Weights:
    sh = shared or (None, None, None)
    W = Weights(*(None if t is None else t.data_ptr() for t in (w_gate, w_up, w_down, s_gate, s_up, s_down, *sh)))
    W._keep = (w_gate, w_up, w_down, s_gate, s_up, s_down, *sh)  # keep the tensors alive
    return W


def route(p, logits, topk_idx, topk_w, ws, stream=None):
    check(lib().moe_route(ctypes.byref(p), _p(logits), _p(topk_idx), _p(topk_w), _p(ws), ws.numel(),
                          _stream(stream)), "moe_route")


STATS = ("kept", "want_k", "balance", "z", "aux")  # moe_route_stats stats[0..4]


def route_stats(p, logits, topk_idx, topk_w, stats, ws, z_weight=1e-3, kept_tok=None, want_tok=None,
                expert_stats=None, stream=None):
    """moe_route_stats: moe_route plus the router telemetry (stats: device fp32 [5], see STATS)."""
    check(lib().moe_route_stats(ctypes.byref(p), _p(logits), _p(topk_idx), _p(topk_w), float(z_weight), _p(stats),
                                _p(kept_tok), _p(want_tok), _p(expert_stats), _p(ws), ws.numel(),
                                _stream(stream)), "moe_route_stats")


def permute(p, topk_idx, counts, kept, offsets, sorted_token, sorted_pair, pair_row, ws, stream=None):
    check(lib().moe_permute(ctypes.byref(p), _p(topk_idx), _p(counts), _p(kept), _p(offsets), _p(sorted_token),
                            _p(sorted_pair), _p(pair_row), _p(ws), ws.numel(), _stream(stream)), "moe_permute")


def permute_noalloc(p, topk_idx, counts, kept, offsets, sorted_token, sorted_pair, pair_row, err_word,
                    stream=None):
    """moe_permute with the library's fixed scratch array instead of a workspace (one stream only)."""
    check(lib().moe_permute_noalloc(ctypes.byref(p), _p(topk_idx), _p(counts), _p(kept), _p(offsets),
                                    _p(sorted_token), _p(sorted_pair), _p(pair_row), _p(err_word),
                                    _stream(stream)), "moe_permute_noalloc")


def expert_ffn(p, x, offsets, sorted_token, sorted_pair, topk_w, W: Weights, y_rows, ws, stream=None):
    check(lib().moe_expert_ffn(ctypes.byref(p), _p(x), _p(offsets), _p(sorted_token), _p(sorted_pair), _p(topk_w),
                               ctypes.byref(W), _p(y_rows), _p(ws), ws.numel(), _stream(stream)), "moe_expert_ffn")


def combine(p, y_rows, pair_row, offsets, out, ws, stream=None):
    check(lib().moe_combine(ctypes.byref(p), _p(y_rows), _p(pair_row), _p(offsets), _p(out), _p(ws), ws.numel(),
                            _stream(stream)), "moe_combine")


def grads(dx, dw_gate, dw_up, dw_down, d_topk_w, dlogits=None, shared=None) -> Grads:
    sh = shared or (None, None, None)
    ts = (dx, dw_gate, dw_up, dw_down, d_topk_w, dlogits, *sh)
    G = Grads(*(None if t is None else t.data_ptr() for t in ts))
    G._keep = ts
    return G


def expert_ffn_backward(p, x, topk_idx, topk_w, offsets, sorted_token, sorted_pair, pair_row, W: Weights, dout,
                        G: Grads, ws, stream=None):
    """moe_expert_ffn_backward: gradients of the layer for dout (fp32 [T, d]) into G (fp32)."""
    check(lib().moe_expert_ffn_backward(ctypes.byref(p), _p(x), _p(topk_idx), _p(topk_w), _p(offsets),
                                        _p(sorted_token), _p(sorted_pair), _p(pair_row), ctypes.byref(W), _p(dout),
                                        ctypes.byref(G), _p(ws), ws.numel(), _stream(stream)),
          "moe_expert_ffn_backward")


def forward(p, x, logits, W: Weights, out, ws, counts_out=None, stream=None):
    check(lib().moe_forward(ctypes.byref(p), _p(x), _p(logits), ctypes.byref(W), _p(out), _p(counts_out), _p(ws),
                            ws.numel(), _stream(stream)), "moe_forward")


def forward_host(p, x_host, logits_host, W: Weights, out_host, ws, stream=None):
    """moe_forward_host: host (CPU, ideally pinned) x/logits/out; synchronises the stream."""
    check(lib().moe_forward_host(ctypes.byref(p), _p(x_host), _p(logits_host), ctypes.byref(W), _p(out_host),
                                 _p(ws), ws.numel(), _stream(stream)), "moe_forward_host")


def forward_host_async(p, x_host, logits_host, W: Weights, out_host, ws, stream=None):
    """moe_forward_host_async: as forward_host, enqueued on the stream without synchronising."""
    check(lib().moe_forward_host_async(ctypes.byref(p), _p(x_host), _p(logits_host), ctypes.byref(W),
                                       _p(out_host), _p(ws), ws.numel(), _stream(stream)), "moe_forward_host_async")


def wait_selftest(err_ws, limit_ns, stream=None):
    """moe_wait_selftest: a bounded wait on a barrier nothing completes; sets DEVERR_TIMEOUT."""
    check(lib().moe_wait_selftest(_p(err_ws), int(limit_ns), _stream(stream)), "moe_wait_selftest")


def get_error(ws, stream=None) -> int:
    v = ctypes.c_uint32()
    st = lib().moe_get_error(_p(ws), ctypes.byref(v), _stream(stream))
    if st not in (MOE_OK, MOE_ERR_DEVICE):
        check(st, "moe_get_error")
    return v.value


def clear_error(ws, stream=None) -> None:
    check(lib().moe_clear_error(_p(ws), _stream(stream)), "moe_clear_error")


def set_wait_limit_ns(ns: int) -> None:
    check(lib().moe_set_wait_limit_ns(ns), "moe_set_wait_limit_ns")


def variant_table():
    """[(tiles_per_sm, max_rows), ...]: the measured rows of the default variant choice."""
    n = lib().moe_variant_table(None, None, 0)
    a, r = (ctypes.c_float * n)(), (ctypes.c_int32 * n)()
    lib().moe_variant_table(a, r, n)
    return [(float(a[i]), int(r[i])) for i in range(n)]


def launch_count(p: Params, which: int) -> int:
    v = ctypes.c_int()
    check(lib().moe_launch_count(ctypes.byref(p), which, ctypes.byref(v)), "moe_launch_count")
    return v.value


def profile_enable(on: bool = True) -> None:
    check(lib().moe_profile_enable(int(on)), "moe_profile_enable")


def profile_collect() -> dict:
    """{kernel name: (total ms, launches)} since the last collect (waits for the events)."""
    n = len(KERNELS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    check(lib().moe_profile_collect(ms, cnt), "moe_profile_collect")
    return {KERNELS[i]: (ms[i], cnt[i]) for i in range(n)}


def convert_bf16_to_f16(src, dst, err_ws=None, stream=None) -> None:
    """Load-time weight preparation: dst (fp16) = src (bf16), elementwise."""
    assert src.numel() == dst.numel()
    check(lib().moe_convert_bf16_to_f16(_p(src), _p(dst), src.numel(), _p(err_ws), _stream(stream)),
          "moe_convert_bf16_to_f16")


def prepare_down_f16(w_down, stream=None):
    """fp16 copy of a bf16 W_down (or shared W_down), for down_dtype=DOWN_F16."""
    import torch
    out = torch.empty(w_down.shape, dtype=torch.float16, device=w_down.device)
    convert_bf16_to_f16(w_down, out, stream=stream)
    return out


# ------------------------------------------------------------------ norms around a block

def _dt(t) -> int:
    """The library's dtype code of a tensor of 32 or 16 bits."""
    return _dtypes("rows").index(t.dtype)  # MOE_DT_F32, _BF16, _F16


def _fits(what, stream, *specs):
    """Checks tensors given as (name, tensor, shape, dtypes, dense): on the device the call runs on, of
    the shape and one of the dtypes, contiguous where dense is true. None passes."""
    import torch
    dev = torch._C._cuda_getDevice()  # as _stream does: a third of torch.cuda.current_device()'s time
    if stream is not None and stream.device_index != dev:
        raise MoeError(f"{what}: the stream is not on the current device")
    for name, t, shape, dtypes, dense in specs:
        if t is None or (t.get_device() == dev and t.dtype in dtypes and t.shape == shape and
                         (not dense or t.is_contiguous())):
            continue
        if t.get_device() != dev:
            raise MoeError(f"{what}: {name} is on {t.device}, the call runs on cuda:{dev}")
        if t.shape != shape:
            raise MoeError(f"{what}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        raise MoeError(f"{what}: {name} is {t.dtype}" if t.dtype not in dtypes else f"{what}: {name} is not contiguous")


def _ws_spec(ws):
    return "ws", ws, () if ws is None else ws.shape, _dtypes("u8"), True


_dtype_table = None


def _dtypes(code):
    """The torch dtypes a dtype code stands for."""
    global _dtype_table
    if _dtype_table is None:
        import torch
        _dtype_table = {DT_F32: (torch.float32,), DT_BF16: (torch.bfloat16,), DT_F16: (torch.float16,),
                        DT_E4M3: (torch.float8_e4m3fn, torch.uint8), "i32": (torch.int32,), "u8": (torch.uint8,),
                        "rows": (torch.float32, torch.bfloat16, torch.float16)}
    return _dtype_table[code]


def norm_params(T, d, kind=NORM_RMS, next_kind=NORM_NONE, eps=1e-6, weight_offset=0.0, stream_dtype=DT_F32,
                block_dtype=DT_BF16, param_dtype=DT_F32, gate_kind=GATE_NONE, alpha=1.0, beta=1.0, ld_stream=0,
                ld_block=0) -> NormParams:
    return NormParams(T, d, kind, next_kind, eps, weight_offset, stream_dtype, block_dtype, param_dtype, gate_kind,
                      alpha, beta, ld_stream, ld_block)


def norm_workspace(p: NormParams, device="cuda"):
    """A device workspace of the size the norms' backward calls need (256-byte aligned)."""
    import torch
    n = int(lib().moe_norm_workspace_size(ctypes.byref(p)))
    if n == 0:
        raise MoeError("invalid parameters")
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def _norm_grads(dw, db, dgate) -> NormGrads:
    return NormGrads(*(None if t is None else t.data_ptr() for t in (dw, db, dgate)))


def _rows_ok(what, p, ld, **tensors):
    """Row tensors: elements next to each other and the params' stride from row to row."""
    d = p.d
    ld = ld or d
    for name, t in tensors.items():
        if t is None or ld == d and t.is_contiguous():
            continue
        if t.shape[0] > 0 and (t.stride(1) != 1 and t.shape[1] > 1 or t.shape[0] > 1 and t.stride(0) != ld):
            raise MoeError(f"{what}: {name} has strides {t.stride()}, the params say {(ld, 1)}")


def norm_forward(p: NormParams, x, y, weight=None, bias=None, q8=None, s8=None, mean=None, rstd=None, stream=None):
    """moe_norm_forward: y = N(x), the norm before a block; q8, s8: N(x) in e4m3 with its scales."""
    f32, par = _dtypes(DT_F32), _dtypes(p.param_dtype)
    row = (p.T, p.d)
    _fits("moe_norm_forward", stream, ("x", x, row, _dtypes(p.stream_dtype), False),
          ("y", y, row, _dtypes(p.block_dtype), False), ("weight", weight, (p.d,), par, True),
          ("bias", bias, (p.d,), par, True), ("q8", q8, row, _dtypes(DT_E4M3), True),
          ("s8", s8, ((p.d + 127) // 128, p.T), f32, True), ("mean", mean, (p.T,), f32, True),
          ("rstd", rstd, (p.T,), f32, True))
    _rows_ok("moe_norm_forward", p, p.ld_stream, x=x)
    _rows_ok("moe_norm_forward", p, p.ld_block, y=y)
    check(lib().moe_norm_forward(ctypes.byref(p), _p(x), _p(weight), _p(bias), _p(y), _p(q8), _p(s8), _p(mean),
                                 _p(rstd), _stream(stream)), "moe_norm_forward")


def norm_backward(p: NormParams, x, dy, mean, rstd, dx, ws=None, weight=None, dres=None, dw=None, db=None,
                  stream=None):
    """moe_norm_backward: gradients of norm_forward; dres is added to dx. ws: norm_workspace(p)."""
    f32, par = _dtypes(DT_F32), _dtypes(p.param_dtype)
    row, st = (p.T, p.d), _dtypes(p.stream_dtype)
    _fits("moe_norm_backward", stream, ("x", x, row, st, False), ("dy", dy, row, _dtypes(p.block_dtype), False),
          ("dres", dres, row, st, False), ("dx", dx, row, st, False), ("weight", weight, (p.d,), par, True),
          ("mean", mean, (p.T,), f32, True), ("rstd", rstd, (p.T,), f32, True), ("dw", dw, (p.d,), f32, True),
          ("db", db, (p.d,), f32, True), _ws_spec(ws))
    _rows_ok("moe_norm_backward", p, p.ld_stream, x=x, dres=dres, dx=dx)
    _rows_ok("moe_norm_backward", p, p.ld_block, dy=dy)
    check(lib().moe_norm_backward(ctypes.byref(p), _p(x), _p(weight), _p(dy), _p(dres), _p(mean), _p(rstd), _p(dx),
                                  ctypes.byref(_norm_grads(dw, db, None)), _p(ws), 0 if ws is None else ws.numel(),
                                  _stream(stream)), "moe_norm_backward")


def norm_residual_forward(p: NormParams, resid, y, out, weight=None, bias=None, gate=None, mean=None, rstd=None,
                          next_weight=None, next_bias=None, x_next=None, q8=None, s8=None, next_mean=None,
                          next_rstd=None, stream=None):
    """moe_norm_residual_forward: out = alpha resid + beta gate N(y), and x_next = N2(out) with p.next_kind."""
    f32, par = _dtypes(DT_F32), _dtypes(p.param_dtype)
    row, st, bl, tok, vec = (p.T, p.d), _dtypes(p.stream_dtype), _dtypes(p.block_dtype), (p.T,), (p.d,)
    _fits("moe_norm_residual_forward", stream, ("resid", resid, row, st, False), ("y", y, row, bl, False),
          ("out", out, row, st, False), ("x_next", x_next, row, bl, False), ("weight", weight, vec, par, True),
          ("bias", bias, vec, par, True), ("gate", gate, tok if p.gate_kind == GATE_TOKEN else vec, par, True),
          ("next_weight", next_weight, vec, par, True), ("next_bias", next_bias, vec, par, True),
          ("q8", q8, row, _dtypes(DT_E4M3), True), ("s8", s8, ((p.d + 127) // 128, p.T), f32, True),
          ("mean", mean, tok, f32, True), ("rstd", rstd, tok, f32, True), ("next_mean", next_mean, tok, f32, True),
          ("next_rstd", next_rstd, tok, f32, True))
    _rows_ok("moe_norm_residual_forward", p, p.ld_stream, resid=resid, out=out)
    _rows_ok("moe_norm_residual_forward", p, p.ld_block, y=y, x_next=x_next)
    check(lib().moe_norm_residual_forward(ctypes.byref(p), _p(resid), _p(y), _p(weight), _p(bias), _p(gate), _p(out),
                                          _p(mean), _p(rstd), _p(next_weight), _p(next_bias), _p(x_next), _p(q8),
                                          _p(s8), _p(next_mean), _p(next_rstd), _stream(stream)),
          "moe_norm_residual_forward")


def norm_residual_backward(p: NormParams, y, dout, mean, rstd, dy, ws=None, weight=None, bias=None, gate=None,
                           dresid=None, dw=None, db=None, dgate=None, stream=None):
    """moe_norm_residual_backward: gradients of norm_residual_forward's out. ws: norm_workspace(p)."""
    f32, par = _dtypes(DT_F32), _dtypes(p.param_dtype)
    row, st, bl, tok, vec = (p.T, p.d), _dtypes(p.stream_dtype), _dtypes(p.block_dtype), (p.T,), (p.d,)
    g = tok if p.gate_kind == GATE_TOKEN else vec
    _fits("moe_norm_residual_backward", stream, ("y", y, row, bl, False), ("dout", dout, row, st, False),
          ("dresid", dresid, row, st, False), ("dy", dy, row, bl, False), ("weight", weight, vec, par, True),
          ("bias", bias, vec, par, True), ("gate", gate, g, par, True), ("mean", mean, tok, f32, True),
          ("rstd", rstd, tok, f32, True), ("dw", dw, vec, f32, True), ("db", db, vec, f32, True),
          ("dgate", dgate, g, f32, True), _ws_spec(ws))
    _rows_ok("moe_norm_residual_backward", p, p.ld_stream, dout=dout, dresid=dresid)
    _rows_ok("moe_norm_residual_backward", p, p.ld_block, y=y, dy=dy)
    check(lib().moe_norm_residual_backward(ctypes.byref(p), _p(y), _p(weight), _p(bias), _p(gate), _p(dout), _p(mean),
                                           _p(rstd), _p(dresid), _p(dy), ctypes.byref(_norm_grads(dw, db, dgate)),
                                           _p(ws), 0 if ws is None else ws.numel(), _stream(stream)),
          "moe_norm_residual_backward")


# ------------------------------------------------------------------ products in 8-bit floating point

def f8_params(rows, K, N, E=1, out_dtype=DT_BF16, swiglu_limit=0.0, variant=VARIANT_AUTO) -> F8Params:
    return F8Params(rows, K, N, E, out_dtype, swiglu_limit, variant)


def f8_workspace(p: F8Params, device="cuda"):
    """A zeroed device workspace for matmul_f8 and gated_f8 (256-byte aligned)."""
    import torch
    n = int(lib().moe_f8_workspace_size(ctypes.byref(p)))
    if n == 0:
        raise MoeError("invalid parameters")
    ws = torch.zeros(n, dtype=torch.uint8, device=device)
    assert ws.data_ptr() % 256 == 0
    return ws


def quantize_f8(x, q, s, ws, row_index=None, n_rows=None, stream=None):
    """moe_quantize_f8: rows of x (x[row_index] when given) to e4m3 q [rows, K] and scales s [ceil(K/128), rows].
    ws: 256 zeroed bytes (the error word); n_rows: device int32, rows from it on are left as they were."""
    rows, K = q.shape
    _fits("moe_quantize_f8", stream, ("x", x, (x.shape[0], K), _dtypes("rows"), False),
          ("q", q, (rows, K), _dtypes(DT_E4M3), True), ("s", s, ((K + 127) // 128, rows), _dtypes(DT_F32), True),
          ("row_index", row_index, (rows,), _dtypes("i32"), True),
          ("n_rows", n_rows, () if n_rows is None else n_rows.shape, _dtypes("i32"), True), _ws_spec(ws))
    if n_rows is not None and n_rows.numel() == 0:
        raise MoeError("moe_quantize_f8: n_rows is empty")
    if x.shape[0] > 0 and (K > 1 and x.stride(1) != 1 or x.shape[0] > 1 and x.stride(0) < K):
        raise MoeError(f"moe_quantize_f8: x has strides {x.stride()}")
    check(lib().moe_quantize_f8(rows, K, _p(x), _dt(x), x.stride(0) if x.shape[0] > 1 else K, x.shape[0],
                                _p(row_index), _p(n_rows), _p(q), _p(s), _p(ws), ws.numel(), _stream(stream)),
          "moe_quantize_f8")


def quantize_f8_weights(w, q, s, transposed=False, stream=None):
    """moe_quantize_f8_weights: w [E, N, K] ([E, K, N] with transposed) to e4m3 q [E, N, K] and its block scales."""
    E, N, K = q.shape
    _fits("moe_quantize_f8_weights", stream, ("w", w, (E, K, N) if transposed else (E, N, K), _dtypes("rows"), True),
          ("q", q, (E, N, K), _dtypes(DT_E4M3), True),
          ("s", s, (E, (N + 127) // 128, (K + 127) // 128), _dtypes(DT_F32), True))
    check(lib().moe_quantize_f8_weights(E, N, K, _p(w), _dt(w), int(bool(transposed)), _p(q), _p(s),
                                        _stream(stream)), "moe_quantize_f8_weights")


def _f8_specs(p, a, a_scale, offsets, ws, *weights):
    """What _fits checks of the operands every product takes; weights: (name, tensor, scales)."""
    f8, f32, i32 = _dtypes(DT_E4M3), _dtypes(DT_F32), _dtypes("i32")
    kb, nb = (p.K + 127) // 128, (p.N + 127) // 128
    specs = [("a", a, (p.rows, p.K), f8, True), ("a_scale", a_scale, (kb, p.rows), f32, True),
             ("offsets", offsets, (p.E + 1,), i32, True), _ws_spec(ws)]
    for name, t, s in weights:
        specs += [(name, t, (p.E, p.N, p.K), f8, True), ("the scales of " + name, s, (p.E, nb, kb), f32, True)]
    return specs


def matmul_f8(p: F8Params, a, a_scale, b, b_scale, out, ws, offsets=None, sorted_pair=None, topk_w=None, stream=None):
    """moe_matmul_f8: out = w_r * a b^T by expert, e4m3 with scales for each block of 128."""
    _fits("moe_matmul_f8", stream, *_f8_specs(p, a, a_scale, offsets, ws, ("b", b, b_scale)),
          ("out", out, (p.rows, p.N), _dtypes(p.out_dtype), True),
          ("sorted_pair", sorted_pair, (p.rows,), _dtypes("i32"), True),
          ("topk_w", topk_w, () if topk_w is None else topk_w.shape, _dtypes(DT_F32), True))
    check(lib().moe_matmul_f8(ctypes.byref(p), _p(a), _p(a_scale), _p(offsets), _p(b), _p(b_scale), _p(sorted_pair),
                              _p(topk_w), _p(out), _p(ws), ws.numel(), _stream(stream)), "moe_matmul_f8")


def gated_f8(p: F8Params, a, a_scale, w_gate, s_gate, w_up, s_up, h, ws, h_scale=None, offsets=None, stream=None):
    """moe_gated_f8: h = silu(clamp(a w_gate^T)) * clamp(a w_up^T) by expert; e4m3 h with h_scale."""
    _fits("moe_gated_f8", stream, *_f8_specs(p, a, a_scale, offsets, ws, ("w_gate", w_gate, s_gate), ("w_up", w_up, s_up)),
          ("h", h, (p.rows, p.N), _dtypes(p.out_dtype), True),
          ("h_scale", h_scale, ((p.N + 127) // 128, p.rows), _dtypes(DT_F32), True))
    check(lib().moe_gated_f8(ctypes.byref(p), _p(a), _p(a_scale), _p(offsets), _p(w_gate), _p(s_gate), _p(w_up),
                             _p(s_up), _p(h), _p(h_scale), _p(ws), ws.numel(), _stream(stream)), "moe_gated_f8")


def f8_wait_selftest(gated, blocks, limit_ns, ws, stream=None):
    """moe_f8_wait_selftest: an 8-bit product whose copies stop after `blocks` blocks along K; sets DEVERR_TIMEOUT."""
    check(lib().moe_f8_wait_selftest(int(bool(gated)), int(blocks), int(limit_ns), _p(ws), ws.numel(), _stream(stream)),
          "moe_f8_wait_selftest")

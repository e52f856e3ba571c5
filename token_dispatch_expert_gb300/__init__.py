"""GB300-native single-GPU Mixture-of-Experts layer.

Python binding of the C ABI in include/moe.h: every function here has the name of the
C entry point it calls and only marshals arguments (torch tensors -> device pointers,
the current CUDA stream -> cudaStream_t).  Every step of the layer runs in the CUDA
kernels of libmoe_gb300.so; there is no Python or CPU fallback -- if the library is
missing, every call raises.

PyTorch is used for device memory and streams only.
"""

from __future__ import annotations

import ctypes
import os

from ._build import LIB_PATH, build  # noqa: F401

__all__ = [
    "MoEConfigC", "MoEError", "make_config", "lib",
    "moe_capacity_from_factor", "moe_workspace_size", "moe_ctx_offsets", "moe_ws_init",
    "moe_route", "moe_route_noalloc", "moe_permute", "moe_grouped_ffn", "moe_combine", "moe_combine_bwd",
    "moe_grouped_ffn_bwd", "moe_unpermute_reduce", "moe_layer_fwd", "moe_layer_bwd",
    "moe_grouped_ffn_gather", "moe_grouped_ffn_bwd_gather", "moe_grouped_ffn_bwd_dispatch",
    "moe_mx_weights_size", "moe_mx_quantize_weights", "moe_mx_act_scales_size",
    "moe_mx_permute_quant", "moe_grouped_ffn_mx", "moe_grouped_ffn_bwd_mx", "moe_layer_fwd_mx",
    "moe_layer_bwd_mx",
    "MoERouterC", "make_router", "moe_route_groups", "moe_route_groups_bwd", "moe_combine_bwd_dw",
    "FP8_WS_BYTES", "moe_fp8_token_blocks", "moe_fp8_quantize", "moe_fp8_quantize_weights",
    "moe_fp8_swiglu", "moe_fp8_swiglu_bwd", "moe_fp8_gemm", "moe_fp8_wgrad", "Fp8MoELayer",
    "moe_status", "moe_status_string", "moe_selftest_wait_timeout", "moe_gemm_clock_trace",
    "moe_gemm_clock_read", "ctx_views", "MoELayer", "CTX_FIELDS",
]

GATES = {"softmax": 0, "sigmoid": 1}
STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_CUDA",
          4: "MOE_ERR_DEVICE_FLAG", 5: "MOE_ERR_TIMEOUT"}
DEVERR = {"NAN_LOGIT": 0x1, "BAD_INDEX": 0x2, "TIMEOUT": 0x4, "BAD_OFFSETS": 0x8}
CTX_FIELDS = ["topk_idx", "topk_w", "counts", "kept", "offsets", "dest_row", "src_tok",
              "src_slot", "drop_mask", "xp", "ab", "h", "yp", "ab_s", "h_s", "ys"]


class MoEConfigC(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("ffn", ctypes.c_int32), ("ffn_shared", ctypes.c_int32),
                ("gate", ctypes.c_int32), ("route_scale", ctypes.c_float),
                ("capacity", ctypes.c_int32), ("select_bias", ctypes.c_void_p),
                ("drop_negative", ctypes.c_int32), ("recompute", ctypes.c_int32),
                ("drop_by_score", ctypes.c_int32), ("mxfp8", ctypes.c_int32)]


class MoERouterC(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("bias", ctypes.c_void_p)]


class _QuantC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("src_rows", ctypes.c_int64), ("G", ctypes.c_int32),
                ("C", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("pow2", ctypes.c_int32)]


class _ActC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("G", ctypes.c_int32), ("f", ctypes.c_int32),
                ("ld", ctypes.c_int64), ("pow2", ctypes.c_int32)]


class _Fp8GemmC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("G", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("lda", ctypes.c_int64), ("ldb", ctypes.c_int64),
                ("ldo", ctypes.c_int64), ("out_type", ctypes.c_int32)]


class _Fp8WgradC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("G", ctypes.c_int32), ("M", ctypes.c_int32),
                ("N", ctypes.c_int32), ("out_type", ctypes.c_int32)]


class MoEError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded CUDA library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(token_dispatch_expert_gb300.build() or __graft_entry__.build())")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        cfgp = ctypes.POINTER(MoEConfigC)
        sig = {
            "moe_capacity_from_factor": ([I64, I32, I32, ctypes.c_double], I32),
            "moe_workspace_size": ([cfgp, ctypes.POINTER(ctypes.c_size_t),
                                    ctypes.POINTER(ctypes.c_size_t)], I32),
            "moe_ctx_offsets": ([cfgp, ctypes.POINTER(ctypes.c_size_t)], I32),
            "moe_ws_init": ([P, P], I32),
            "moe_route": ([cfgp] + [P] * 12, I32),
            "moe_route_noalloc": ([cfgp] + [P] * 12, I32),
            "moe_permute": ([cfgp] + [P] * 6, I32),
            "moe_grouped_ffn": ([cfgp] + [P] * 9, I32),
            "moe_grouped_ffn_gather": ([cfgp] + [P] * 10, I32),
            "moe_grouped_ffn_bwd_gather": ([cfgp] + [P] * 14, I32),
            "moe_grouped_ffn_bwd_dispatch": ([cfgp] + [P] * 17, I32),
            "moe_combine": ([cfgp] + [P] * 7, I32),
            "moe_combine_bwd": ([cfgp] + [P] * 10, I32),
            "moe_grouped_ffn_bwd": ([cfgp] + [P] * 13, I32),
            "moe_unpermute_reduce": ([cfgp] + [P] * 6, I32),
            "moe_layer_fwd": ([cfgp] + [P] * 10, I32),
            "moe_mx_weights_size": ([cfgp, ctypes.POINTER(ctypes.c_size_t),
                                     ctypes.POINTER(ctypes.c_size_t)], I32),
            "moe_mx_quantize_weights": ([cfgp] + [P] * 4, I32),
            "moe_mx_act_scales_size": ([cfgp, I32, ctypes.POINTER(ctypes.c_size_t)], I32),
            "moe_mx_permute_quant": ([cfgp] + [P] * 8, I32),
            "moe_grouped_ffn_mx": ([cfgp] + [P] * 11, I32),
            "moe_layer_fwd_mx": ([cfgp] + [P] * 9, I32),
            "moe_grouped_ffn_bwd_mx": ([cfgp] + [P] * 12, I32),
            "moe_layer_bwd_mx": ([cfgp] + [P] * 15, I32),
            "moe_layer_bwd": ([cfgp] + [P] * 16, I32),
            # (the structs by address: an int converts faster than a byref, and the binding has
            # read their fields before)
            "moe_route_groups": ([P] * 14, I32),
            "moe_route_groups_bwd": ([P] * 8, I32),
            "moe_combine_bwd_dw": ([cfgp] + [P] * 8, I32),
            "moe_fp8_token_blocks": ([I64, I32], I64),
            "moe_fp8_quantize": ([ctypes.POINTER(_QuantC)] + [P] * 9, I32),
            "moe_fp8_quantize_weights": ([P, I32, I32, I32, P, I64, P, P, I64, P, I32, P], I32),
            "moe_fp8_swiglu": ([ctypes.POINTER(_ActC)] + [P] * 8, I32),
            "moe_fp8_swiglu_bwd": ([ctypes.POINTER(_ActC)] + [P] * 11, I32),
            "moe_fp8_gemm": ([ctypes.POINTER(_Fp8GemmC)] + [P] * 8, I32),
            "moe_fp8_wgrad": ([ctypes.POINTER(_Fp8WgradC)] + [P] * 8, I32),
            "moe_status": ([P, P, ctypes.POINTER(ctypes.c_int32)], I32),
            "moe_gemm_clock_trace": ([I32], I32),
            "moe_gemm_clock_read": ([ctypes.POINTER(ctypes.c_uint64)] * 3, I32),
            "moe_selftest_wait_timeout": ([P, I64, P], I32),
            "moe_status_string": ([I32], ctypes.c_char_p),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def make_config(T, d, E, k, ffn, ffn_shared=0, gate="softmax", route_scale=1.0,
                capacity=0, select_bias=None, drop_negative=False,
                recompute=False, drop_by_score=False, mxfp8=False) -> MoEConfigC:
    """select_bias: a float32 device tensor [E] (kept alive by the returned config) or None.
    mxfp8: 0 / False (bf16), 1 / True (routed forward and data gradients in MXFP8) or 2 (and
    the weight gradients)."""
    cfg = MoEConfigC(int(T), int(d), int(E), int(k), int(ffn), int(ffn_shared),
                     GATES[gate] if isinstance(gate, str) else int(gate), float(route_scale),
                     int(capacity), _p(select_bias), int(bool(drop_negative)),
                     int(bool(recompute)), int(bool(drop_by_score)), int(mxfp8))
    cfg._keep = select_bias
    return cfg


def _p(t):
    """Device pointer of a tensor (or an int address); None -> NULL.  The C calls take
    dense row-major device buffers: a host tensor or a strided view is refused here rather
    than handed to a kernel as a pointer."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    raise ValueError(f"expected a contiguous tensor, got strides {tuple(t.stride())}")


def _s(stream):
    if stream is None:
        return _raw_stream() if _raw_stream else _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


_raw_stream = None


def _current_stream():
    """The current stream's handle.  A small call's time is mostly the host's, and torch's own
    accessor builds a Stream object around the handle."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        dev = getattr(torch._C, "_cuda_getDevice", None)
        torch.cuda.init()
        _raw_stream = ((lambda: torch.cuda.current_stream().cuda_stream)
                       if raw is None or dev is None else (lambda: raw(dev())))
    return _raw_stream()


def _check(status, where):
    if status != 0:
        raise MoEError(status, where)


_cfg = ctypes.byref
_addr = ctypes.addressof


# --------------------------------------------------------------------------- host helpers
def moe_capacity_from_factor(T, k, E, c) -> int:
    return lib().moe_capacity_from_factor(int(T), int(k), int(E), float(c))


def moe_workspace_size(cfg):
    ws, ctx = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(_cfg(cfg), ctypes.byref(ws), ctypes.byref(ctx)),
           "moe_workspace_size")
    return ws.value, ctx.value


def moe_ctx_offsets(cfg):
    arr = (ctypes.c_size_t * len(CTX_FIELDS))()
    _check(lib().moe_ctx_offsets(_cfg(cfg), arr), "moe_ctx_offsets")
    return list(arr)


def moe_status_string(s) -> str:
    return lib().moe_status_string(int(s)).decode()


# --------------------------------------------------------------------------- device calls
def moe_ws_init(ws, stream=None):
    _check(lib().moe_ws_init(_p(ws), _s(stream)), "moe_ws_init")


def moe_route(cfg, logits, topk_idx, topk_w, counts, kept, offsets, dest_row, src_tok, src_slot,
              drop_mask, ws, stream=None):
    _check(lib().moe_route(_cfg(cfg), _p(logits), _p(topk_idx), _p(topk_w), _p(counts), _p(kept),
                           _p(offsets), _p(dest_row), _p(src_tok), _p(src_slot), _p(drop_mask),
                           _p(ws), _s(stream)), "moe_route")


def moe_route_noalloc(cfg, logits, topk_idx, topk_w, counts, kept, offsets, dest_row, src_tok,
                      src_slot, drop_mask, dev_flags=None, stream=None):
    """moe_route without a workspace, for callers that cannot allocate device memory
    (see include/moe.h); dev_flags is an optional device int32 for the error bits."""
    _check(lib().moe_route_noalloc(_cfg(cfg), _p(logits), _p(topk_idx), _p(topk_w), _p(counts),
                                   _p(kept), _p(offsets), _p(dest_row), _p(src_tok),
                                   _p(src_slot), _p(drop_mask), _p(dev_flags), _s(stream)),
           "moe_route_noalloc")


def moe_permute(cfg, x, src_tok, offsets, xp, ws, stream=None):
    _check(lib().moe_permute(_cfg(cfg), _p(x), _p(src_tok), _p(offsets), _p(xp), _p(ws),
                             _s(stream)), "moe_permute")


def moe_grouped_ffn(cfg, xp, offsets, W1, W2, ab, h, yp, ws, stream=None):
    _check(lib().moe_grouped_ffn(_cfg(cfg), _p(xp), _p(offsets), _p(W1), _p(W2), _p(ab), _p(h),
                                 _p(yp), _p(ws), _s(stream)), "moe_grouped_ffn")


def moe_combine(cfg, yp, dest_row, topk_w, ys, y, ws, stream=None):
    _check(lib().moe_combine(_cfg(cfg), _p(yp), _p(dest_row), _p(topk_w), _p(ys), _p(y), _p(ws),
                             _s(stream)), "moe_combine")


def moe_combine_bwd(cfg, dy, yp, logits, topk_idx, topk_w, dest_row, dyp, dlogits, ws,
                    stream=None):
    _check(lib().moe_combine_bwd(_cfg(cfg), _p(dy), _p(yp), _p(logits), _p(topk_idx), _p(topk_w),
                                 _p(dest_row), _p(dyp), _p(dlogits), _p(ws), _s(stream)),
           "moe_combine_bwd")


def moe_grouped_ffn_gather(cfg, x, src_tok, offsets, W1, W2, ab, h, yp, ws, stream=None):
    _check(lib().moe_grouped_ffn_gather(_cfg(cfg), _p(x), _p(src_tok), _p(offsets), _p(W1),
                                        _p(W2), _p(ab), _p(h), _p(yp), _p(ws), _s(stream)),
           "moe_grouped_ffn_gather")


def moe_grouped_ffn_bwd_gather(cfg, dyp, x, src_tok, offsets, W1, W2, ab, h, dab, dxp, dW1, dW2,
                               ws, stream=None):
    _check(lib().moe_grouped_ffn_bwd_gather(_cfg(cfg), _p(dyp), _p(x), _p(src_tok), _p(offsets),
                                            _p(W1), _p(W2), _p(ab), _p(h), _p(dab), _p(dxp),
                                            _p(dW1), _p(dW2), _p(ws), _s(stream)),
           "moe_grouped_ffn_bwd_gather")


def moe_grouped_ffn_bwd_dispatch(cfg, dy, topk_w, src_tok, src_slot, dyp, xp, offsets, W1, W2,
                                 ab, h, dab, dxp, dW1, dW2, ws, stream=None):
    """moe_grouped_ffn_bwd with the FC2 data-gradient reading dy through src_tok and scaling
    by the slot's gate weight (see include/moe.h)."""
    _check(lib().moe_grouped_ffn_bwd_dispatch(_cfg(cfg), _p(dy), _p(topk_w), _p(src_tok),
                                              _p(src_slot), _p(dyp), _p(xp), _p(offsets),
                                              _p(W1), _p(W2), _p(ab), _p(h), _p(dab), _p(dxp),
                                              _p(dW1), _p(dW2), _p(ws), _s(stream)),
           "moe_grouped_ffn_bwd_dispatch")


def moe_mx_weights_size(cfg):
    """(bytes, offsets of the MXFP8 blob's parts: W1 codes, W1 scales, W2 codes, W2 scales,
    W2^T codes, W2^T scales, W1^T codes, W1^T scales)."""
    b = ctypes.c_size_t(0)
    offs = (ctypes.c_size_t * 8)()
    _check(lib().moe_mx_weights_size(_cfg(cfg), ctypes.byref(b), offs), "moe_mx_weights_size")
    return b.value, [o for o in offs]


def moe_mx_act_scales_size(cfg, K) -> int:
    b = ctypes.c_size_t(0)
    _check(lib().moe_mx_act_scales_size(_cfg(cfg), int(K), ctypes.byref(b)),
           "moe_mx_act_scales_size")
    return b.value


def moe_mx_quantize_weights(cfg, W1, W2, wq, stream=None):
    _check(lib().moe_mx_quantize_weights(_cfg(cfg), _p(W1), _p(W2), _p(wq), _s(stream)),
           "moe_mx_quantize_weights")


def moe_mx_permute_quant(cfg, x, src_tok, offsets, xp, xq, x_sf, ws, stream=None):
    _check(lib().moe_mx_permute_quant(_cfg(cfg), _p(x), _p(src_tok), _p(offsets), _p(xp),
                                      _p(xq), _p(x_sf), _p(ws), _s(stream)),
           "moe_mx_permute_quant")


def moe_grouped_ffn_mx(cfg, xq, x_sf, offsets, wq, ab, h, hq, h_sf, yp, ws, stream=None):
    _check(lib().moe_grouped_ffn_mx(_cfg(cfg), _p(xq), _p(x_sf), _p(offsets), _p(wq), _p(ab),
                                    _p(h), _p(hq), _p(h_sf), _p(yp), _p(ws), _s(stream)),
           "moe_grouped_ffn_mx")


def moe_layer_fwd_mx(cfg, logits, x, wq, W1s, W2s, y, ctx, ws, stream=None):
    _check(lib().moe_layer_fwd_mx(_cfg(cfg), _p(logits), _p(x), _p(wq), _p(W1s), _p(W2s), _p(y),
                                  _p(ctx), _p(ws), _s(stream)), "moe_layer_fwd_mx")


def moe_grouped_ffn_bwd_mx(cfg, dyp, xp, offsets, wq, ab, h, dab, dxp, dW1, dW2, ws,
                           stream=None):
    _check(lib().moe_grouped_ffn_bwd_mx(_cfg(cfg), _p(dyp), _p(xp), _p(offsets), _p(wq), _p(ab),
                                        _p(h), _p(dab), _p(dxp), _p(dW1), _p(dW2), _p(ws),
                                        _s(stream)), "moe_grouped_ffn_bwd_mx")


def moe_layer_bwd_mx(cfg, ctx, logits, x, dy, wq, W1s, W2s, dx, dW1, dW2, dW1s, dW2s, dlogits,
                     ws, stream=None):
    _check(lib().moe_layer_bwd_mx(_cfg(cfg), _p(ctx), _p(logits), _p(x), _p(dy), _p(wq),
                                  _p(W1s), _p(W2s), _p(dx), _p(dW1), _p(dW2), _p(dW1s), _p(dW2s),
                                  _p(dlogits), _p(ws), _s(stream)), "moe_layer_bwd_mx")


def moe_grouped_ffn_bwd(cfg, dyp, xp, offsets, W1, W2, ab, h, dab, dxp, dW1, dW2, ws,
                        stream=None):
    _check(lib().moe_grouped_ffn_bwd(_cfg(cfg), _p(dyp), _p(xp), _p(offsets), _p(W1), _p(W2),
                                     _p(ab), _p(h), _p(dab), _p(dxp), _p(dW1), _p(dW2), _p(ws),
                                     _s(stream)), "moe_grouped_ffn_bwd")


def moe_unpermute_reduce(cfg, dxp, dest_row, dxs, dx, ws, stream=None):
    _check(lib().moe_unpermute_reduce(_cfg(cfg), _p(dxp), _p(dest_row), _p(dxs), _p(dx), _p(ws),
                                      _s(stream)), "moe_unpermute_reduce")


def moe_layer_fwd(cfg, logits, x, W1, W2, W1s, W2s, y, ctx, ws, stream=None):
    _check(lib().moe_layer_fwd(_cfg(cfg), _p(logits), _p(x), _p(W1), _p(W2), _p(W1s), _p(W2s),
                               _p(y), _p(ctx), _p(ws), _s(stream)), "moe_layer_fwd")


def moe_layer_bwd(cfg, ctx, logits, x, dy, W1, W2, W1s, W2s, dx, dW1, dW2, dW1s, dW2s, dlogits,
                  ws, stream=None):
    _check(lib().moe_layer_bwd(_cfg(cfg), _p(ctx), _p(logits), _p(x), _p(dy), _p(W1), _p(W2),
                               _p(W1s), _p(W2s), _p(dx), _p(dW1), _p(dW2), _p(dW1s), _p(dW2s),
                               _p(dlogits), _p(ws), _s(stream)), "moe_layer_bwd")


def moe_selftest_wait_timeout(ws, budget_cycles, stream=None):
    """Enqueue a bounded wait that is never satisfied (see include/moe.h)."""
    _check(lib().moe_selftest_wait_timeout(_p(ws), int(budget_cycles), _s(stream)),
           "moe_selftest_wait_timeout")


def moe_gemm_clock_trace(enable):
    """Turn the grouped GEMMs' clock tracing on (zeroing its sums) or off (keeping them)."""
    _check(lib().moe_gemm_clock_trace(1 if enable else 0), "moe_gemm_clock_trace")


def moe_gemm_clock_read():
    """The traced sums: (SM cycles, nanoseconds, loops) of the GEMM tile loops."""
    c, n, k = ctypes.c_uint64(0), ctypes.c_uint64(0), ctypes.c_uint64(0)
    _check(lib().moe_gemm_clock_read(ctypes.byref(c), ctypes.byref(n), ctypes.byref(k)),
           "moe_gemm_clock_read")
    return c.value, n.value, k.value


# ------------------------------------------------------------------- group-limited routing
SCORES = {"softmax": 0, "sigmoid": 1}


def make_router(score="softmax", groups=1, top_groups=None, group_top=1, renorm=True, bias=None):
    """A router for moe_route_groups (see include/moe.h): score "softmax" or "sigmoid";
    top_groups of `groups` groups stay (None: all); bias: a float32 device tensor [E] (kept
    alive by the returned struct) or None."""
    r = MoERouterC(SCORES[score] if isinstance(score, str) else int(score), int(groups),
                   int(groups if top_groups is None else top_groups), int(group_top),
                   int(renorm), _typed(bias, "float32", "bias"))
    r._keep = bias
    return r


_dtypes = {}   # name -> torch dtype


def _dtype(name):
    import torch
    return _dtypes.setdefault(name, getattr(torch, name))


def _typed(t, dtype, name):
    """_p for a buffer of one element type (a torch dtype's name)."""
    if t is None:
        return None
    if not isinstance(t, int) and t.dtype is not (_dtypes.get(dtype) or _dtype(dtype)):
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    return _p(t)


def _buf(t, dtype, n, name):
    """_p for a buffer of at least n elements of a torch dtype (None: one byte an element): what a
    kernel takes for int32 or fp32 must not be another type, and all that it writes must be there."""
    if t is None or isinstance(t, int):
        return t
    if t.element_size() != 1 if dtype is None else t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype or 'one byte an element'}, got {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")
    return _p(t)


class _Buffers:
    """The buffers of one entry point: their names, and their torch dtypes (looked up once)."""

    def __init__(self, *names):
        self.names = names
        self.dtypes = None

    def _load(self):
        import torch
        i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
        kind = dict(logits=f32, topk_w=f32, dw=f32, dlogits=f32, dy=bf, yp=bf, dyp=bf,
                    drop_mask=torch.uint8)
        t = torch.Tensor
        self.numel, self.contiguous, self.data_ptr = t.numel, t.is_contiguous, t.data_ptr
        self.dtypes = [kind.get(n, i32) for n in self.names]

    def __call__(self, tensors, sizes):
        """_buf for each.  The usual call, tensors of just these types and sizes, is told by
        comparing lists, which takes less of a small call's time than a call of _buf for each."""
        if self.dtypes is None:
            self._load()
        try:
            if ([t.dtype for t in tensors] == self.dtypes
                    and list(map(self.numel, tensors)) == sizes
                    and all([t.is_cuda for t in tensors])
                    and all(map(self.contiguous, tensors))):
                return map(self.data_ptr, tensors)
        except AttributeError:   # an address among them
            pass
        return [_buf(t, None if name == "drop_mask" else dt, n, name)
                for t, dt, n, name in zip(tensors, self.dtypes, sizes, self.names)]


_route_buffers = _Buffers("logits", "topk_idx", "topk_w", "counts", "kept", "offsets", "dest_row",
                          "src_tok", "src_slot", "drop_mask")
_route_bwd_buffers = _Buffers("logits", "topk_idx", "dw", "dlogits")
_combine_dw_buffers = _Buffers("dy", "yp", "topk_w", "dest_row", "dyp", "dw")


def _check_bias(bias, E):
    if bias is not None and not isinstance(bias, int) and bias.numel() < E:
        raise ValueError(f"bias: expected {E} elements, got {bias.numel()}")


def moe_route_groups(cfg, router, logits, topk_idx, topk_w, counts, kept, offsets, dest_row,
                     src_tok, src_slot, drop_mask, ws, stream=None):
    T, E = cfg.T, cfg.E
    n = T * cfg.k
    if router.bias:
        _check_bias(getattr(router, "_keep", None), E)
    ptrs = _route_buffers((logits, topk_idx, topk_w, counts, kept, offsets, dest_row, src_tok,
                           src_slot, drop_mask), [T * E, n, n, E, E, E + 1, n, n, n, n])
    _check(lib().moe_route_groups(_addr(cfg), _addr(router), *ptrs, _p(ws), _s(stream)),
           "moe_route_groups")


def moe_route_groups_bwd(cfg, router, logits, topk_idx, dw, dlogits, ws, stream=None):
    T, E = cfg.T, cfg.E
    n = T * cfg.k
    if not isinstance(router, MoERouterC):
        raise TypeError(f"router: expected a MoERouterC, got {type(router).__name__}")
    # (the bias is not read: the choice is given)
    ptrs = _route_bwd_buffers((logits, topk_idx, dw, dlogits), [T * E, n, n, T * E])
    _check(lib().moe_route_groups_bwd(_addr(cfg), _addr(router), *ptrs, _p(ws), _s(stream)),
           "moe_route_groups_bwd")


def moe_combine_bwd_dw(cfg, dy, yp, topk_w, dest_row, dyp, dw, ws, stream=None):
    n = cfg.T * cfg.k
    # (yp and dyp: as many rows as dest_row names, which the host does not see)
    ptrs = _combine_dw_buffers((dy, yp, topk_w, dest_row, dyp, dw),
                               [cfg.T * cfg.d, 0, n, n, 0, n])
    _check(lib().moe_combine_bwd_dw(_cfg(cfg), *ptrs, _p(ws), _s(stream)), "moe_combine_bwd_dw")


# ------------------------------------------------- 8-bit operands, a scale per block of 128
FP8_WS_BYTES = 256


def moe_fp8_token_blocks(rows, G) -> int:
    """The number of 128-row blocks that `rows` rows in G segments can need."""
    return lib().moe_fp8_token_blocks(int(rows), int(G))


def _shape(name, t, shape):
    if t.shape != shape:   # (a tuple's comparison: half the cost of building one)
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")


def _bytes(t, name):
    if t is not None and t.element_size() != 1:
        raise ValueError(f"{name}: expected 8-bit codes, got {t.dtype}")
    return _p(t)


def _groups(offsets):
    return 1 if offsets is None else offsets.numel() - 1


def _quant_outputs(rows, G, cols, codes, scales, codes_t, scales_t):
    """Check what a quantiser writes; the distance of the codes' rows."""
    ld = 0
    if codes is not None:
        ld = codes.shape[-1]
        _shape("codes", codes, (rows, ld))
        _shape("scales", scales, (rows, (cols + 127) // 128))
    if codes_t is not None:
        blocks = moe_fp8_token_blocks(rows, G)
        _shape("codes_t", codes_t, (cols, 128 * blocks))
        _shape("scales_t", scales_t, (blocks, cols))
    return ld


def moe_fp8_quantize(x, codes=None, scales=None, codes_t=None, scales_t=None, *, offsets=None,
                     src_tok=None, pow2=False, ws, stream=None):
    """Quantise rows of x (bf16, rows may be strided) along the row (codes, scales) and, or, along
    the tokens of the segments (codes_t, scales_t); row p is x[src_tok[p]] when src_tok is
    given."""
    if (x.dim() != 2 or x.stride(1) != 1 or not x.is_cuda or
            x.dtype is not (_dtypes.get("bfloat16") or _dtype("bfloat16"))):
        raise ValueError("x: expected a CUDA bf16 matrix with adjacent columns")
    G = _groups(offsets)
    rows = x.shape[0] if src_tok is None else src_tok.numel()
    ld = _quant_outputs(rows, G, x.shape[1], codes, scales, codes_t, scales_t)
    ldx = x.stride(0) if x.shape[0] > 1 else x.shape[1]
    q = _QuantC(rows, x.shape[0], G, x.shape[1], ldx, ld, int(pow2))
    _check(lib().moe_fp8_quantize(ctypes.byref(q), x.data_ptr(), _typed(src_tok, "int32", "src_tok"),
                                  _typed(offsets, "int32", "offsets"), _bytes(codes, "codes"),
                                  _typed(scales, "float32", "scales"), _bytes(codes_t, "codes_t"),
                                  _typed(scales_t, "float32", "scales_t"), _p(ws), _s(stream)),
           "moe_fp8_quantize")


def moe_fp8_quantize_weights(w, codes, scales, codes_t=None, scales_t=None, *, pow2=False,
                             stream=None):
    """Quantise weights w [G, N, K] (bf16) in 128 x 128 blocks, optionally transposed too."""
    G, N, K = w.shape
    _shape("codes", codes, (G, N, codes.shape[-1]))
    _shape("scales", scales, (G, (N + 127) // 128, (K + 127) // 128))
    if codes_t is not None:
        _shape("codes_t", codes_t, (G, K, codes_t.shape[-1]))
        _shape("scales_t", scales_t, (G, (K + 127) // 128, (N + 127) // 128))
    _check(lib().moe_fp8_quantize_weights(_typed(w, "bfloat16", "w"), G, N, K,
                                          _bytes(codes, "codes"), codes.shape[-1],
                                          _typed(scales, "float32", "scales"),
                                          _bytes(codes_t, "codes_t"),
                                          0 if codes_t is None else codes_t.shape[-1],
                                          _typed(scales_t, "float32", "scales_t"), int(pow2),
                                          _s(stream)), "moe_fp8_quantize_weights")


def moe_fp8_swiglu(ab, codes=None, scales=None, codes_t=None, scales_t=None, *, offsets=None,
                   pow2=False, ws, stream=None):
    """silu(a) * b of ab = [a | b] (bf16), quantised."""
    rows, G, f = ab.shape[0], _groups(offsets), ab.shape[1] // 2
    _shape("ab", ab, (rows, 2 * f))
    ld = _quant_outputs(rows, G, f, codes, scales, codes_t, scales_t)
    _check(lib().moe_fp8_swiglu(ctypes.byref(_ActC(rows, G, f, ld, int(pow2))),
                                _typed(ab, "bfloat16", "ab"), _typed(offsets, "int32", "offsets"),
                                _bytes(codes, "codes"), _typed(scales, "float32", "scales"),
                                _bytes(codes_t, "codes_t"),
                                _typed(scales_t, "float32", "scales_t"), _p(ws), _s(stream)),
           "moe_fp8_swiglu")


def moe_fp8_swiglu_bwd(dh, ab, codes, scales, codes_t=None, scales_t=None, h_codes_t=None,
                       h_scales_t=None, *, offsets=None, pow2=False, ws, stream=None):
    """[da | db] of the SwiGLU from dh (bf16), quantised; h_codes_t: also h along the tokens."""
    rows, f = dh.shape
    G = _groups(offsets)
    _shape("ab", ab, (rows, 2 * f))
    ld = _quant_outputs(rows, G, 2 * f, codes, scales, codes_t, scales_t)
    if h_codes_t is not None:
        _quant_outputs(rows, G, f, None, None, h_codes_t, h_scales_t)
    _check(lib().moe_fp8_swiglu_bwd(ctypes.byref(_ActC(rows, G, f, ld, int(pow2))),
                                    _typed(dh, "bfloat16", "dh"), _typed(ab, "bfloat16", "ab"),
                                    _typed(offsets, "int32", "offsets"), _bytes(codes, "codes"),
                                    _typed(scales, "float32", "scales"),
                                    _bytes(codes_t, "codes_t"),
                                    _typed(scales_t, "float32", "scales_t"),
                                    _bytes(h_codes_t, "h_codes_t"),
                                    _typed(h_scales_t, "float32", "h_scales_t"), _p(ws),
                                    _s(stream)), "moe_fp8_swiglu_bwd")


def _out_type(t, name):
    if t.dtype is (_dtypes.get("bfloat16") or _dtype("bfloat16")):
        return 0
    if t.dtype is (_dtypes.get("float32") or _dtype("float32")):
        return 1
    raise ValueError(f"{name}: expected bfloat16 or float32, got {t.dtype}")


def moe_fp8_gemm(a, a_scales, b, b_scales, out, K, *, offsets=None, ws, stream=None):
    """out[p] = A[p] B[g]^T for the rows p of each segment g, over K columns of the codes a
    [rows, lda] and b [G, N, ldb]; out (bf16 or fp32) may have strided rows."""
    rows, G, N = a.shape[0], _groups(offsets), b.shape[1]
    _shape("a_scales", a_scales, (rows, (K + 127) // 128))
    _shape("b", b, (G, N, b.shape[2]))
    _shape("b_scales", b_scales, (G, (N + 127) // 128, (K + 127) // 128))
    _shape("out", out, (rows, N))
    if out.stride(1) != 1 and N > 1 or not out.is_cuda:
        raise ValueError("out: expected a CUDA matrix with adjacent columns")
    ldo = out.stride(0) if rows > 1 else N
    g = _Fp8GemmC(rows, G, N, int(K), a.shape[1], b.shape[2], ldo, _out_type(out, "out"))
    _check(lib().moe_fp8_gemm(ctypes.byref(g), _bytes(a, "a"),
                              _typed(a_scales, "float32", "a_scales"), _bytes(b, "b"),
                              _typed(b_scales, "float32", "b_scales"),
                              _typed(offsets, "int32", "offsets"), out.data_ptr(), _p(ws),
                              _s(stream)), "moe_fp8_gemm")


def moe_fp8_wgrad(a, a_scales, b, b_scales, dw, *, offsets=None, rows=None, ws, stream=None):
    """dw[g] = A_g^T B_g over the rows of each segment, from along-token operands a [M, 128 B] and
    b [N, 128 B] with scales [B, M] and [B, N].  `rows`: the row capacity the operands were made
    for (default: the largest that gives the same B)."""
    G, M, N = dw.shape
    blocks = a_scales.shape[0]
    if G != _groups(offsets):
        raise ValueError(f"dw: expected {_groups(offsets)} gradients, got {G}")
    if rows is None:
        rows = 128 * (blocks - G)
    if moe_fp8_token_blocks(rows, G) != blocks:
        raise ValueError(f"a_scales: {blocks} token blocks do not fit {rows} rows in {G} segments")
    _shape("a", a, (M, 128 * blocks))
    _shape("a_scales", a_scales, (blocks, M))
    _shape("b", b, (N, 128 * blocks))
    _shape("b_scales", b_scales, (blocks, N))
    g = _Fp8WgradC(rows, G, M, N, _out_type(dw, "dw"))
    _check(lib().moe_fp8_wgrad(ctypes.byref(g), _bytes(a, "a"),
                               _typed(a_scales, "float32", "a_scales"), _bytes(b, "b"),
                               _typed(b_scales, "float32", "b_scales"),
                               _typed(offsets, "int32", "offsets"), _p(dw), _p(ws), _s(stream)),
           "moe_fp8_wgrad")


def moe_status(ws, stream=None):
    """Synchronise the stream and read + clear the device error word: (status, flags)."""
    flags = ctypes.c_int32(0)
    s = lib().moe_status(_p(ws), _s(stream), ctypes.byref(flags))
    return s, flags.value


# --------------------------------------------------------------------------- conveniences
def ctx_views(cfg, ctx):
    """Typed torch views of the saved tensors inside a forward context buffer."""
    import torch
    off = moe_ctx_offsets(cfg)
    T, k, E, d, f, fs = cfg.T, cfg.k, cfg.E, cfg.d, cfg.ffn, cfg.ffn_shared
    R = T * k
    spec = {
        "topk_idx": (torch.int32, (T, k)), "topk_w": (torch.float32, (T, k)),
        "counts": (torch.int32, (E,)), "kept": (torch.int32, (E,)),
        "offsets": (torch.int32, (E + 1,)), "dest_row": (torch.int32, (T, k)),
        "src_tok": (torch.int32, (R,)), "src_slot": (torch.int32, (R,)),
        "drop_mask": (torch.uint8, (T, k)), "xp": (torch.bfloat16, (R, d)),
        "ab": (torch.bfloat16, (R, 2 * f)), "h": (torch.bfloat16, (R, f)),
        "yp": (torch.bfloat16, (R, d)), "ab_s": (torch.bfloat16, (T, 2 * fs)),
        "h_s": (torch.bfloat16, (T, fs)), "ys": (torch.bfloat16, (T, d if fs else 0)),
    }
    if cfg.recompute:   # FC1's outputs are not kept in ctx
        for name, cols in (("ab", 2 * f), ("h", f), ("ab_s", 2 * fs), ("h_s", fs)):
            spec[name] = (torch.bfloat16, (0, cols))
    out = {}
    for i, name in enumerate(CTX_FIELDS):
        dt, shape = spec[name]
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        out[name] = ctx[off[i]: off[i] + nbytes].view(dt).view(shape)
    return out


class MoELayer:
    """Owns the workspace and forward context (torch device buffers) of one layer shape
    and calls moe_layer_fwd / moe_layer_bwd on them."""

    def __init__(self, cfg: MoEConfigC, device="cuda"):
        import torch
        self.cfg = cfg
        ws_b, ctx_b = moe_workspace_size(cfg)
        self.ws = torch.empty(ws_b, dtype=torch.uint8, device=device)
        self.ctx = torch.empty(ctx_b, dtype=torch.uint8, device=device)
        moe_ws_init(self.ws)

    def views(self):
        return ctx_views(self.cfg, self.ctx)

    def forward(self, logits, x, W1, W2, W1s=None, W2s=None, y=None, stream=None):
        import torch
        if y is None:
            y = torch.empty_like(x)
        moe_layer_fwd(self.cfg, logits, x, W1, W2, W1s, W2s, y, self.ctx, self.ws, stream)
        return y

    def quantize_weights(self, W1, W2, stream=None):
        """MXFP8 blob of the routed weights (cache it while W1, W2 are unchanged)."""
        import torch
        nbytes, _ = moe_mx_weights_size(self.cfg)
        wq = torch.empty(nbytes, dtype=torch.uint8, device=W1.device)
        moe_mx_quantize_weights(self.cfg, W1, W2, wq, stream)
        return wq

    def forward_mx(self, logits, x, wq, W1s=None, W2s=None, y=None, stream=None):
        """Forward with the routed experts in MXFP8 (config made with mxfp8=1 or 2); the
        bf16 backward() may follow it, or backward_mx()."""
        import torch
        if y is None:
            y = torch.empty_like(x)
        moe_layer_fwd_mx(self.cfg, logits, x, wq, W1s, W2s, y, self.ctx, self.ws, stream)
        return y

    def backward_mx(self, logits, x, dy, wq, W1s=None, W2s=None, out=None, stream=None):
        """Backward with the data-gradient GEMMs in MXFP8 (after forward_mx), and with
        mxfp8=2 the routed weight gradients too; `out` as in backward(); the
        weight-gradient shapes come from the config."""
        import torch
        c = self.cfg
        if out is None:
            bf = dict(dtype=torch.bfloat16, device=x.device)
            out = {"dx": torch.empty_like(x),
                   "dW1": torch.empty((c.E, 2 * c.ffn, c.d), **bf),
                   "dW2": torch.empty((c.E, c.d, c.ffn), **bf),
                   "dlogits": torch.empty_like(logits)}
            if c.ffn_shared:
                out["dW1s"] = torch.empty_like(W1s)
                out["dW2s"] = torch.empty_like(W2s)
        moe_layer_bwd_mx(c, self.ctx, logits, x, dy, wq, W1s, W2s, out["dx"], out["dW1"],
                         out["dW2"], out.get("dW1s"), out.get("dW2s"), out["dlogits"], self.ws,
                         stream)
        return out

    def backward(self, logits, x, dy, W1, W2, W1s=None, W2s=None, out=None, stream=None):
        import torch
        if out is None:
            out = {"dx": torch.empty_like(x), "dW1": torch.empty_like(W1),
                   "dW2": torch.empty_like(W2),
                   "dlogits": torch.empty_like(logits)}
            if self.cfg.ffn_shared:
                out["dW1s"] = torch.empty_like(W1s)
                out["dW2s"] = torch.empty_like(W2s)
        moe_layer_bwd(self.cfg, self.ctx, logits, x, dy, W1, W2, W1s, W2s, out["dx"], out["dW1"],
                      out["dW2"], out.get("dW1s"), out.get("dW2s"), out["dlogits"], self.ws,
                      stream)
        return out

    def status(self, stream=None):
        return moe_status(self.ws, stream)


class Fp8MoELayer:
    """A layer whose router limits the choice to groups of experts and whose routed experts run
    on 8-bit operands with a scale per block of 128, forward and backward.  Owns its buffers;
    the weights are quantised once per update (quantize_weights) and passed to every call.

        layer = Fp8MoELayer(cfg, make_router("sigmoid", groups=8, top_groups=4, group_top=2))
        w = layer.quantize_weights(W1, W2)
        y = layer.forward(logits, x, w)
        g = layer.backward(logits, x, dy, w)      # dx, dW1, dW2, dlogits
    """

    def __init__(self, cfg: MoEConfigC, router: MoERouterC, device="cuda", grad_dtype=None):
        import torch
        if cfg.ffn_shared:
            raise ValueError("Fp8MoELayer has no shared expert")
        self.cfg, self.router, self.device = cfg, router, device
        self.grad_dtype = torch.bfloat16 if grad_dtype is None else grad_dtype
        T, k, E, d, f = cfg.T, cfg.k, cfg.E, cfg.d, cfg.ffn
        R = T * k
        B = moe_fp8_token_blocks(R, E)
        self.ws = torch.empty(moe_workspace_size(cfg)[0], dtype=torch.uint8, device=device)
        moe_ws_init(self.ws)
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
        e4 = torch.float8_e4m3fn
        blk = lambda n: (n + 127) // 128  # noqa: E731
        self.r = {"topk_idx": new((T, k), i32), "topk_w": new((T, k), f32),
                  "counts": new((E,), i32), "kept": new((E,), i32), "offsets": new((E + 1,), i32),
                  "dest_row": new((T, k), i32), "src_tok": new((R,), i32),
                  "src_slot": new((R,), i32), "drop_mask": new((T, k), torch.uint8)}
        self.ab, self.yp = new((R, 2 * f), bf), new((R, d), bf)
        # along the row: the operands of the products; along the tokens: of the weight gradients
        self.q = {n: (new((R, c), e4), new((R, blk(c)), f32))
                  for n, c in (("x", d), ("h", f), ("dy", d), ("dab", 2 * f))}
        self.qt = {n: (new((c, 128 * B), e4), new((B, c), f32))
                   for n, c in (("x", d), ("h", f), ("dy", d), ("dab", 2 * f))}
        self.dyp, self.dh, self.dxp = new((R, d), bf), new((R, f), bf), new((R, d), bf)
        self.dw = new((T, k), f32)

    def quantize_weights(self, W1, W2, stream=None):
        """W1 [E, 2f, d], W2 [E, d, f] (bf16) -> what forward and backward read."""
        import torch
        out = {}
        for name, w in (("W1", W1), ("W2", W2)):
            G, N, K = w.shape
            new = lambda shape, dt: torch.empty(shape, dtype=dt, device=w.device)  # noqa: E731
            blk = lambda n: (n + 127) // 128  # noqa: E731
            t = (new((G, N, K), torch.float8_e4m3fn), new((G, blk(N), blk(K)), torch.float32),
                 new((G, K, N), torch.float8_e4m3fn), new((G, blk(K), blk(N)), torch.float32))
            moe_fp8_quantize_weights(w, *t, stream=stream)
            out[name], out[name + "_t"] = t[:2], t[2:]
        return out

    def forward(self, logits, x, w, y=None, stream=None):
        import torch
        c, r, ws = self.cfg, self.r, self.ws
        if y is None:
            y = torch.empty_like(x)
        moe_route_groups(c, self.router, logits, *r.values(), ws, stream)
        seg = dict(offsets=r["offsets"], ws=ws, stream=stream)
        moe_fp8_quantize(x, *self.q["x"], src_tok=r["src_tok"], **seg)
        moe_fp8_gemm(*self.q["x"], *w["W1"], self.ab, c.d, **seg)
        moe_fp8_swiglu(self.ab, *self.q["h"], **seg)
        moe_fp8_gemm(*self.q["h"], *w["W2"], self.yp, c.ffn, **seg)
        moe_combine(c, self.yp, r["dest_row"], r["topk_w"], None, y, ws, stream)
        return y

    def backward(self, logits, x, dy, w, out=None, stream=None):
        """After forward() on the same logits, x and w."""
        import torch
        c, r, ws = self.cfg, self.r, self.ws
        R = c.T * c.k
        if out is None:
            out = {"dx": torch.empty_like(x), "dlogits": torch.empty_like(logits),
                   "dW1": torch.empty((c.E, 2 * c.ffn, c.d), dtype=self.grad_dtype,
                                      device=x.device),
                   "dW2": torch.empty((c.E, c.d, c.ffn), dtype=self.grad_dtype, device=x.device)}
        seg = dict(offsets=r["offsets"], ws=ws, stream=stream)
        moe_combine_bwd_dw(c, dy, self.yp, r["topk_w"], r["dest_row"], self.dyp, self.dw, ws,
                           stream)
        moe_route_groups_bwd(c, self.router, logits, r["topk_idx"], self.dw, out["dlogits"], ws,
                             stream)
        moe_fp8_quantize(self.dyp, *self.q["dy"], *self.qt["dy"], **seg)
        moe_fp8_gemm(*self.q["dy"], *w["W2_t"], self.dh, c.d, **seg)
        moe_fp8_swiglu_bwd(self.dh, self.ab, *self.q["dab"], *self.qt["dab"], *self.qt["h"], **seg)
        moe_fp8_wgrad(*self.qt["dy"], *self.qt["h"], out["dW2"], rows=R, **seg)
        moe_fp8_gemm(*self.q["dab"], *w["W1_t"], self.dxp, 2 * c.ffn, **seg)
        moe_unpermute_reduce(c, self.dxp, r["dest_row"], None, out["dx"], ws, stream)
        moe_fp8_quantize(x, codes_t=self.qt["x"][0], scales_t=self.qt["x"][1],
                         src_tok=r["src_tok"], **seg)
        moe_fp8_wgrad(*self.qt["dab"], *self.qt["x"], out["dW1"], rows=R, **seg)
        return out

    def status(self, stream=None):
        return moe_status(self.ws, stream)

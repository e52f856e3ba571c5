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
import functools
import os

from ._build import LIB_PATH, build  # noqa: F401

__all__ = [
    "MoEConfigC", "MoEError", "make_config", "lib",
    "moe_capacity_from_factor", "moe_workspace_size", "moe_stage_workspace_size", "moe_ctx_offsets",
    "moe_ws_init",
    "moe_route", "moe_route_noalloc", "moe_permute", "moe_grouped_ffn", "moe_combine", "moe_combine_bwd",
    "moe_grouped_ffn_bwd", "moe_unpermute_reduce", "moe_layer_fwd", "moe_layer_bwd",
    "moe_grouped_ffn_gather", "moe_grouped_ffn_bwd_gather", "moe_grouped_ffn_bwd_dispatch",
    "moe_mx_weights_size", "moe_mx_quantize_weights", "moe_mx_act_scales_size",
    "moe_mx_permute_quant", "moe_grouped_ffn_mx", "moe_grouped_ffn_bwd_mx", "moe_layer_fwd_mx",
    "moe_layer_bwd_mx",
    "MoERouterC", "make_router", "moe_route_groups", "moe_route_groups_bwd", "moe_combine_bwd_dw",
    "FP8_WS_BYTES", "moe_fp8_token_blocks", "moe_fp8_quantize", "moe_fp8_quantize_weights",
    "moe_fp8_swiglu", "moe_fp8_swiglu_bwd", "moe_fp8_gemm", "moe_fp8_wgrad", "Fp8MoELayer",
    "moe_norm", "moe_norm_ws_size", "moe_norm_bwd", "moe_ckpt_norm", "moe_ckpt_save",
    "moe_ckpt_load", "moe_ckpt_swiglu", "moe_ckpt_swiglu_bwd", "moe_ckpt_combine_bwd",
    "MoEScratch", "CheckpointedMoELayer", "MoENorm",
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


class _NormC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("C", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("eps", ctypes.c_float), ("x_type", ctypes.c_int32), ("y_type", ctypes.c_int32),
                ("p_type", ctypes.c_int32), ("g_type", ctypes.c_int32),
                ("format", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ld_add", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_out", ctypes.c_int64), ("ld_codes", ctypes.c_int64)]


class _CkptC(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("C", ctypes.c_int32), ("format", ctypes.c_int32),
                ("x_type", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ld", ctypes.c_int64)]


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
            "moe_stage_workspace_size": ([cfgp, ctypes.POINTER(ctypes.c_size_t)], I32),
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
            "moe_norm": ([P] * 12, I32),
            "moe_norm_ws_size": ([I64, I32], I64),
            "moe_norm_bwd": ([P] * 13, I32),
            "moe_ckpt_norm": ([P] * 9, I32),
            "moe_ckpt_save": ([P] * 7, I32),
            "moe_ckpt_load": ([P] * 7, I32),
            "moe_ckpt_swiglu": ([P] * 8, I32),
            "moe_ckpt_swiglu_bwd": ([P] * 9, I32),
            "moe_ckpt_combine_bwd": ([P, P, P, I64, P, I32, P, P, P, P, P, P], I32),
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


def moe_stage_workspace_size(cfg):
    """Bytes of a workspace for the calls of single stages alone (see include/moe.h)."""
    ws = ctypes.c_size_t(0)
    _check(lib().moe_stage_workspace_size(_cfg(cfg), ctypes.byref(ws)), "moe_stage_workspace_size")
    return ws.value


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


# --------------------------------------------------- normalisation and 8-bit checkpoints of rows
NORMS = {"layer": 0, "rms": 1}
_row_types = {}   # torch dtype -> moe_out_t
_formats = {}     # torch dtype of the codes -> moe_ckpt_t


def _load_row_types():
    import torch
    _row_types.update({torch.bfloat16: 0, torch.float32: 1})
    _formats.update({torch.int8: 0, torch.float8_e4m3fn: 1})


# A small call's time is the host's.  The structs depend on sizes, types and distances alone and are
# never changed, so one of each is kept and passed by its address.
@functools.lru_cache(maxsize=1024)
def _norm_struct(*fields):
    p = _NormC(*fields)
    return p, _addr(p)


@functools.lru_cache(maxsize=1024)
def _ckpt_struct(*fields):
    p = _CkptC(*fields)
    return p, _addr(p)


def _row_type(t, name):
    """moe_out_t of a tensor."""
    k = _row_types.get(t.dtype)
    if k is None:
        if not _row_types:
            _load_row_types()
            return _row_type(t, name)
        raise ValueError(f"{name}: expected bfloat16 or float32, got {t.dtype}")
    return k


def _rows(t, name, shape, kind=None):
    """(pointer, moe_out_t, elements between rows) of a matrix whose rows may be strided; kind: the
    type that it has to be of."""
    k = _row_types.get(t.dtype)
    if k is None:
        k = _row_type(t, name)
    if kind is not None and k != kind:
        raise ValueError(f"{name}: expected {'float32' if kind else 'bfloat16'}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    ld = shape[1]
    if not t.is_contiguous():
        step, one = t.stride()
        if one != 1 and ld > 1:
            raise ValueError(f"{name}: expected a matrix with adjacent columns")
        if shape[0] > 1:
            ld = step
    if not t.is_cuda:
        raise ValueError(f"expected a CUDA tensor, got one on {t.device}")
    return t.data_ptr(), k, ld


def _vector(t, name, n):
    """The address of n fp32 elements."""
    if t is None:
        return None
    if _row_types.get(t.dtype) != 1:
        raise ValueError(f"{name}: expected float32, got {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")
    return t.data_ptr() if t.is_cuda and t.is_contiguous() else _p(t)


def _bf16(t, name):
    """The address of a dense bf16 buffer."""
    if t is None:
        return None
    if _row_types.get(t.dtype) != 0:
        raise ValueError(f"{name}: expected bfloat16, got {t.dtype}")
    return t.data_ptr() if t.is_cuda and t.is_contiguous() else _p(t)


def _params(C, a, b, names):
    """(type, pointer, pointer) of two vectors of one type, each of which may be missing."""
    kind, pa, pb = 0, None, None
    if a is not None:
        kind = _row_type(a, names[0])
        if a.numel() != C:
            raise ValueError(f"{names[0]}: expected {C} elements, got {a.numel()}")
        pa = a.data_ptr() if a.is_cuda and a.is_contiguous() else _p(a)
    if b is not None:
        kb = _row_type(b, names[1])
        if b.numel() != C:
            raise ValueError(f"{names[1]}: expected {C} elements, got {b.numel()}")
        if a is not None and kb != kind:
            raise ValueError(f"{names[1]}: expected {a.dtype}, got {b.dtype}")
        kind = kb
        pb = b.data_ptr() if b.is_cuda and b.is_contiguous() else _p(b)
    return kind, pa, pb


def _checkpoint(codes, scales, rows, C):
    """(format, bytes between rows, pointer, pointer) of a checkpoint of [rows, C]."""
    fmt = _formats.get(codes.dtype)
    if fmt is None:
        if not _formats:
            _load_row_types()
            return _checkpoint(codes, scales, rows, C)
        raise ValueError(f"codes: expected int8 or float8_e4m3fn, got {codes.dtype}")
    shape = codes.shape
    ld = shape[-1]
    if shape != (rows, ld):
        _shape("codes", codes, (rows, ld))
    if scales is None or scales.shape != (rows, (C + 127) // 128):
        raise ValueError(f"scales: expected shape {(rows, (C + 127) // 128)}, got "
                         f"{None if scales is None else tuple(scales.shape)}")
    if _row_types.get(scales.dtype) != 1:
        raise ValueError(f"scales: expected float32, got {scales.dtype}")
    if codes.is_cuda and scales.is_cuda and codes.is_contiguous() and scales.is_contiguous():
        return fmt, ld, codes.data_ptr(), scales.data_ptr()
    return fmt, ld, _p(codes), _p(scales)


def _live(offsets):
    """Address of the last of the segments' offsets: the number of live rows."""
    if offsets is None:
        return None
    if offsets.numel() < 1:
        raise ValueError("offsets: expected at least one element, got 0")
    return _typed(offsets, "int32", "offsets") + 4 * (offsets.numel() - 1)


def _kind(kind):
    k = NORMS.get(kind)
    if k is None:
        raise ValueError(f"kind: expected 'layer' or 'rms', got {kind!r}")
    return k


def moe_norm(x, y, gamma=None, beta=None, *, residual=None, total=None, mean=None, rstd=None,
             codes=None, scales=None, eps=1e-5, kind="layer", stream=None):
    """y = normalised rows of x (or of x + residual, written to total) times gamma plus beta; mean
    and rstd [rows] and the 8-bit checkpoint (codes, scales) of what was normalised are for the
    backward pass.  kind: "layer" or "rms" (no mean).  x, residual and total are of one type, y of
    its own (bf16 or fp32), rows may be strided."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x: expected a matrix, got {len(shape)} dimensions")
    rows, C = shape
    px, xt, ldx = _rows(x, "x", shape)
    py, yt, ldy = _rows(y, "y", shape)
    pr = pt = pc = ps = None
    ldr = ldt = fmt = ldc = 0
    if residual is not None:
        pr, _, ldr = _rows(residual, "residual", shape, xt)
    if total is not None:
        pt, _, ldt = _rows(total, "total", shape, xt)
    if codes is not None:
        fmt, ldc, pc, ps = _checkpoint(codes, scales, rows, C)
    elif scales is not None:
        raise ValueError("scales: given without codes")
    kt, pg, pb = _params(C, gamma, beta, ("gamma", "beta"))
    p, at = _norm_struct(rows, C, _kind(kind), eps, xt, yt, kt, 0, fmt, ldx, ldr, ldy, ldt, ldc)
    s = (_lib or lib()).moe_norm(at, px, pr, pg, pb, py, pt, _vector(mean, "mean", rows),
                                 _vector(rstd, "rstd", rows), pc, ps, _s(stream))
    if s:
        raise MoEError(s, "moe_norm")


def moe_norm_ws_size(rows, C) -> int:
    """Bytes of the workspace of moe_norm_bwd."""
    return lib().moe_norm_ws_size(int(rows), int(C))


def moe_norm_bwd(dy, x, mean, rstd, dx, dgamma=None, dbeta=None, *, gamma=None, scales=None,
                 add=None, kind="layer", ws, stream=None):
    """Gradient of moe_norm: dx (plus add, the gradient that reaches the rows by another way),
    dgamma and dbeta.  x: the rows that were normalised, or with scales the codes of their
    checkpoint.  dx and add are of one type (x's, if x is not codes); mean is None for kind="rms"."""
    shape = dy.shape
    if len(shape) != 2:
        raise ValueError(f"dy: expected a matrix, got {len(shape)} dimensions")
    rows, C = shape
    py, yt, ldy = _rows(dy, "dy", shape)
    pd, xt, ldd = _rows(dx, "dx", shape)
    pa = ps = None
    lda = ldx = fmt = ldc = 0
    if scales is None:
        px, _, ldx = _rows(x, "x", shape, xt)
    else:
        fmt, ldc, px, ps = _checkpoint(x, scales, rows, C)
    if add is not None:
        pa, _, lda = _rows(add, "add", shape, xt)
    kt, pg, _ = _params(C, gamma, None, ("gamma", ""))
    gt, pdg, pdb = _params(C, dgamma, dbeta, ("dgamma", "dbeta"))
    if (dgamma is not None or dbeta is not None) and not isinstance(ws, int):
        need = moe_norm_ws_size(rows, C)
        if ws.numel() * ws.element_size() < need:
            raise ValueError(f"ws: expected {need} bytes, got {ws.numel() * ws.element_size()}")
    p, at = _norm_struct(rows, C, _kind(kind), 0.0, xt, yt, kt, gt, fmt, ldx, lda, ldy, ldd, ldc)
    _check(lib().moe_norm_bwd(at, py, px, ps, _vector(mean, "mean", rows),
                              _vector(rstd, "rstd", rows), pg, pa, pd, pdg, pdb, _p(ws),
                              _s(stream)), "moe_norm_bwd")


def moe_ckpt_norm(codes, scales, mean, rstd, y, gamma=None, beta=None, *, kind="layer",
                  stream=None):
    """moe_norm's y again, from the checkpoint and the statistics of what was normalised."""
    shape = y.shape
    if len(shape) != 2:
        raise ValueError(f"y: expected a matrix, got {len(shape)} dimensions")
    rows, C = shape
    py, yt, ldy = _rows(y, "y", shape)
    fmt, ldc, pc, ps = _checkpoint(codes, scales, rows, C)
    kt, pg, pb = _params(C, gamma, beta, ("gamma", "beta"))
    p, at = _norm_struct(rows, C, _kind(kind), 0.0, yt, yt, kt, 0, fmt, 0, 0, ldy, 0, ldc)
    _check(lib().moe_ckpt_norm(at, pc, ps, _vector(mean, "mean", rows),
                               _vector(rstd, "rstd", rows), pg, pb, py, _s(stream)),
           "moe_ckpt_norm")


def moe_ckpt_save(x, codes, scales, *, offsets=None, ws, stream=None):
    """Rows of x (bf16 or fp32) into 8 bits: codes int8 or float8_e4m3fn [rows, ld], scales [rows,
    ceil(C / 128)].  offsets: the segments' offsets, whose last entry says how many rows are
    live."""
    if x.dim() != 2:
        raise ValueError(f"x: expected a matrix, got {x.dim()} dimensions")
    rows, C = x.shape
    px, xt, ldx = _rows(x, "x", x.shape)
    fmt, ld, pc, ps = _checkpoint(codes, scales, rows, C)
    p, at = _ckpt_struct(rows, C, fmt, xt, ldx, ld)
    _check(lib().moe_ckpt_save(at, px, _live(offsets), pc, ps, _p(ws), _s(stream)),
           "moe_ckpt_save")


def moe_ckpt_load(codes, scales, x, *, offsets=None, ws, stream=None):
    """The rows x (bf16 or fp32) that a checkpoint stands for."""
    if x.dim() != 2:
        raise ValueError(f"x: expected a matrix, got {x.dim()} dimensions")
    rows, C = x.shape
    px, xt, ldx = _rows(x, "x", x.shape)
    fmt, ld, pc, ps = _checkpoint(codes, scales, rows, C)
    p, at = _ckpt_struct(rows, C, fmt, xt, ldx, ld)
    _check(lib().moe_ckpt_load(at, pc, ps, _live(offsets), px, _p(ws), _s(stream)),
           "moe_ckpt_load")


def moe_ckpt_swiglu(codes, scales, ab=None, h=None, *, offsets=None, ws, stream=None):
    """ab = [a | b] (bf16) and h = silu(a) * b (bf16) from the checkpoint of [a | b]."""
    if ab is None and h is None:
        raise ValueError("ab, h: expected at least one of them")
    rows = codes.shape[0]
    C = ab.shape[-1] if ab is not None else 2 * h.shape[-1]
    if C % 2:
        raise ValueError(f"ab: expected an even number of columns, got {C}")
    if ab is not None:
        _shape("ab", ab, (rows, C))
    if h is not None:
        _shape("h", h, (rows, C // 2))
    fmt, ld, pc, ps = _checkpoint(codes, scales, rows, C)
    p, at = _ckpt_struct(rows, C, fmt, 0, C, ld)
    _check(lib().moe_ckpt_swiglu(at, pc, ps, _live(offsets), _bf16(ab, "ab"),
                                 _bf16(h, "h"), _p(ws), _s(stream)),
           "moe_ckpt_swiglu")


def moe_ckpt_swiglu_bwd(dh, codes, scales, dab, h=None, *, offsets=None, ws, stream=None):
    """dab = [da | db] of h = silu(a) * b (bf16), and h, from dh (bf16) and the checkpoint of
    [a | b]."""
    if dh.dim() != 2:
        raise ValueError(f"dh: expected a matrix, got {dh.dim()} dimensions")
    rows, f = dh.shape
    _shape("dab", dab, (rows, 2 * f))
    if h is not None:
        _shape("h", h, (rows, f))
    fmt, ld, pc, ps = _checkpoint(codes, scales, rows, 2 * f)
    p, at = _ckpt_struct(rows, 2 * f, fmt, 0, 2 * f, ld)
    _check(lib().moe_ckpt_swiglu_bwd(at, _bf16(dh, "dh"), pc, ps,
                                     _live(offsets), _bf16(dab, "dab"),
                                     _bf16(h, "h"), _p(ws), _s(stream)),
           "moe_ckpt_swiglu_bwd")


_ckpt_combine_buffers = _Buffers("dy", "topk_w", "dest_row", "dyp", "dw")


def moe_ckpt_combine_bwd(cfg, dy, codes, scales, topk_w, dest_row, dyp, dw, ws, stream=None):
    """moe_combine_bwd_dw with the experts' outputs from their checkpoint."""
    n = cfg.T * cfg.k
    fmt, ld, pc, ps = _checkpoint(codes, scales, n, cfg.d)
    pdy, pw, pr, pdyp, pdw = _ckpt_combine_buffers((dy, topk_w, dest_row, dyp, dw),
                                                   [cfg.T * cfg.d, n, n, n * cfg.d, n])
    _check(lib().moe_ckpt_combine_bwd(_addr(cfg), pdy, pc, ld, ps, fmt, pw, pr, pdyp, pdw, _p(ws),
                                      _s(stream)), "moe_ckpt_combine_bwd")


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


CKPT_FORMATS = ("int8", "e4m3")


def _new_checkpoint(rows, C, fmt, device):
    """(codes, scales) for rows of C columns."""
    import torch
    if fmt not in CKPT_FORMATS:
        raise ValueError(f"checkpoint: expected one of {CKPT_FORMATS}, got {fmt!r}")
    codes = torch.empty((rows, (C + 15) // 16 * 16), dtype=torch.int8, device=device)
    if fmt == "e4m3":
        codes = codes.view(torch.float8_e4m3fn)
    return codes, torch.empty((rows, (C + 127) // 128), dtype=torch.float32, device=device)


class MoEScratch:
    """The full-size buffers of a CheckpointedMoELayer: none is read after the call that wrote it, so
    the layers of one configuration share one (on one stream).  Its ws serves the norms of the same
    rows too: MoENorm(T, d, ws=scratch.ws)."""

    def __init__(self, cfg: MoEConfigC, device="cuda"):
        import torch
        R, d, f = cfg.T * cfg.k, cfg.d, cfg.ffn
        bf = dict(dtype=torch.bfloat16, device=device)
        self.cfg, self.device = cfg, device
        self.ws = torch.empty(max(moe_stage_workspace_size(cfg), moe_norm_ws_size(cfg.T, d)),
                              dtype=torch.uint8, device=device)
        moe_ws_init(self.ws)
        self.ab, self.dab = torch.empty((R, 2 * f), **bf), torch.empty((R, 2 * f), **bf)
        self.h = torch.empty((R, f), **bf)
        self.rows, self.dxp = torch.empty((R, d), **bf), torch.empty((R, d), **bf)
        self.dw = torch.empty((cfg.T, cfg.k), dtype=torch.float32, device=device)


class CheckpointedMoELayer:
    """MoELayer (bf16, no shared expert) that keeps for its backward pass the routing and, in 8 bits,
    the first product's output and the experts' outputs; everything else is scratch.

        scratch = MoEScratch(cfg)
        layers = [CheckpointedMoELayer(scratch) for _ in range(n)]
        y = layer.forward(logits, x, W1, W2)
        g = layer.backward(logits, x, dy, W1, W2)     # dx, dW1, dW2, dlogits
    """

    def __init__(self, scratch: MoEScratch, checkpoint="int8"):
        import torch
        c, device = scratch.cfg, scratch.device
        if c.ffn_shared:
            raise ValueError("CheckpointedMoELayer has no shared expert")
        if c.mxfp8 or c.recompute:
            raise ValueError("CheckpointedMoELayer: cfg.mxfp8 and cfg.recompute must be unset")
        self.cfg, self.scratch = c, scratch
        T, k, E, R = c.T, c.k, c.E, c.T * c.k
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        i32 = torch.int32
        self.r = {"topk_idx": new((T, k), i32), "topk_w": new((T, k), torch.float32),
                  "counts": new((E,), i32), "kept": new((E,), i32), "offsets": new((E + 1,), i32),
                  "dest_row": new((T, k), i32), "src_tok": new((R,), i32),
                  "src_slot": new((R,), i32), "drop_mask": new((T, k), torch.uint8)}
        self.ab = _new_checkpoint(R, 2 * c.ffn, checkpoint, device)
        self.yp = _new_checkpoint(R, c.d, checkpoint, device)
        # the gate's gradient: that of weights renormalised over the chosen, whatever chose them (for
        # logits whose weights are no numbers, such as infinities, the limit's, where moe_combine_bwd's
        # are NaN too)
        softmax = c.gate == GATES["softmax"]
        self._gate = (make_config(T, c.d, E, k, c.ffn, route_scale=1.0 if softmax else c.route_scale),
                      make_router("softmax" if softmax else "sigmoid", renorm=True))

    def forward(self, logits, x, W1, W2, y=None, stream=None):
        import torch
        c, r, s = self.cfg, self.r, self.scratch
        if y is None:
            y = torch.empty_like(x)
        moe_route(c, logits, *r.values(), s.ws, stream)
        moe_grouped_ffn_gather(c, x, r["src_tok"], r["offsets"], W1, W2, s.ab, s.h, s.rows, s.ws,
                               stream)
        moe_ckpt_save(s.ab, *self.ab, offsets=r["offsets"], ws=s.ws, stream=stream)
        moe_ckpt_save(s.rows, *self.yp, offsets=r["offsets"], ws=s.ws, stream=stream)
        moe_combine(c, s.rows, r["dest_row"], r["topk_w"], None, y, s.ws, stream)
        return y

    def backward(self, logits, x, dy, W1, W2, out=None, stream=None):
        """After forward() on the same logits, x and weights; other layers may have used the scratch
        in between."""
        import torch
        c, r, s = self.cfg, self.r, self.scratch
        if out is None:
            out = {"dx": torch.empty_like(x), "dW1": torch.empty_like(W1),
                   "dW2": torch.empty_like(W2), "dlogits": torch.empty_like(logits)}
        moe_ckpt_combine_bwd(c, dy, *self.yp, r["topk_w"], r["dest_row"], s.rows, s.dw, s.ws, stream)
        moe_route_groups_bwd(*self._gate, logits, r["topk_idx"], s.dw, out["dlogits"], s.ws, stream)
        moe_ckpt_swiglu(*self.ab, s.ab, s.h, offsets=r["offsets"], ws=s.ws, stream=stream)
        moe_grouped_ffn_bwd_gather(c, s.rows, x, r["src_tok"], r["offsets"], W1, W2, s.ab, s.h, s.dab,
                                   s.dxp, out["dW1"], out["dW2"], s.ws, stream)
        moe_unpermute_reduce(c, s.dxp, r["dest_row"], None, out["dx"], s.ws, stream)
        return out

    def status(self, stream=None):
        return moe_status(self.scratch.ws, stream)


class MoENorm:
    """The normalisation in front of a layer, with what its backward pass needs: the statistics and,
    in 8 bits, the rows that were normalised (checkpoint None: the caller's tensor itself).

        norm = MoENorm(T, d)
        n, s = norm.forward(x, gamma, beta, residual=r)     # s = x + r, n = norm(s)
        n = norm.restore(gamma, beta)                       # n again, for the layer's backward pass
        g = norm.backward(dn, gamma, add=ds)                # dx (of x and of r), dgamma, dbeta

    ws: the workspace of another call on the same stream (a layer's or a MoEScratch's, or any of
    moe_norm_ws_size(T, d) bytes after moe_ws_init), written only while backward runs.  Up to 608 d
    pairs of fp32 sums: below some 5000 rows more than the checkpoint saves, so the norms of a model
    share one.  None: one of its own.
    """

    def __init__(self, T, d, kind="layer", eps=1e-5, dtype=None, checkpoint="int8", device="cuda",
                 ws=None):
        import torch
        _kind(kind)
        self.T, self.d, self.kind, self.eps = int(T), int(d), kind, float(eps)
        self.dtype = torch.bfloat16 if dtype is None else dtype     # of the stream
        f32 = dict(dtype=torch.float32, device=device)
        self.mean = torch.empty(self.T, **f32) if kind == "layer" else None
        self.rstd = torch.empty(self.T, **f32)
        self.kept = _new_checkpoint(self.T, self.d, checkpoint, device) if checkpoint else None
        self.x = None
        need = moe_norm_ws_size(self.T, self.d)
        if ws is None:
            ws = torch.empty(need, dtype=torch.uint8, device=device)
            moe_ws_init(ws)
        elif ws.numel() * ws.element_size() < need:
            raise ValueError(f"ws: expected {need} bytes, got {ws.numel() * ws.element_size()}")
        self.ws = ws

    def forward(self, x, gamma=None, beta=None, residual=None, stream=None):
        """(y in bf16, what was normalised: x itself or the sum)."""
        import torch
        _shape("x", x, (self.T, self.d))
        if x.dtype is not self.dtype:
            raise ValueError(f"x: expected {self.dtype}, got {x.dtype}")
        y = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
        total = None if residual is None else torch.empty_like(x)
        codes, scales = self.kept or (None, None)
        moe_norm(x, y, gamma, beta, residual=residual, total=total, mean=self.mean, rstd=self.rstd,
                 codes=codes, scales=scales, eps=self.eps, kind=self.kind, stream=stream)
        v = x if total is None else total
        self.x = None if self.kept else v
        return y, v

    def restore(self, gamma=None, beta=None, stream=None):
        import torch
        y = torch.empty((self.T, self.d), dtype=torch.bfloat16, device=self.rstd.device)
        if self.kept:
            moe_ckpt_norm(*self.kept, self.mean, self.rstd, y, gamma, beta, kind=self.kind,
                          stream=stream)
        else:
            moe_norm(self.x, y, gamma, beta, eps=self.eps, kind=self.kind, stream=stream)
        return y

    def backward(self, dy, gamma=None, add=None, beta=False, stream=None):
        """dx (plus add), dgamma in fp32, and with beta=True dbeta."""
        import torch
        f32 = dict(dtype=torch.float32, device=dy.device)
        out = {"dx": torch.empty((self.T, self.d), dtype=self.dtype, device=dy.device),
               "dgamma": torch.empty(self.d, **f32)}
        if beta:
            out["dbeta"] = torch.empty(self.d, **f32)
        x, scales = self.kept or (self.x, None)
        moe_norm_bwd(dy, x, self.mean, self.rstd, out["dx"], out["dgamma"], out.get("dbeta"),
                     gamma=gamma, scales=scales, add=add, kind=self.kind, ws=self.ws, stream=stream)
        return out

    def status(self, stream=None):
        """Of backward, whose copies are waited for with a limit (and of all that share the workspace)."""
        return moe_status(self.ws, stream)


class Fp8MoELayer:
    """A layer whose router limits the choice to groups of experts and whose routed experts run
    on 8-bit operands with a scale per block of 128, forward and backward.  Owns its buffers;
    the weights are quantised once per update (quantize_weights) and passed to every call.

        layer = Fp8MoELayer(cfg, make_router("sigmoid", groups=8, top_groups=4, group_top=2))
        w = layer.quantize_weights(W1, W2)
        y = layer.forward(logits, x, w)
        g = layer.backward(logits, x, dy, w)      # dx, dW1, dW2, dlogits

    checkpoint ("int8" or "e4m3"): what the backward pass reads of the forward's, the first product's
    output and the experts' outputs, is kept in 8 bits instead of bf16.  Then everything else but the
    routing is scratch, and `scratch`, another layer of the same configuration, lends its own: a
    model's layers keep 8 bits each and share one set of full-size buffers (on one stream).
    The gradient then differs in two ways: it is taken at the restored values, and [da | db] and h are
    rounded to bf16 before they become 8-bit operands, where the layer without checkpoints quantises
    them from fp32.
    """

    def __init__(self, cfg: MoEConfigC, router: MoERouterC, device="cuda", grad_dtype=None,
                 checkpoint=None, scratch=None):
        import torch
        if cfg.ffn_shared:
            raise ValueError("Fp8MoELayer has no shared expert")
        if scratch is not None and (checkpoint is None or scratch.checkpoint is None):
            raise ValueError("scratch: only between layers with checkpoints")
        self.cfg, self.router, self.device = cfg, router, device
        self.grad_dtype = torch.bfloat16 if grad_dtype is None else grad_dtype
        T, k, E, d, f = cfg.T, cfg.k, cfg.E, cfg.d, cfg.ffn
        R = T * k
        B = moe_fp8_token_blocks(R, E)
        new = lambda shape, dt: torch.empty(shape, dtype=dt, device=device)  # noqa: E731
        i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
        e4 = torch.float8_e4m3fn
        blk = lambda n: (n + 127) // 128  # noqa: E731
        self.r = {"topk_idx": new((T, k), i32), "topk_w": new((T, k), f32),
                  "counts": new((E,), i32), "kept": new((E,), i32), "offsets": new((E + 1,), i32),
                  "dest_row": new((T, k), i32), "src_tok": new((R,), i32),
                  "src_slot": new((R,), i32), "drop_mask": new((T, k), torch.uint8)}
        self.checkpoint = checkpoint
        if checkpoint is not None:
            self.kept = {n: _new_checkpoint(R, c, checkpoint, device)
                         for n, c in (("ab", 2 * f), ("yp", d))}
        if scratch is not None:
            o = scratch.cfg
            if (o.T, o.k, o.E, o.d, o.ffn) != (T, k, E, d, f):
                raise ValueError("scratch: expected a layer of the same configuration")
            for n in ("ws", "ab", "yp", "q", "qt", "dyp", "dh", "dxp", "dw", "h"):
                setattr(self, n, getattr(scratch, n))
            return
        stages = moe_workspace_size(cfg)[0] if checkpoint is None else moe_stage_workspace_size(cfg)
        self.ws = new((max(stages, moe_norm_ws_size(T, d)),), torch.uint8)
        moe_ws_init(self.ws)
        self.h = new((R, f), bf) if checkpoint is not None else None
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
        if self.checkpoint is not None:
            moe_ckpt_save(self.ab, *self.kept["ab"], **seg)
        moe_fp8_swiglu(self.ab, *self.q["h"], **seg)
        moe_fp8_gemm(*self.q["h"], *w["W2"], self.yp, c.ffn, **seg)
        if self.checkpoint is not None:
            moe_ckpt_save(self.yp, *self.kept["yp"], **seg)
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
        if self.checkpoint is not None:
            moe_ckpt_combine_bwd(c, dy, *self.kept["yp"], r["topk_w"], r["dest_row"], self.dyp,
                                 self.dw, ws, stream)
        else:
            moe_combine_bwd_dw(c, dy, self.yp, r["topk_w"], r["dest_row"], self.dyp, self.dw, ws,
                               stream)
        moe_route_groups_bwd(c, self.router, logits, r["topk_idx"], self.dw, out["dlogits"], ws,
                             stream)
        moe_fp8_quantize(self.dyp, *self.q["dy"], *self.qt["dy"], **seg)
        moe_fp8_gemm(*self.q["dy"], *w["W2_t"], self.dh, c.d, **seg)
        if self.checkpoint is not None:
            dab = self.ab          # (the forward's is not read any more)
            # The checkpoint's gradient leaves [da | db] and h in bf16, which the quantiser reads: a
            # rounding of at most 2^-8 of a value before E4M3's own of up to 2^-4, and 21 bytes a column
            # of f moved where one pass from fp32 would move 9.  8192 tokens, top-8 of 128 experts of
            # 2048 x 768: the backward takes 1.53 ms, without checkpoints 1.54.
            moe_ckpt_swiglu_bwd(self.dh, *self.kept["ab"], dab, self.h, **seg)
            moe_fp8_quantize(dab, *self.q["dab"], *self.qt["dab"], **seg)
            moe_fp8_quantize(self.h, codes_t=self.qt["h"][0], scales_t=self.qt["h"][1], **seg)
        else:
            moe_fp8_swiglu_bwd(self.dh, self.ab, *self.q["dab"], *self.qt["dab"], *self.qt["h"],
                               **seg)
        moe_fp8_wgrad(*self.qt["dy"], *self.qt["h"], out["dW2"], rows=R, **seg)
        moe_fp8_gemm(*self.q["dab"], *w["W1_t"], self.dxp, 2 * c.ffn, **seg)
        moe_unpermute_reduce(c, self.dxp, r["dest_row"], None, out["dx"], ws, stream)
        moe_fp8_quantize(x, codes_t=self.qt["x"][0], scales_t=self.qt["x"][1],
                         src_tok=r["src_tok"], **seg)
        moe_fp8_wgrad(*self.qt["dab"], *self.qt["x"], out["dW1"], rows=R, **seg)
        return out

    def status(self, stream=None):
        return moe_status(self.ws, stream)

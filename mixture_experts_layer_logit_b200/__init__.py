"""Python binding of libmoe, the sm_100a MoE-layer forward library.

Argument marshalling only: every step of the layer runs in the CUDA kernels of
``libmoe.so`` behind the C ABI declared in ``include/moe.h``.  PyTorch is used
for device memory and streams; tensors are passed as raw device pointers and
the current torch stream is used unless another one is given.  There is no
CPU fallback: if the library is missing, loading it raises.

Python names match the C entry points: ``moe_route``, ``moe_permute``,
``moe_expert_ffn``, ``moe_combine``, ``moe_layer_forward``, plus
``moe_scratch_size``, ``moe_workspace_size`` and ``moe_status_string``.
Around the layer: ``moe_layer_norm_forward`` / ``_backward``,
``moe_balance_loss`` and ``moe_adamw_step``; these also check that a tensor they
are given is contiguous, of the configured type and size, and on the current
device.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "LIB_PATH", "MoeError", "moe_config", "moe_stats", "moe_ws_layout", "lib", "make_config",
    "moe_status_string", "moe_scratch_size", "moe_workspace_size", "moe_route", "moe_permute",
    "moe_expert_ffn", "moe_combine", "moe_layer_forward", "moe_convert_bf16_to_f16", "moe_permute_static",
    "moe_expert_ffn_combine", "MOE_STATIC_SCRATCH_BYTES", "prepare_w2", "moe_aux_coef_update",
    "moe_aux_coef_next", "moe_testing_set_expert_wait", "moe_testing_set_norm_wait", "moe_segments_scratch_size",
    "moe_expert_ffn_segments",
    "moe_backward_workspace_size", "moe_layer_backward", "moe_mxfp8_weight_bytes", "moe_prepare_mxfp8_weights",
    "moe_workspace_size_mxfp8", "moe_layer_forward_mxfp8", "prepare_mxfp8", "moe_workspace_size_shared",
    "moe_layer_forward_shared",
    "moe_route_scores", "moe_layer_forward_scores", "moe_layer_backward_scores",
    "moe_norm_config", "make_norm_config", "moe_layer_norm_workspace_size", "moe_layer_norm_forward",
    "moe_layer_norm_backward", "moe_balance_config", "make_balance_config", "moe_balance_workspace_size",
    "moe_balance_loss", "moe_adamw_tensor", "moe_adamw_hyper", "adamw_tensor", "adamw_states", "AdamWPlan",
    "make_adamw_plan", "moe_adamw_step", "MOE_ADAMW_BLOCK", "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID",
    "read_stats", "STATS_BYTES", "MOE_ACT_RELU", "MOE_ACT_SWIGLU", "MOE_DTYPE_F32", "MOE_DTYPE_BF16",
    "MOE_DTYPE_F16", "MOE_DEV_TIMEOUT", "MOE_DEV_BOUNDS", "MOE_DEV_RANGE", "EXPORTED_SYMBOLS",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe.so")

MOE_ACT_RELU, MOE_ACT_SWIGLU = 0, 1
MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_F16 = 0, 1, 2
MOE_DEV_TIMEOUT, MOE_DEV_BOUNDS, MOE_DEV_RANGE = 1, 2, 4
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_WORKSPACE", 4: "MOE_ERR_CUDA"}

EXPORTED_SYMBOLS = ["moe_status_string", "moe_scratch_size", "moe_workspace_size", "moe_route",
                    "moe_permute", "moe_expert_ffn", "moe_combine", "moe_layer_forward",
                    "moe_convert_bf16_to_f16", "moe_permute_static", "moe_expert_ffn_combine",
                    "moe_aux_coef_update", "moe_aux_coef_next", "moe_testing_set_expert_wait",
                    "moe_testing_set_norm_wait",
                    "moe_segments_scratch_size", "moe_expert_ffn_segments", "moe_backward_workspace_size",
                    "moe_layer_backward", "moe_mxfp8_weight_bytes", "moe_prepare_mxfp8_weights",
                    "moe_workspace_size_mxfp8", "moe_layer_forward_mxfp8", "moe_workspace_size_shared",
                    "moe_layer_forward_shared", "moe_layer_norm_workspace_size", "moe_layer_norm_forward",
                    "moe_layer_norm_backward", "moe_route_scores", "moe_layer_forward_scores",
                    "moe_layer_backward_scores", "moe_balance_workspace_size", "moe_balance_loss", "moe_adamw_step"]
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_ADAMW_BLOCK = 256
MOE_STATIC_SCRATCH_BYTES = 2 << 20


class moe_config(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32), ("F", ctypes.c_int32),
                ("k", ctypes.c_int32), ("act", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("capacity_factor", ctypes.c_float), ("lambda_", ctypes.c_float),
                ("hidden_dtype", ctypes.c_int32)]


class moe_stats(ctypes.Structure):
    _fields_ = [("drop_count", ctypes.c_int32), ("rows_kept", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("near_tie_count", ctypes.c_int32), ("drop_rate", ctypes.c_float), ("aux_loss", ctypes.c_float),
                ("status", ctypes.c_uint32), ("z_loss", ctypes.c_float)]


class moe_ws_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ["topk_idx", "topk_w", "gap", "counts", "kept", "offsets", "row_of", "src_tok", "row_w",
                 "xp", "h", "yp", "scratch", "total"]]


class moe_norm_config(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("d", ctypes.c_int32), ("eps", ctypes.c_float)] + [
        (n, ctypes.c_int32) for n in ["x_dtype", "y_dtype", "w_dtype", "add_dtype", "dy_dtype", "dx_dtype"]]


class moe_balance_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ["T", "E", "k", "S", "score", "dtype"]]


class moe_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ["param", "grad", "master", "m", "v", "m_scale", "v_scale"]] + [
        ("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
        ("state_bits", ctypes.c_int32), ("weight_decay", ctypes.c_float)]


class moe_adamw_hyper(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ["lr", "beta1", "beta2", "eps"]]


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int, why: str = ""):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)} ({moe_status_string(code)})"
                         + (f": {why}" if why else ""))
        self.code = code


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """Load libmoe.so (built in-tree by ``build.py``); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: run `python -m mixture_experts_layer_logit_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    cfgp = ctypes.POINTER(moe_config)
    st = ctypes.c_int
    L.moe_status_string.argtypes = [st]
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_scratch_size.argtypes = [cfgp]
    L.moe_scratch_size.restype = ctypes.c_size_t
    L.moe_workspace_size.argtypes = [cfgp, ctypes.POINTER(moe_ws_layout)]
    L.moe_workspace_size.restype = ctypes.c_size_t
    L.moe_route.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_permute.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_expert_ffn.argtypes = [cfgp, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_combine.argtypes = [cfgp, P, P, P, P, P]
    L.moe_layer_forward.argtypes = [cfgp, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_convert_bf16_to_f16.argtypes = [P, P, ctypes.c_size_t, P]
    L.moe_permute_static.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, P, P]
    L.moe_expert_ffn_combine.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    f32 = ctypes.c_float
    L.moe_aux_coef_update.argtypes = [P, P, f32, f32, P]
    L.moe_aux_coef_next.argtypes = [f32, f32, f32, f32, ctypes.POINTER(f32)]
    L.moe_testing_set_expert_wait.argtypes = [ctypes.c_uint64, ctypes.c_int32]
    L.moe_testing_set_norm_wait.argtypes = [ctypes.c_uint64, ctypes.c_int32]
    i32 = ctypes.c_int32
    L.moe_segments_scratch_size.argtypes = [cfgp, i32, i32]
    L.moe_segments_scratch_size.restype = ctypes.c_size_t
    L.moe_expert_ffn_segments.argtypes = [cfgp, i32, i32, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    sz = ctypes.POINTER(ctypes.c_size_t)
    L.moe_mxfp8_weight_bytes.argtypes = [cfgp, sz, sz, sz, sz]
    L.moe_mxfp8_weight_bytes.restype = ctypes.c_size_t
    L.moe_prepare_mxfp8_weights.argtypes = [cfgp, P, P, P, P, P, P, P]
    L.moe_workspace_size_mxfp8.argtypes = [cfgp]
    L.moe_workspace_size_mxfp8.restype = ctypes.c_size_t
    L.moe_layer_forward_mxfp8.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_workspace_size_shared.argtypes = [cfgp, i32]
    L.moe_workspace_size_shared.restype = ctypes.c_size_t
    L.moe_layer_forward_shared.argtypes = [cfgp, i32, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_backward_workspace_size.argtypes = [cfgp]
    L.moe_backward_workspace_size.restype = ctypes.c_size_t
    L.moe_layer_backward.argtypes = [cfgp, P, P, P, P, P, P, f32, f32, P, ctypes.c_size_t, P, P, P, P, P, P, P, P,
                                     ctypes.c_size_t, P]
    normp, balp = ctypes.POINTER(moe_norm_config), ctypes.POINTER(moe_balance_config)
    L.moe_layer_norm_workspace_size.argtypes = [normp]
    L.moe_layer_norm_workspace_size.restype = ctypes.c_size_t
    L.moe_layer_norm_forward.argtypes = [normp] + [P] * 9
    L.moe_layer_norm_backward.argtypes = [normp] + [P] * 11 + [ctypes.c_size_t, P]
    L.moe_route_scores.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_layer_forward_scores.argtypes = [cfgp, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    L.moe_layer_backward_scores.argtypes = [cfgp, P, P, P, P, P, P, P, f32, f32, P, ctypes.c_size_t, P, P, P, P, P, P,
                                            P, P, ctypes.c_size_t, P]
    L.moe_balance_workspace_size.argtypes = [balp]
    L.moe_balance_workspace_size.restype = ctypes.c_size_t
    L.moe_balance_loss.argtypes = [balp] + [P] * 10 + [ctypes.c_size_t, P]
    L.moe_adamw_step.argtypes = [ctypes.POINTER(moe_adamw_tensor), i32, ctypes.POINTER(moe_adamw_hyper), P, P, P, P]
    for n in ["moe_route", "moe_permute", "moe_expert_ffn", "moe_combine", "moe_layer_forward",
              "moe_convert_bf16_to_f16", "moe_permute_static", "moe_expert_ffn_combine", "moe_aux_coef_update",
              "moe_aux_coef_next", "moe_testing_set_expert_wait", "moe_testing_set_norm_wait",
              "moe_expert_ffn_segments", "moe_layer_backward",
              "moe_prepare_mxfp8_weights", "moe_layer_forward_mxfp8", "moe_layer_forward_shared",
              "moe_layer_norm_forward", "moe_layer_norm_backward", "moe_route_scores", "moe_layer_forward_scores",
              "moe_layer_backward_scores", "moe_balance_loss", "moe_adamw_step"]:
        getattr(L, n).restype = st
    _lib = L
    return L


_DTYPES = {"f32": MOE_DTYPE_F32, "bf16": MOE_DTYPE_BF16, "f16": MOE_DTYPE_F16}


def make_config(T: int, d: int, E: int, F: int, k: int, act: str = "relu", dtype: str = "bf16",
                capacity_factor: float = 0.0, lam: float = 0.0, hidden: Optional[str] = None) -> moe_config:
    """hidden: element type of the expert hidden activation and of W2 on the bf16
    path ("f16", the default, or "bf16"); always "f32" on the fp32 path."""
    if hidden is None:
        hidden = "f16" if dtype == "bf16" else "f32"
    return moe_config(T, d, E, F, k, MOE_ACT_SWIGLU if act == "swiglu" else MOE_ACT_RELU, _DTYPES[dtype],
                      capacity_factor, lam, _DTYPES[hidden])


def _ptr(t) -> Optional[int]:
    """Device pointer of a tensor (None -> NULL); also accepts raw ints."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # without a Stream object: 0.1 us instead of 3
        return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def _check(fn: str, code: int):
    if code != 0:
        raise MoeError(fn, code)


def moe_status_string(code: int) -> str:
    return lib().moe_status_string(code).decode()


def moe_scratch_size(cfg: moe_config) -> int:
    return lib().moe_scratch_size(ctypes.byref(cfg))


def moe_workspace_size(cfg: moe_config):
    """(bytes, moe_ws_layout) of the moe_layer_forward workspace."""
    L = moe_ws_layout()
    n = lib().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(L))
    return n, L


def moe_route(cfg, x, Wg, bg, topk_idx, topk_w, gap, prob_mean, ws, stream=None, z_loss=None):
    """z_loss: optional device fp32 scalar that receives the router z-loss."""
    _check("moe_route", lib().moe_route(ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(topk_idx),
                                        _ptr(topk_w), _ptr(gap), _ptr(prob_mean), _ptr(z_loss), _ptr(ws),
                                        _nbytes(ws), _stream(stream)))


def moe_permute(cfg, x, topk_idx, gap, prob_mean, counts, kept, offsets, row_of, src_tok, xp, stats, ws,
                stream=None):
    _check("moe_permute", lib().moe_permute(ctypes.byref(cfg), _ptr(x), _ptr(topk_idx), _ptr(gap),
                                            _ptr(prob_mean), _ptr(counts), _ptr(kept), _ptr(offsets),
                                            _ptr(row_of), _ptr(src_tok), _ptr(xp), _ptr(stats), _ptr(ws),
                                            _nbytes(ws), _stream(stream)))


def moe_permute_static(cfg, x, topk_idx, gap, prob_mean, counts, kept, offsets, row_of, src_tok, xp, stats,
                       stream=None):
    """moe_permute with its scratch in the library's fixed device array (no
    workspace argument; calls that overlap in time race on that array)."""
    _check("moe_permute_static", lib().moe_permute_static(ctypes.byref(cfg), _ptr(x), _ptr(topk_idx), _ptr(gap),
                                                          _ptr(prob_mean), _ptr(counts), _ptr(kept),
                                                          _ptr(offsets), _ptr(row_of), _ptr(src_tok), _ptr(xp),
                                                          _ptr(stats), _stream(stream)))


def moe_expert_ffn(cfg, xp, offsets, W1, W2, h, yp, stats, ws, stream=None):
    _check("moe_expert_ffn", lib().moe_expert_ffn(ctypes.byref(cfg), _ptr(xp), _ptr(offsets), _ptr(W1),
                                                  _ptr(W2), _ptr(h), _ptr(yp), _ptr(stats), _ptr(ws),
                                                  _nbytes(ws), _stream(stream)))


def moe_expert_ffn_combine(cfg, xp, offsets, src_tok, row_w, W1, W2, h, out, stats, ws, stream=None):
    """Steps 4-5 fused (bf16, k <= 2): out (zeroed by the caller) += gate-weighted expert outputs.
    ws is a moe_layer_forward workspace."""
    _check("moe_expert_ffn_combine",
           lib().moe_expert_ffn_combine(ctypes.byref(cfg), _ptr(xp), _ptr(offsets), _ptr(src_tok), _ptr(row_w),
                                        _ptr(W1), _ptr(W2), _ptr(h), _ptr(out), _ptr(stats), _ptr(ws), _nbytes(ws),
                                        _stream(stream)))


def moe_segments_scratch_size(cfg: moe_config, nseg: int, rows: int) -> int:
    return lib().moe_segments_scratch_size(ctypes.byref(cfg), nseg, rows)


def moe_expert_ffn_segments(cfg, nseg, rows, seg_offsets, xp, W1, W2, h, yp, stats, ws, stream=None):
    """Step 4 over nseg caller-given segments of a rows-row buffer; segment i
    runs through local expert i % cfg.E (the expert-parallel form)."""
    _check("moe_expert_ffn_segments",
           lib().moe_expert_ffn_segments(ctypes.byref(cfg), nseg, rows, _ptr(seg_offsets), _ptr(xp), _ptr(W1),
                                         _ptr(W2), _ptr(h), _ptr(yp), _ptr(stats), _ptr(ws), _nbytes(ws),
                                         _stream(stream)))


def moe_combine(cfg, yp, row_of, topk_w, out, stream=None):
    _check("moe_combine", lib().moe_combine(ctypes.byref(cfg), _ptr(yp), _ptr(row_of), _ptr(topk_w),
                                            _ptr(out), _stream(stream)))


def moe_layer_forward(cfg, x, Wg, bg, W1, W2, out, stats, ws, stream=None):
    _check("moe_layer_forward", lib().moe_layer_forward(ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(bg),
                                                        _ptr(W1), _ptr(W2), _ptr(out), _ptr(stats), _ptr(ws),
                                                        _nbytes(ws), _stream(stream)))


def moe_aux_coef_update(stats, coef, beta: float, xi: float, stream=None):
    """On the device: coef <- beta * coef + (1 - beta) * xi * stats.drop_rate
    (stats: device moe_stats bytes, coef: device fp32 scalar)."""
    _check("moe_aux_coef_update", lib().moe_aux_coef_update(_ptr(stats), _ptr(coef), beta, xi, _stream(stream)))


def moe_aux_coef_next(coef: float, drop_rate: float, beta: float, xi: float) -> float:
    """The same update on the host (no device involved)."""
    out = ctypes.c_float()
    _check("moe_aux_coef_next", lib().moe_aux_coef_next(coef, drop_rate, beta, xi, ctypes.byref(out)))
    return out.value


def moe_testing_set_expert_wait(wait_ns: int, extra_dependency: int):
    """Test hook: limit of the one-launch expert kernel's waits (0 = default)
    and an amount added to its layer-2 dependency target (> 0: unreachable)."""
    _check("moe_testing_set_expert_wait", lib().moe_testing_set_expert_wait(wait_ns, extra_dependency))


def moe_testing_set_norm_wait(wait_ns: int, kept_rounds: int):
    """Test hook: limit of the norm backward's waits (0 = default) and how many
    rounds of rows each of its blocks copies (-1: all)."""
    _check("moe_testing_set_norm_wait", lib().moe_testing_set_norm_wait(wait_ns, kept_rounds))


def moe_workspace_size_shared(cfg: moe_config, F_shared: int) -> int:
    return lib().moe_workspace_size_shared(ctypes.byref(cfg), F_shared)


def moe_layer_forward_shared(cfg, F_shared, x, Wg, bg, W1, W2, W1_shared, W2_shared, out, stats, ws, stream=None):
    """The layer plus a shared expert of hidden width F_shared (every token, weight 1)."""
    _check("moe_layer_forward_shared",
           lib().moe_layer_forward_shared(ctypes.byref(cfg), F_shared, _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1),
                                          _ptr(W2), _ptr(W1_shared), _ptr(W2_shared), _ptr(out), _ptr(stats),
                                          _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_mxfp8_weight_bytes(cfg: moe_config):
    """(total, (w1q, w1s, w2q, w2s)) bytes of the prepared FP8 weights (0 if unsupported)."""
    v = [ctypes.c_size_t() for _ in range(4)]
    n = lib().moe_mxfp8_weight_bytes(ctypes.byref(cfg), *[ctypes.byref(x) for x in v])
    return n, tuple(x.value for x in v)


def moe_prepare_mxfp8_weights(cfg, W1, W2, W1q, W1s, W2q, W2s, stream=None):
    _check("moe_prepare_mxfp8_weights",
           lib().moe_prepare_mxfp8_weights(ctypes.byref(cfg), _ptr(W1), _ptr(W2), _ptr(W1q), _ptr(W1s), _ptr(W2q),
                                           _ptr(W2s), _stream(stream)))


def prepare_mxfp8(cfg, W1, W2):
    """Weight preparation for the FP8 layer: four new uint8 device tensors
    (W1q, W1s, W2q, W2s) from bf16 W1, W2.  Run once at load time."""
    import torch
    n, sizes = moe_mxfp8_weight_bytes(cfg)
    if n == 0:
        raise MoeError("moe_mxfp8_weight_bytes", 2)
    bufs = [torch.empty(max(sz, 16), dtype=torch.uint8, device=W1.device) for sz in sizes]
    moe_prepare_mxfp8_weights(cfg, W1, W2, *bufs)
    return tuple(bufs)


def moe_workspace_size_mxfp8(cfg: moe_config) -> int:
    return lib().moe_workspace_size_mxfp8(ctypes.byref(cfg))


def moe_layer_forward_mxfp8(cfg, x, Wg, bg, W1q, W1s, W2q, W2s, out, stats, ws, stream=None):
    _check("moe_layer_forward_mxfp8",
           lib().moe_layer_forward_mxfp8(ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1q), _ptr(W1s),
                                         _ptr(W2q), _ptr(W2s), _ptr(out), _ptr(stats), _ptr(ws), _nbytes(ws),
                                         _stream(stream)))


def moe_backward_workspace_size(cfg: moe_config) -> int:
    return lib().moe_backward_workspace_size(ctypes.byref(cfg))


def moe_layer_backward(cfg, x, Wg, bg, W1, W2, dout, aux_coef, z_coef, fws, dx, dWg, dbg, dW1, dW2, dw, stats, ws,
                       stream=None):
    """Gradients of <dout, out> + aux_coef * aux + z_coef * z_loss for the forward
    whose workspace is fws (see include/moe.h)."""
    _check("moe_layer_backward",
           lib().moe_layer_backward(ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1), _ptr(W2), _ptr(dout),
                                    aux_coef, z_coef, _ptr(fws), _nbytes(fws), _ptr(dx), _ptr(dWg), _ptr(dbg),
                                    _ptr(dW1), _ptr(dW2), _ptr(dw), _ptr(stats), _ptr(ws), _nbytes(ws),
                                    _stream(stream)))


def moe_convert_bf16_to_f16(src, dst, n: Optional[int] = None, stream=None):
    """Weight preparation: dst = fp16(src) for bf16 src (device tensors)."""
    n = src.numel() if n is None else n
    _check("moe_convert_bf16_to_f16", lib().moe_convert_bf16_to_f16(_ptr(src), _ptr(dst), n, _stream(stream)))


def prepare_w2(cfg: moe_config, w2):
    """W2 in the storage type the layer expects (a new fp16 tensor when the
    hidden activation is fp16, else w2 itself).  Run once at load time."""
    if cfg.hidden_dtype != MOE_DTYPE_F16:
        return w2
    import torch
    out = torch.empty(w2.shape, dtype=torch.float16, device=w2.device)
    moe_convert_bf16_to_f16(w2, out)
    return out


# ------------------------------------------------------------ around the layer
_TORCH_DTYPES = None


def _torch_dtype(code: int):
    global _TORCH_DTYPES
    if _TORCH_DTYPES is None:
        import torch
        _TORCH_DTYPES = {MOE_DTYPE_F32: torch.float32, MOE_DTYPE_BF16: torch.bfloat16, MOE_DTYPE_F16: torch.float16}
    return _TORCH_DTYPES.get(code)


def _current_device() -> int:
    import torch
    try:
        return torch.cuda.current_device()
    except (RuntimeError, AssertionError):   # no CUDA device: -1 is what a CPU tensor says, so nothing matches
        return -2


def _arg(fn: str, name: str, t, dev: int, dtype, n: int) -> Optional[int]:
    """Device pointer of an operand of n contiguous elements of dtype (None and
    raw ints pass as they are); anything else is refused before it is read."""
    if t is None or isinstance(t, int):
        return t
    if t.get_device() != dev:
        raise MoeError(fn, 1, f"{name} is on {t.device}, not on the current CUDA device")
    if t.dtype != dtype:
        raise MoeError(fn, 1, f"{name} is {t.dtype}, not {dtype}")
    if t.numel() != n:
        raise MoeError(fn, 1, f"{name} has {t.numel()} elements, not {n}")
    if not t.is_contiguous():
        raise MoeError(fn, 1, f"{name} is not contiguous")
    return t.data_ptr()


def _stats(fn: str, stats, dev: int) -> Optional[int]:
    return None if stats is None else _arg(fn, "stats", stats, dev, stats.dtype, STATS_BYTES // stats.element_size())


def _workspace(fn: str, ws, dev: int):
    """(pointer, bytes) of a workspace tensor (None: no workspace)."""
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise MoeError(fn, 3, "ws is not a contiguous tensor on the current CUDA device")
    return ws.data_ptr(), _nbytes(ws)


def make_norm_config(rows: int, d: int, eps: float = 1e-5, x: str = "bf16", y: Optional[str] = None, w: str = "f32",
                     add: Optional[str] = None, dy: Optional[str] = None, dx: Optional[str] = None) -> moe_norm_config:
    """Types of the operands ("f32", "bf16", "f16"): y and dx follow x unless
    given; add and dy are fp32 unless given (the layer's out, and its dx)."""
    return moe_norm_config(rows, d, eps, _DTYPES[x], _DTYPES[y or x], _DTYPES[w], _DTYPES[add or "f32"],
                           _DTYPES[dy or "f32"], _DTYPES[dx or x])


def moe_layer_norm_workspace_size(cfg: moe_norm_config) -> int:
    return lib().moe_layer_norm_workspace_size(ctypes.byref(cfg))


def moe_layer_norm_forward(cfg, x, gamma, beta, y, add=None, sum=None, mean=None, rstd=None, stream=None):
    """y = norm(x) * gamma + beta, or of x + add, which sum receives; mean and
    rstd (fp32, one per row) are what the backward takes."""
    fn, dev, n = "moe_layer_norm_forward", _current_device(), cfg.rows * cfg.d
    xt, wt, f32 = _torch_dtype(cfg.x_dtype), _torch_dtype(cfg.w_dtype), _torch_dtype(MOE_DTYPE_F32)
    _check(fn, lib().moe_layer_norm_forward(
        ctypes.byref(cfg), _arg(fn, "x", x, dev, xt, n), _arg(fn, "add", add, dev, _torch_dtype(cfg.add_dtype), n),
        _arg(fn, "gamma", gamma, dev, wt, cfg.d), _arg(fn, "beta", beta, dev, wt, cfg.d),
        _arg(fn, "y", y, dev, _torch_dtype(cfg.y_dtype), n), _arg(fn, "sum", sum, dev, xt, n),
        _arg(fn, "mean", mean, dev, f32, cfg.rows), _arg(fn, "rstd", rstd, dev, f32, cfg.rows), _stream(stream)))


def moe_layer_norm_backward(cfg, dy, x, mean, rstd, gamma, dx, dgamma=None, dbeta=None, ws=None, dsum=None,
                            stats=None, stream=None):
    """dx (of what the forward normalised; dsum is added to it), dgamma, dbeta."""
    fn, dev, n = "moe_layer_norm_backward", _current_device(), cfg.rows * cfg.d
    dxt, f32 = _torch_dtype(cfg.dx_dtype), _torch_dtype(MOE_DTYPE_F32)
    wp, wn = _workspace(fn, ws, dev)
    _check(fn, lib().moe_layer_norm_backward(
        ctypes.byref(cfg), _arg(fn, "dy", dy, dev, _torch_dtype(cfg.dy_dtype), n),
        _arg(fn, "x", x, dev, _torch_dtype(cfg.x_dtype), n), _arg(fn, "mean", mean, dev, f32, cfg.rows),
        _arg(fn, "rstd", rstd, dev, f32, cfg.rows), _arg(fn, "gamma", gamma, dev, _torch_dtype(cfg.w_dtype), cfg.d),
        _arg(fn, "dsum", dsum, dev, dxt, n), _arg(fn, "dx", dx, dev, dxt, n),
        _arg(fn, "dgamma", dgamma, dev, f32, cfg.d), _arg(fn, "dbeta", dbeta, dev, f32, cfg.d),
        _stats(fn, stats, dev), wp, wn, _stream(stream)))


def moe_route_scores(cfg, x, Wg, bg, topk_idx, topk_w, gap, prob_mean, scores, ws, stream=None, z_loss=None):
    """moe_route that also writes the scores the softmax takes (fp32 [T, E])."""
    fn = "moe_route_scores"
    sp = _arg(fn, "scores", scores, _current_device(), _torch_dtype(MOE_DTYPE_F32), cfg.T * cfg.E)
    _check(fn, lib().moe_route_scores(ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(topk_idx), _ptr(topk_w),
                                      _ptr(gap), _ptr(prob_mean), _ptr(z_loss), sp, _ptr(ws), _nbytes(ws),
                                      _stream(stream)))


def moe_layer_forward_scores(cfg, x, Wg, bg, W1, W2, out, stats, scores, ws, stream=None):
    """moe_layer_forward that also writes the router's scores (fp32 [T, E])."""
    fn = "moe_layer_forward_scores"
    sp = _arg(fn, "scores", scores, _current_device(), _torch_dtype(MOE_DTYPE_F32), cfg.T * cfg.E)
    _check(fn, lib().moe_layer_forward_scores(ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1), _ptr(W2),
                                              _ptr(out), _ptr(stats), sp, _ptr(ws), _nbytes(ws), _stream(stream)))


def moe_layer_backward_scores(cfg, x, Wg, bg, W1, W2, dout, dscores, aux_coef, z_coef, fws, dx, dWg, dbg, dW1, dW2,
                              dw, stats, ws, stream=None):
    """moe_layer_backward with a gradient of the scores (fp32 [T, E], e.g.
    moe_balance_loss's dscores) added on its way to dx, dWg and dbg."""
    fn = "moe_layer_backward_scores"
    sp = _arg(fn, "dscores", dscores, _current_device(), _torch_dtype(MOE_DTYPE_F32), cfg.T * cfg.E)
    _check(fn, lib().moe_layer_backward_scores(
        ctypes.byref(cfg), _ptr(x), _ptr(Wg), _ptr(bg), _ptr(W1), _ptr(W2), _ptr(dout), sp, aux_coef, z_coef,
        _ptr(fws), _nbytes(fws), _ptr(dx), _ptr(dWg), _ptr(dbg), _ptr(dW1), _ptr(dW2), _ptr(dw), _ptr(stats),
        _ptr(ws), _nbytes(ws), _stream(stream)))


def make_balance_config(T: int, E: int, k: int, S: int = 1, score: str = "softmax",
                        dtype: str = "f32") -> moe_balance_config:
    """score: "softmax" or "sigmoid" (normalised over the experts); dtype: of the scores."""
    return moe_balance_config(T, E, k, S, {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}[score],
                              _DTYPES[dtype])


def moe_balance_workspace_size(cfg: moe_balance_config) -> int:
    return lib().moe_balance_workspace_size(ctypes.byref(cfg))


def moe_balance_loss(cfg, scores, topk_idx, counts, loss, ws, seq_offsets=None, mask=None, coef=None, dscores=None,
                     stats=None, stream=None):
    """Balance loss, per-expert counts and coef * dloss/dscores (see
    include/moe.h).  topk_idx None: counts is read; scores, loss and dscores
    None: only counts."""
    import torch
    fn, dev, n = "moe_balance_loss", _current_device(), cfg.T * cfg.E
    zt, f32, i32 = _torch_dtype(cfg.dtype), torch.float32, torch.int32
    cp = _arg(fn, "counts", counts, dev, i32, cfg.S * cfg.E)
    ip = _arg(fn, "topk_idx", topk_idx, dev, i32, cfg.T * cfg.k)
    if topk_idx is not None and cfg.T == 0:
        ip = cp   # an empty tensor has no address: any other than NULL says that counts is written
    if mask is not None and not isinstance(mask, int) and mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    wp, wn = _workspace(fn, ws, dev)
    _check(fn, lib().moe_balance_loss(
        ctypes.byref(cfg), _arg(fn, "scores", scores, dev, zt, n), ip,
        _arg(fn, "seq_offsets", seq_offsets, dev, i32, cfg.S + 1), _arg(fn, "mask", mask, dev, torch.uint8, cfg.T),
        _arg(fn, "coef", coef, dev, f32, 1), cp, _arg(fn, "loss", loss, dev, f32, 1),
        _arg(fn, "dscores", dscores, dev, zt, n), _stats(fn, stats, dev), wp, wn,
        _stream(stream)))


def adamw_states(param, bits: int = 32):
    """New optimiser states of a tensor: (m, v, m_scale, v_scale), zeros; the scales are None for 32 bits."""
    import torch
    n = param.numel()
    if bits not in (8, 32):
        raise ValueError(f"states have 8 or 32 bits, not {bits}")
    if bits == 32:
        return (torch.zeros(n, device=param.device), torch.zeros(n, device=param.device), None, None)
    blocks = (n + MOE_ADAMW_BLOCK - 1) // MOE_ADAMW_BLOCK
    return tuple(torch.zeros(n, dtype=torch.float8_e4m3fn, device=param.device) for _ in range(2)) + tuple(
        torch.zeros(blocks, device=param.device) for _ in range(2))


def adamw_tensor(param, grad, m, v, m_scale=None, v_scale=None, master=None, weight_decay: float = 0.0) -> dict:
    """One tensor of an AdamW plan.  fp32 m and v: 32-bit states; float8_e4m3fn
    (or uint8) ones with their scales: 8-bit states."""
    return dict(param=param, grad=grad, m=m, v=v, m_scale=m_scale, v_scale=v_scale, master=master,
                weight_decay=weight_decay)


class AdamWPlan:
    """The tensors and constants of an optimiser, laid out once for
    moe_adamw_step.  It keeps the tensors alive; their contents (the gradients
    above all) are read at each step."""

    def __init__(self, tensors, lr: float, beta1: float, beta2: float, eps: float):
        import torch
        fn, dev = "make_adamw_plan", _current_device()
        codes = {v: k for k, v in ((c, _torch_dtype(c)) for c in (MOE_DTYPE_F32, MOE_DTYPE_BF16, MOE_DTYPE_F16))}
        self.tensors = [dict(t) for t in tensors]
        self.device = dev
        self.hyper = moe_adamw_hyper(lr, beta1, beta2, eps)
        self.table = (moe_adamw_tensor * len(self.tensors))()
        for i, t in enumerate(self.tensors):
            n = t["param"].numel()
            eight = t["m"].dtype != torch.float32
            if t["param"].dtype not in codes or t["grad"].dtype not in codes:
                raise MoeError(fn, 1, f"tensor {i}: param and grad are float32, bfloat16 or float16")
            if eight and (t["m"].dtype not in (torch.float8_e4m3fn, torch.uint8)
                          or t["m_scale"] is None or t["v_scale"] is None):
                raise MoeError(fn, 1, f"tensor {i}: 8-bit m and v are float8_e4m3fn or uint8, with scales")
            nb = (n + MOE_ADAMW_BLOCK - 1) // MOE_ADAMW_BLOCK
            e = self.table[i]
            for name, dtype, count in (("param", t["param"].dtype, n), ("grad", t["grad"].dtype, n),
                                       ("master", torch.float32, n), ("m", t["m"].dtype, n), ("v", t["m"].dtype, n),
                                       ("m_scale", torch.float32, nb), ("v_scale", torch.float32, nb)):
                setattr(e, name, _arg(fn, f"tensor {i}: {name}", t[name], dev, dtype, count))
            e.n, e.state_bits, e.weight_decay = n, 8 if eight else 32, t["weight_decay"]
            e.param_dtype, e.grad_dtype = codes[t["param"].dtype], codes[t["grad"].dtype]


def make_adamw_plan(tensors, lr: float = 1e-3, beta1: float = 0.9, beta2: float = 0.999,
                    eps: float = 1e-8) -> AdamWPlan:
    """tensors: adamw_tensor(...)s.  plan.hyper may be changed between steps."""
    return AdamWPlan(tensors, lr, beta1, beta2, eps)


def moe_adamw_step(plan: AdamWPlan, state, lr=None, grad_scale=None, stream=None):
    """One step over the plan's tensors.  state: int32[2] device tensor, zeros
    before the first step (state[0] counts the steps).  lr, grad_scale: device
    fp32 scalars or None (plan.hyper.lr, 1)."""
    import torch
    fn, dev = "moe_adamw_step", _current_device()
    if plan.device != dev:
        raise MoeError(fn, 1, f"the plan's tensors are on cuda:{plan.device}, not on the current CUDA device")
    _check(fn, lib().moe_adamw_step(plan.table, len(plan.table), ctypes.byref(plan.hyper),
                                    _arg(fn, "lr", lr, dev, torch.float32, 1),
                                    _arg(fn, "grad_scale", grad_scale, dev, torch.float32, 1),
                                    _arg(fn, "state", state, dev, torch.int32, 2), _stream(stream)))


def read_stats(stats_tensor) -> dict:
    """Copy a device moe_stats (a uint8 tensor of sizeof(moe_stats) bytes) to a dict (synchronises)."""
    raw = bytes(stats_tensor.cpu().numpy().tobytes())
    s = moe_stats.from_buffer_copy(raw[:ctypes.sizeof(moe_stats)])
    return {f: getattr(s, f) for f, _ in moe_stats._fields_}


STATS_BYTES = ctypes.sizeof(moe_stats)

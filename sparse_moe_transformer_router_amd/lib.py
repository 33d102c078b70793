"""Python binding of libmoe (include/moe.h): argument marshalling only.

Every function takes torch tensors that live on the GPU and passes their
device pointers and sizes to the C ABI; all arithmetic runs in the library's
HIP kernels.  torch supplies the memory and the stream (the current stream
unless one is given).  If libmoe.so has not been built, importing this module
raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_F32, MOE_BF16 = 0, 1
MOE_W_INT8, MOE_W_FP8, MOE_W_MXFP4, MOE_W_MXFP8 = 1, 2, 3, 4
MOE_NOALLOC_SCRATCH_BYTES = 64 << 20   # the no-allocation entry point's device array


class MoeDims(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("num_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("expert_inter", ctypes.c_int32),
                ("dense_inter", ctypes.c_int32), ("eps", ctypes.c_float),
                ("act_dtype", ctypes.c_int32), ("slot_dtype", ctypes.c_int32)]


class Gemma4FfnWeights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "g_pre", "g_pre2", "g_post1", "g_post2", "g_post", "dense_gate", "dense_up",
        "dense_down", "router_w", "router_scale", "per_expert_scale", "w_gate_up", "w_down")] + \
        [("layer_scalar", ctypes.c_float)]


class Gemma4FfnWeightsQ(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in (
        "g_pre", "g_pre2", "g_post1", "g_post2", "g_post", "dense_gate_q", "dense_gate_scale",
        "dense_up_q", "dense_up_scale", "dense_down_q", "dense_down_scale", "router_w",
        "router_scale", "per_expert_scale", "gate_up_q", "gate_up_scale", "down_q",
        "down_scale")] + [("layer_scalar", ctypes.c_float)]


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libmoe error {code}: {msg}")
        self.code = code


# Size functions of the workspaces: of the calls named, of all others ("layer").
_WS_SIZES = {"layer": "moe_workspace_size", "balance_loss": "moe_balance_loss_workspace_size",
             "router_grad": "moe_router_grad_workspace_size",
             "expert_ffn_b128": "moe_expert_ffn_b128_workspace_size"}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_moe_transformer_router_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(MoeDims)
    for f in _WS_SIZES.values():
        getattr(L, f).argtypes = [D, I32]
        getattr(L, f).restype = SZ
    L.moe_last_error.argtypes = []
    L.moe_last_error.restype = ctypes.c_char_p
    L.moe_router.argtypes = [D, I32] + [P] * 8 + [SZ, P]
    F = ctypes.c_float
    L.moe_router_logits.argtypes = [D, I32] + [P] * 9 + [SZ, P]
    L.moe_balance_loss.argtypes = [D, I32] + [P] * 3 + [F, F] + [P] * 4 + [SZ, P]
    L.moe_balance_loss_grad.argtypes = [D, I32] + [P] * 4 + [F, F] + [P] * 3
    L.moe_router_grad.argtypes = [D, I32] + [P] * 16 + [SZ, P]
    I64 = ctypes.c_int64
    L.moe_quantize_b128.argtypes = [I32, I64, I32, I32, P, P, P, P]
    L.moe_dequantize_b128.argtypes = [I32, I64, I32, I32, P, P, P, P]
    L.moe_linear_b128_workspace_size.argtypes = [I32, I32]
    L.moe_linear_b128_workspace_size.restype = SZ
    L.moe_linear_b128.argtypes = [I32, I32, I32] + [P] * 4 + [I32, P, SZ, P]
    L.moe_expert_ffn_b128.argtypes = [D, I32] + [P] * 10 + [SZ, P]
    L.moe_route.argtypes = [D, I32] + [P] * 11 + [SZ, P]
    L.moe_dispatch.argtypes = [D, I32] + [P] * 5 + [SZ, P]
    L.moe_expert_ffn.argtypes = [D, I32] + [P] * 8 + [SZ, P]
    L.moe_dense_mask_dispatch.argtypes = [D, I32] + [P] * 6
    L.moe_expert_gate_up.argtypes = [D, I32] + [P] * 6
    L.moe_expert_gate_up_timed.argtypes = [D, I32] + [P] * 8
    L.moe_expert_down.argtypes = [D, I32] + [P] * 7
    L.moe_combine.argtypes = [D, I32, P, P, P, P]
    L.moe_forward.argtypes = [D, I32] + [P] * 10 + [SZ, P]
    L.moe_forward_noalloc.argtypes = [D, I32] + [P] * 10
    L.moe_expert_ffn_mx.argtypes = [D, I32, I32] + [P] * 10 + [SZ, P]
    L.moe_quantize_int8.argtypes = [ctypes.c_int64, I32, P, P, P, P]
    L.moe_expert_ffn_int8.argtypes = [D, I32] + [P] * 10 + [SZ, P]
    L.moe_quantize.argtypes = [I32, ctypes.c_int64, I32, P, P, P, P]
    L.moe_dequantize.argtypes = [I32, ctypes.c_int64, I32, P, P, P, P]
    L.moe_expert_ffn_q.argtypes = [D, I32, I32] + [P] * 10 + [SZ, P]
    L.gemma4_ffn_block.argtypes = [D, I32, P, ctypes.POINTER(Gemma4FfnWeights)] + [P] * 5 + \
        [SZ, P]
    L.gemma4_ffn_block_q.argtypes = [D, I32, P, ctypes.POINTER(Gemma4FfnWeightsQ)] + [P] * 5 + \
        [SZ, P]
    for f in ("moe_router", "moe_route", "moe_dispatch", "moe_expert_ffn", "moe_expert_gate_up",
              "moe_expert_down", "moe_combine", "moe_forward", "gemma4_ffn_block",
              "moe_quantize_int8", "moe_expert_ffn_int8", "moe_dense_mask_dispatch",
              "moe_quantize", "moe_dequantize", "moe_expert_ffn_q", "moe_expert_gate_up_timed",
              "gemma4_ffn_block_q", "moe_forward_noalloc", "moe_expert_ffn_mx",
              "moe_router_logits", "moe_balance_loss", "moe_balance_loss_grad",
              "moe_router_grad", "moe_quantize_b128", "moe_dequantize_b128", "moe_linear_b128",
              "moe_expert_ffn_b128"):
        getattr(L, f).restype = ctypes.c_int
    return L


_lib = _load()


def raw():
    """The ctypes library object (for tests of the exported symbols)."""
    return _lib


def dims(hidden, num_experts, top_k, expert_inter, dense_inter=0, eps=1e-6, act=MOE_BF16,
         slot=MOE_F32) -> MoeDims:
    """Layer dimensions.  The per-slot expert outputs default to fp32: rounding
    them to bf16 adds a third rounding stage to the bf16 path."""
    return MoeDims(hidden, num_experts, top_k, expert_inter, dense_inter, eps, act, slot)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _device() -> int:
    """Index of the current GPU, -2 before torch has set one up (a CPU tensor's
    device is -1)."""
    return torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2


def _arg(name: str, t: Optional[torch.Tensor], dtype, numel: int, dev: int,
         optional: bool = False):
    """Device pointer of an array argument, after its type and size: a contiguous
    tensor of dtype (or of one of several) with at least numel elements, on
    device dev."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype and not (type(dtype) is tuple and t.dtype in dtype):
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, {numel} needed")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


def _work(ws: Optional[torch.Tensor], dev: int):
    """Pointer and size of a workspace (its size is the library's to check)."""
    if ws is None:
        return None, 0
    return _arg("ws", ws, torch.uint8, 0, dev), ws.numel()


_MASK = (torch.uint8, torch.bool)
_CODE = (torch.uint8, torch.float8_e4m3fn)


def _act(d: MoeDims):
    return torch.bfloat16 if d.act_dtype == MOE_BF16 else torch.float32


def _stream(stream, dev: int = -1):
    """The hipStream_t of a torch stream, the current one (of device dev, if the
    caller knows it) if none is given: asked for by its raw handle, a
    torch.cuda.Stream object costs a few microseconds, as much as a small call's
    launches."""
    if stream is not None:
        return stream.cuda_stream
    if dev < 0:
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        dev = torch._C._cuda_getDevice()
    return torch._C._cuda_getCurrentRawStream(dev)


def _check(rc: int):
    if rc != MOE_OK:
        raise MoeError(rc, _lib.moe_last_error().decode())


def last_error() -> str:
    return _lib.moe_last_error().decode()


def workspace_size(d: MoeDims, max_tokens: int, calls=tuple(_WS_SIZES)) -> int:
    """Bytes that serve the calls named (any of "layer", "balance_loss", "router_grad",
    "expert_ffn_b128", where "layer" is every call but the other three), all of
    them by default."""
    need = 0
    for c in calls:
        if c not in _WS_SIZES:
            raise ValueError(f"calls names {c!r}, expected some of {tuple(_WS_SIZES)}")
        n = getattr(_lib, _WS_SIZES[c])(ctypes.byref(d), max_tokens)
        if n == 0:
            raise MoeError(MOE_ERR_UNSUPPORTED, last_error())
        need = max(need, n)
    return need


def workspace(d: MoeDims, max_tokens: int, device="cuda", calls=tuple(_WS_SIZES)) -> torch.Tensor:
    """A uint8 device buffer of workspace_size bytes (256-byte aligned)."""
    return torch.empty(workspace_size(d, max_tokens, calls), dtype=torch.uint8, device=device)


def moe_router(d, T, x, router_w, router_scale, per_expert_scale, pre_norm_gain, topk_idx,
               topk_w, ws, stream=None):
    _check(_lib.moe_router(ctypes.byref(d), T, _ptr(x), _ptr(router_w), _ptr(router_scale),
                           _ptr(per_expert_scale), _ptr(pre_norm_gain), _ptr(topk_idx),
                           _ptr(topk_w), _ptr(ws), ws.numel() if ws is not None else 0,
                           _stream(stream)))


def moe_router_logits(d, T, x, router_w, router_scale, per_expert_scale, pre_norm_gain, topk_idx,
                      topk_w, logits, ws, stream=None):
    """moe_router, with the logits [T, E] as an output."""
    E, H, K, f32, dev = d.num_experts, d.hidden, d.top_k, torch.float32, _device()
    _check(_lib.moe_router_logits(
        ctypes.byref(d), T, _arg("x", x, _act(d), T * H, dev),
        _arg("router_w", router_w, f32, E * H, dev),
        _arg("router_scale", router_scale, f32, H, dev),
        _arg("per_expert_scale", per_expert_scale, f32, E, dev),
        _arg("pre_norm_gain", pre_norm_gain, f32, H, dev, True),
        _arg("topk_idx", topk_idx, torch.int32, T * K, dev),
        _arg("topk_w", topk_w, f32, T * K, dev),
        _arg("logits", logits, f32, T * E, dev), *_work(ws, dev), _stream(stream, dev)))


def moe_balance_loss(d, T, logits, topk_idx, token_mask, balance_coef, z_coef, loss,
                     expert_counts, mean_probs, ws, stream=None):
    """Balance loss, z-loss, per-expert counts and mean probabilities of a batch."""
    E, f32, dev = d.num_experts, torch.float32, _device()
    _check(_lib.moe_balance_loss(
        ctypes.byref(d), T, _arg("logits", logits, f32, T * E, dev),
        _arg("topk_idx", topk_idx, torch.int32, T * d.top_k, dev),
        _arg("token_mask", token_mask, _MASK, T, dev, True), balance_coef, z_coef,
        _arg("loss", loss, f32, 4, dev), _arg("expert_counts", expert_counts, torch.int32, E, dev),
        _arg("mean_probs", mean_probs, f32, E, dev), *_work(ws, dev), _stream(stream, dev)))


def moe_balance_loss_grad(d, T, logits, token_mask, expert_counts, loss, balance_coef, z_coef,
                          d_loss, d_logits, stream=None):
    """Gradient of d_loss * loss[0] in the logits."""
    E, f32, dev = d.num_experts, torch.float32, _device()
    _check(_lib.moe_balance_loss_grad(
        ctypes.byref(d), T, _arg("logits", logits, f32, T * E, dev),
        _arg("token_mask", token_mask, _MASK, T, dev, True),
        _arg("expert_counts", expert_counts, torch.int32, E, dev), _arg("loss", loss, f32, 4, dev),
        balance_coef, z_coef, _arg("d_loss", d_loss, f32, 1, dev),
        _arg("d_logits", d_logits, f32, T * E, dev), _stream(stream, dev)))


def moe_router_grad(d, T, x, router_w, router_scale, per_expert_scale, pre_norm_gain, logits,
                    topk_idx, token_mask, d_topk_w, d_logits, d_x, d_router_w, d_router_scale,
                    d_per_expert_scale, d_pre_norm_gain, ws, stream=None):
    """Backward pass of moe_router_logits."""
    E, H, K, f32, dev = d.num_experts, d.hidden, d.top_k, torch.float32, _device()
    _check(_lib.moe_router_grad(
        ctypes.byref(d), T, _arg("x", x, _act(d), T * H, dev),
        _arg("router_w", router_w, f32, E * H, dev),
        _arg("router_scale", router_scale, f32, H, dev),
        _arg("per_expert_scale", per_expert_scale, f32, E, dev, True),
        _arg("pre_norm_gain", pre_norm_gain, f32, H, dev, True),
        _arg("logits", logits, f32, T * E, dev),
        _arg("topk_idx", topk_idx, torch.int32, T * K, dev, True),
        _arg("token_mask", token_mask, _MASK, T, dev, True),
        _arg("d_topk_w", d_topk_w, f32, T * K, dev, True),
        _arg("d_logits", d_logits, f32, T * E, dev, True),
        _arg("d_x", d_x, _act(d), T * H, dev, True),
        _arg("d_router_w", d_router_w, f32, E * H, dev),
        _arg("d_router_scale", d_router_scale, f32, H, dev),
        _arg("d_per_expert_scale", d_per_expert_scale, f32, E, dev),
        _arg("d_pre_norm_gain", d_pre_norm_gain, f32, H, dev, True), *_work(ws, dev),
        _stream(stream, dev)))


def moe_route(d, T, x, router_w, router_scale, per_expert_scale, pre_norm_gain, topk_idx, topk_w,
              counts, offsets, sorted_slots, ws, stream=None):
    _check(_lib.moe_route(ctypes.byref(d), T, _ptr(x), _ptr(router_w), _ptr(router_scale),
                          _ptr(per_expert_scale), _ptr(pre_norm_gain), _ptr(topk_idx),
                          _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(sorted_slots), _ptr(ws),
                          ws.numel() if ws is not None else 0, _stream(stream)))


def moe_dispatch(d, T, topk_idx, counts, offsets, sorted_slots, ws, stream=None):
    _check(_lib.moe_dispatch(ctypes.byref(d), T, _ptr(topk_idx), _ptr(counts), _ptr(offsets),
                             _ptr(sorted_slots), _ptr(ws), ws.numel() if ws is not None else 0,
                             _stream(stream)))


def moe_dense_mask_dispatch(d, T, topk_idx, topk_w, offsets, sorted_slots, w_dense, stream=None):
    _check(_lib.moe_dense_mask_dispatch(ctypes.byref(d), T, _ptr(topk_idx), _ptr(topk_w),
                                        _ptr(offsets), _ptr(sorted_slots), _ptr(w_dense),
                                        _stream(stream)))


def moe_expert_ffn(d, T, x, w_gate_up, w_down, topk_w, offsets, sorted_slots, y_slots, ws,
                   stream=None):
    _check(_lib.moe_expert_ffn(ctypes.byref(d), T, _ptr(x), _ptr(w_gate_up), _ptr(w_down),
                               _ptr(topk_w), _ptr(offsets), _ptr(sorted_slots), _ptr(y_slots),
                               _ptr(ws), ws.numel() if ws is not None else 0, _stream(stream)))


def moe_quantize_int8(w, q, scale, stream=None):
    """Per-row symmetric int8 codes and scales of a bf16 weight whose last axis
    is the row (input) dimension."""
    cols = w.shape[-1]
    rows = w.numel() // cols if cols else 0
    _check(_lib.moe_quantize_int8(rows, cols, _ptr(w), _ptr(q), _ptr(scale), _stream(stream)))


def moe_expert_ffn_int8(d, T, x, w_gate_up_q, w_gate_up_scale, w_down_q, w_down_scale, topk_w,
                        offsets, sorted_slots, y_slots, ws, stream=None):
    _check(_lib.moe_expert_ffn_int8(ctypes.byref(d), T, _ptr(x), _ptr(w_gate_up_q),
                                    _ptr(w_gate_up_scale), _ptr(w_down_q), _ptr(w_down_scale),
                                    _ptr(topk_w), _ptr(offsets), _ptr(sorted_slots),
                                    _ptr(y_slots), _ptr(ws), ws.numel() if ws is not None else 0,
                                    _stream(stream)))


def moe_quantize(fmt, w, q, scale, stream=None):
    """Codes and scales of a bf16 weight whose last axis is the row (input)
    dimension, in format fmt (MOE_W_INT8, MOE_W_FP8 or MOE_W_MXFP4)."""
    cols = w.shape[-1]
    rows = w.numel() // cols if cols else 0
    _check(_lib.moe_quantize(fmt, rows, cols, _ptr(w), _ptr(q), _ptr(scale), _stream(stream)))


def moe_dequantize(fmt, rows, cols, q, scale, out, stream=None):
    _check(_lib.moe_dequantize(fmt, rows, cols, _ptr(q), _ptr(scale), _ptr(out),
                               _stream(stream)))


def moe_expert_ffn_q(d, fmt, T, x, w_gate_up_q, w_gate_up_scale, w_down_q, w_down_scale, topk_w,
                     offsets, sorted_slots, y_slots, ws, stream=None):
    _check(_lib.moe_expert_ffn_q(ctypes.byref(d), fmt, T, _ptr(x), _ptr(w_gate_up_q),
                                 _ptr(w_gate_up_scale), _ptr(w_down_q), _ptr(w_down_scale),
                                 _ptr(topk_w), _ptr(offsets), _ptr(sorted_slots),
                                 _ptr(y_slots), _ptr(ws), ws.numel() if ws is not None else 0,
                                 _stream(stream)))


def moe_expert_ffn_mx(d, fmt, T, x, w_gate_up_q, w_gate_up_scale, w_down_q, w_down_scale,
                      topk_w, offsets, sorted_slots, y_slots, ws, stream=None):
    """E4M3 / MXFP4 experts on the 8-bit / 4-bit matrix instructions, MXFP8
    activations."""
    _check(_lib.moe_expert_ffn_mx(ctypes.byref(d), fmt, T, _ptr(x), _ptr(w_gate_up_q),
                                  _ptr(w_gate_up_scale), _ptr(w_down_q), _ptr(w_down_scale),
                                  _ptr(topk_w), _ptr(offsets), _ptr(sorted_slots),
                                  _ptr(y_slots), _ptr(ws), ws.numel() if ws is not None else 0,
                                  _stream(stream)))


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _b128_shape(block_rows, t, name):
    if t.dim() < 2:
        raise ValueError(f"{name} needs two axes or more")
    rows, cols = t.shape[-2:]
    batch = t.numel() // (rows * cols) if rows and cols else 0
    nscale = batch * (rows if block_rows == 1 else _blocks(rows)) * _blocks(cols)
    return batch, rows, cols, nscale


def moe_quantize_b128(block_rows, w, q, scale, stream=None):
    """E4M3 codes (uint8 or float8_e4m3fn) and fp32 scales of a bf16 [..., rows,
    cols]: per 128 x 128 block (block_rows = 128, weights) or per 128 values of a
    row (block_rows = 1, activations)."""
    batch, rows, cols, ns = _b128_shape(block_rows, w, "w")
    dev = _device()
    _check(_lib.moe_quantize_b128(block_rows, batch, rows, cols,
                                  _arg("w", w, torch.bfloat16, w.numel(), dev),
                                  _arg("q", q, _CODE, w.numel(), dev),
                                  _arg("scale", scale, torch.float32, ns, dev),
                                  _stream(stream, dev)))


def moe_dequantize_b128(block_rows, q, scale, out, stream=None):
    batch, rows, cols, ns = _b128_shape(block_rows, q, "q")
    dev = _device()
    _check(_lib.moe_dequantize_b128(block_rows, batch, rows, cols,
                                    _arg("q", q, _CODE, q.numel(), dev),
                                    _arg("scale", scale, torch.float32, ns, dev),
                                    _arg("out", out, torch.float32, q.numel(), dev),
                                    _stream(stream, dev)))


def linear_b128_workspace(max_tokens: int, in_features: int, device="cuda") -> torch.Tensor:
    """A uint8 device buffer of moe_linear_b128_workspace_size bytes."""
    n = _lib.moe_linear_b128_workspace_size(max_tokens, in_features)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, last_error())
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_linear_b128(T, x, w_q, w_scale, y, ws, stream=None):
    """y [T, out] (fp32 or bf16) = x [T, in] (bf16) times the block-scaled weights
    w_q [out, in]; x is quantized inside."""
    if w_q.dim() != 2:
        raise ValueError("w_q needs two axes")
    (n, k), dev = w_q.shape, _device()
    _check(_lib.moe_linear_b128(
        T, n, k, _arg("x", x, torch.bfloat16, T * k, dev), _arg("w_q", w_q, _CODE, n * k, dev),
        _arg("w_scale", w_scale, torch.float32, _blocks(n) * _blocks(k), dev),
        _arg("y", y, (torch.bfloat16, torch.float32), T * n, dev),
        MOE_BF16 if y.dtype == torch.bfloat16 else MOE_F32, *_work(ws, dev), _stream(stream, dev)))


def moe_expert_ffn_b128(d, T, x, w_gate_up_q, w_gate_up_scale, w_down_q, w_down_scale, topk_w,
                        offsets, sorted_slots, y_slots, ws, stream=None):
    """The experts with E4M3 weights scaled per 128 x 128 block, activations per
    128 values."""
    H, E, I, S = d.hidden, d.num_experts, d.expert_inter, T * d.top_k
    f32, i32, dev = torch.float32, torch.int32, _device()
    _check(_lib.moe_expert_ffn_b128(
        ctypes.byref(d), T, _arg("x", x, torch.bfloat16, T * H, dev),
        _arg("w_gate_up_q", w_gate_up_q, _CODE, E * 2 * I * H, dev),
        _arg("w_gate_up_scale", w_gate_up_scale, f32, E * _blocks(2 * I) * _blocks(H), dev),
        _arg("w_down_q", w_down_q, _CODE, E * H * I, dev),
        _arg("w_down_scale", w_down_scale, f32, E * _blocks(H) * _blocks(I), dev),
        _arg("topk_w", topk_w, f32, S, dev), _arg("offsets", offsets, i32, E + 1, dev),
        _arg("sorted_slots", sorted_slots, i32, S, dev),
        _arg("y_slots", y_slots, torch.bfloat16 if d.slot_dtype == MOE_BF16 else f32, S * H, dev),
        *_work(ws, dev), _stream(stream, dev)))


def moe_expert_gate_up(d, T, x, w_gate_up, offsets, sorted_slots, h, stream=None):
    _check(_lib.moe_expert_gate_up(ctypes.byref(d), T, _ptr(x), _ptr(w_gate_up), _ptr(offsets),
                                   _ptr(sorted_slots), _ptr(h), _stream(stream)))


def moe_expert_gate_up_timed(d, T, x, w_gate_up, offsets, sorted_slots, h, start, stop,
                             stream=None):
    """moe_expert_gate_up recording torch.cuda.Event start / stop on the
    kernel's own dispatch; both events must have been recorded once before
    (torch creates its events at their first record)."""
    hs, he = start.cuda_event, stop.cuda_event
    if not hs or not he:
        raise RuntimeError("moe_expert_gate_up_timed: record both events once before use")
    _check(_lib.moe_expert_gate_up_timed(ctypes.byref(d), T, _ptr(x), _ptr(w_gate_up),
                                         _ptr(offsets), _ptr(sorted_slots), _ptr(h),
                                         _stream(stream), ctypes.c_void_p(hs),
                                         ctypes.c_void_p(he)))


def moe_expert_down(d, T, h, w_down, topk_w, offsets, sorted_slots, y_slots, stream=None):
    _check(_lib.moe_expert_down(ctypes.byref(d), T, _ptr(h), _ptr(w_down), _ptr(topk_w),
                                _ptr(offsets), _ptr(sorted_slots), _ptr(y_slots),
                                _stream(stream)))


def moe_combine(d, T, y_slots, addend, out, stream=None):
    _check(_lib.moe_combine(ctypes.byref(d), T, _ptr(y_slots), _ptr(addend), _ptr(out),
                            _stream(stream)))


def moe_forward(d, T, x, router_w, router_scale, per_expert_scale, w_gate_up, w_down, out,
                topk_idx, topk_w, ws, stream=None):
    _check(_lib.moe_forward(ctypes.byref(d), T, _ptr(x), _ptr(router_w), _ptr(router_scale),
                            _ptr(per_expert_scale), _ptr(w_gate_up), _ptr(w_down), _ptr(out),
                            _ptr(topk_idx), _ptr(topk_w), _ptr(ws),
                            ws.numel() if ws is not None else 0, _stream(stream)))


def moe_forward_noalloc(d, T, x, router_w, router_scale, per_expert_scale, w_gate_up, w_down,
                        out, topk_idx, topk_w, stream=None):
    """moe_forward with the library's own device scratch array as workspace."""
    _check(_lib.moe_forward_noalloc(ctypes.byref(d), T, _ptr(x), _ptr(router_w),
                                    _ptr(router_scale), _ptr(per_expert_scale), _ptr(w_gate_up),
                                    _ptr(w_down), _ptr(out), _ptr(topk_idx), _ptr(topk_w),
                                    _stream(stream)))


def ffn_weights(g_pre, g_pre2, g_post1, g_post2, g_post, dense_gate, dense_up, dense_down,
                router_w, router_scale, per_expert_scale, w_gate_up, w_down,
                layer_scalar) -> Gemma4FfnWeights:
    ts = (g_pre, g_pre2, g_post1, g_post2, g_post, dense_gate, dense_up, dense_down, router_w,
          router_scale, per_expert_scale, w_gate_up, w_down)
    return Gemma4FfnWeights(*[_ptr(t) for t in ts], float(layer_scalar))


def ffn_weights_q(fmt, g_pre, g_pre2, g_post1, g_post2, g_post, dense_gate_q, dense_gate_scale,
                  dense_up_q, dense_up_scale, dense_down_q, dense_down_scale, router_w,
                  router_scale, per_expert_scale, gate_up_q, gate_up_scale, down_q, down_scale,
                  layer_scalar) -> Gemma4FfnWeightsQ:
    ts = (g_pre, g_pre2, g_post1, g_post2, g_post, dense_gate_q, dense_gate_scale, dense_up_q,
          dense_up_scale, dense_down_q, dense_down_scale, router_w, router_scale,
          per_expert_scale, gate_up_q, gate_up_scale, down_q, down_scale)
    return Gemma4FfnWeightsQ(int(fmt), *[_ptr(t) for t in ts], float(layer_scalar))


def gemma4_ffn_block_q(d, T, residual, weights: Gemma4FfnWeightsQ, out, ffn_out, topk_idx,
                       topk_w, ws, stream=None):
    _check(_lib.gemma4_ffn_block_q(ctypes.byref(d), T, _ptr(residual), ctypes.byref(weights),
                                   _ptr(out), _ptr(ffn_out), _ptr(topk_idx), _ptr(topk_w),
                                   _ptr(ws), ws.numel() if ws is not None else 0,
                                   _stream(stream)))


def gemma4_ffn_block(d, T, residual, weights: Gemma4FfnWeights, out, ffn_out, topk_idx, topk_w,
                     ws, stream=None):
    _check(_lib.gemma4_ffn_block(ctypes.byref(d), T, _ptr(residual), ctypes.byref(weights),
                                 _ptr(out), _ptr(ffn_out), _ptr(topk_idx), _ptr(topk_w),
                                 _ptr(ws), ws.numel() if ws is not None else 0,
                                 _stream(stream)))

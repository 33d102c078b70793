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
import weakref
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


class MoeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libmoe error {code}: {msg}")
        self.code = code


# Size functions of the workspaces: of the calls named, of all others that have none of
# their own ("layer").  A default workspace serves the first four.
_WS_SIZES = {"layer": "moe_workspace_size", "balance_loss": "moe_balance_loss_workspace_size",
             "router_grad": "moe_router_grad_workspace_size",
             "expert_ffn_b128": "moe_expert_ffn_b128_workspace_size"}
_WS_SIZES_ALL = {**_WS_SIZES, "expert_ffn_grad": "moe_expert_ffn_grad_workspace_size",
                 "dense_mlp_grad": "gemma4_dense_mlp_grad_workspace_size",
                 "norms_grad": "gemma4_norms_grad_workspace_size"}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m sparse_moe_transformer_router_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(MoeDims)
    for f in _WS_SIZES_ALL.values():
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
    TN = ctypes.POINTER(MoeTensor)
    L.moe_grad_norm_workspace_size.argtypes = [I32, TN]
    L.moe_grad_norm_workspace_size.restype = SZ
    L.moe_expert_ffn_keep.argtypes = [D, I32] + [P] * 9 + [SZ, P]
    L.moe_expert_ffn_grad.argtypes = [D, I32] + [P] * 11 + [I32] + [P] * 3 + [SZ, P]
    L.gemma4_dense_mlp.argtypes = [D, I32] + [P] * 7 + [SZ, P]
    L.gemma4_dense_mlp_grad.argtypes = [D, I32] + [P] * 8 + [I32] + [P] * 4 + [SZ, P]
    L.gemma4_pre_norms.argtypes = [D, I32] + [P] * 6
    L.gemma4_post_norms.argtypes = [D, I32] + [P] * 6 + [F] + [P] * 4
    L.gemma4_pre_norms_grad.argtypes = [D, I32] + [P] * 8 + [F] + [P] * 4 + [SZ, P]
    L.gemma4_post_norms_grad.argtypes = [D, I32] + [P] * 6 + [F] + [P] * 9 + [SZ, P]
    L.moe_grad_norm.argtypes = [I32, TN, F, P, P, SZ, P]
    L.moe_grad_clip.argtypes = [I32, TN, P, TN, P]
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
              "moe_expert_ffn_b128", "moe_expert_ffn_keep", "moe_expert_ffn_grad",
              "gemma4_dense_mlp", "gemma4_dense_mlp_grad", "gemma4_pre_norms",
              "gemma4_post_norms", "gemma4_pre_norms_grad", "gemma4_post_norms_grad",
              "moe_grad_norm", "moe_grad_clip"):
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
    """Bytes that serve the calls named: any of "layer", "balance_loss", "router_grad",
    "expert_ffn_b128" (all four by default), "expert_ffn_grad", "dense_mlp_grad" and
    "norms_grad", where "layer" is every call that has no size function of its own."""
    need = 0
    for c in calls:
        if c not in _WS_SIZES_ALL:
            raise ValueError(f"calls names {c!r}, expected some of {tuple(_WS_SIZES_ALL)}")
        n = getattr(_lib, _WS_SIZES_ALL[c])(ctypes.byref(d), max_tokens)
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


def _slot(d: MoeDims):
    return torch.bfloat16 if d.slot_dtype == MOE_BF16 else torch.float32


_FLOAT = (torch.bfloat16, torch.float32)


def _dtype(*tensors):
    """moe_dtype code that the tensors given share (MOE_F32 where none is)."""
    kinds = {t.dtype for t in tensors if t is not None}
    if len(kinds) > 1:
        raise TypeError(f"weight gradients of several types: {sorted(map(str, kinds))}")
    return MOE_BF16 if kinds == {torch.bfloat16} else MOE_F32


def expert_ffn_grad_workspace(d: MoeDims, max_tokens: int, device="cuda") -> torch.Tensor:
    """A uint8 device buffer of moe_expert_ffn_grad_workspace_size bytes."""
    return workspace(d, max_tokens, device, ("expert_ffn_grad",))


def dense_mlp_grad_workspace(d: MoeDims, max_tokens: int, device="cuda") -> torch.Tensor:
    """A uint8 device buffer of gemma4_dense_mlp_grad_workspace_size bytes."""
    return workspace(d, max_tokens, device, ("dense_mlp_grad",))


def norms_grad_workspace(d: MoeDims, max_tokens: int, device="cuda") -> torch.Tensor:
    """A uint8 device buffer of gemma4_norms_grad_workspace_size bytes."""
    return workspace(d, max_tokens, device, ("norms_grad",))


def moe_expert_ffn_keep(d, T, x, w_gate_up, w_down, topk_w, offsets, sorted_slots, gate_up,
                        y_slots, ws, stream=None):
    """moe_expert_ffn, with the projections gate_up [T * K, 2I] as an output."""
    H, E, I, S, a = d.hidden, d.num_experts, d.expert_inter, T * d.top_k, _act(d)
    f32, i32, dev = torch.float32, torch.int32, _device()
    _check(_lib.moe_expert_ffn_keep(
        ctypes.byref(d), T, _arg("x", x, a, T * H, dev),
        _arg("w_gate_up", w_gate_up, a, E * 2 * I * H, dev),
        _arg("w_down", w_down, a, E * H * I, dev), _arg("topk_w", topk_w, f32, S, dev),
        _arg("offsets", offsets, i32, E + 1, dev),
        _arg("sorted_slots", sorted_slots, i32, S, dev),
        _arg("gate_up", gate_up, a, S * 2 * I, dev),
        _arg("y_slots", y_slots, _slot(d), S * H, dev), *_work(ws, dev), _stream(stream, dev)))


def moe_expert_ffn_grad(d, T, x, w_gate_up, w_down, topk_w, offsets, sorted_slots, gate_up,
                        token_mask, d_out, d_x, d_topk_w, d_w_gate_up, d_w_down, ws,
                        stream=None):
    """Backward pass of moe_expert_ffn_keep and the slots' sum.  The weights' gradients
    are both fp32 or both of the activations' type."""
    H, E, I, S, a = d.hidden, d.num_experts, d.expert_inter, T * d.top_k, _act(d)
    f32, i32, dev = torch.float32, torch.int32, _device()
    _check(_lib.moe_expert_ffn_grad(
        ctypes.byref(d), T, _arg("x", x, a, T * H, dev),
        _arg("w_gate_up", w_gate_up, a, E * 2 * I * H, dev),
        _arg("w_down", w_down, a, E * H * I, dev), _arg("topk_w", topk_w, f32, S, dev),
        _arg("offsets", offsets, i32, E + 1, dev),
        _arg("sorted_slots", sorted_slots, i32, S, dev),
        _arg("gate_up", gate_up, a, S * 2 * I, dev),
        _arg("token_mask", token_mask, _MASK, T, dev, True), _arg("d_out", d_out, a, T * H, dev),
        _arg("d_x", d_x, a, T * H, dev, True), _arg("d_topk_w", d_topk_w, f32, S, dev, True),
        _dtype(d_w_gate_up, d_w_down),
        _arg("d_w_gate_up", d_w_gate_up, _FLOAT, E * 2 * I * H, dev, True),
        _arg("d_w_down", d_w_down, _FLOAT, E * H * I, dev, True), *_work(ws, dev),
        _stream(stream, dev)))


def gemma4_dense_mlp(d, T, x, dense_gate, dense_up, dense_down, gate_up, y, ws, stream=None):
    """The dense MLP; gate_up [T, 2D] or None receives its projections."""
    H, D, a, dev = d.hidden, d.dense_inter, _act(d), _device()
    _check(_lib.gemma4_dense_mlp(
        ctypes.byref(d), T, _arg("x", x, a, T * H, dev),
        _arg("dense_gate", dense_gate, a, D * H, dev), _arg("dense_up", dense_up, a, D * H, dev),
        _arg("dense_down", dense_down, a, H * D, dev),
        _arg("gate_up", gate_up, a, T * 2 * D, dev, True), _arg("y", y, _slot(d), T * H, dev),
        *_work(ws, dev), _stream(stream, dev)))


def gemma4_dense_mlp_grad(d, T, x, dense_gate, dense_up, dense_down, gate_up, token_mask, d_y,
                          d_x, d_gate, d_up, d_down, ws, stream=None):
    """Backward pass of gemma4_dense_mlp.  The weights' gradients are all fp32 or all of
    the activations' type."""
    H, D, a, dev = d.hidden, d.dense_inter, _act(d), _device()
    _check(_lib.gemma4_dense_mlp_grad(
        ctypes.byref(d), T, _arg("x", x, a, T * H, dev),
        _arg("dense_gate", dense_gate, a, D * H, dev), _arg("dense_up", dense_up, a, D * H, dev),
        _arg("dense_down", dense_down, a, H * D, dev), _arg("gate_up", gate_up, a, T * 2 * D, dev),
        _arg("token_mask", token_mask, _MASK, T, dev, True), _arg("d_y", d_y, a, T * H, dev),
        _arg("d_x", d_x, a, T * H, dev, True), _dtype(d_gate, d_up, d_down),
        _arg("d_gate", d_gate, _FLOAT, D * H, dev, True),
        _arg("d_up", d_up, _FLOAT, D * H, dev, True),
        _arg("d_down", d_down, _FLOAT, H * D, dev, True), *_work(ws, dev), _stream(stream, dev)))


def gemma4_pre_norms(d, T, x, g_pre, g_pre2, xd, xm, stream=None):
    """xd, xm: the two pre-norms of x."""
    n, H, a, f32, dev = T * d.hidden, d.hidden, _act(d), torch.float32, _device()
    _check(_lib.gemma4_pre_norms(
        ctypes.byref(d), T, _arg("x", x, a, n, dev), _arg("g_pre", g_pre, f32, H, dev),
        _arg("g_pre2", g_pre2, f32, H, dev), _arg("xd", xd, a, n, dev),
        _arg("xm", xm, a, n, dev), _stream(stream, dev)))


def gemma4_post_norms(d, T, x, y_slots, dn, g_post1, g_post2, g_post, layer_scalar, out, moe_sum,
                      ffn_out, stream=None):
    """The layer's end: the slots' sum (to moe_sum unless None), the post-norms, the
    residual and layer_scalar."""
    n, H, a, f32, dev = T * d.hidden, d.hidden, _act(d), torch.float32, _device()
    _check(_lib.gemma4_post_norms(
        ctypes.byref(d), T, _arg("x", x, a, n, dev),
        _arg("y_slots", y_slots, _slot(d), n * d.top_k, dev), _arg("dn", dn, _slot(d), n, dev),
        _arg("g_post1", g_post1, f32, H, dev), _arg("g_post2", g_post2, f32, H, dev),
        _arg("g_post", g_post, f32, H, dev), layer_scalar, _arg("out", out, a, n, dev),
        _arg("moe_sum", moe_sum, _slot(d), n, dev, True),
        _arg("ffn_out", ffn_out, f32, n, dev, True), _stream(stream, dev)))


def gemma4_pre_norms_grad(d, T, x, g_pre, g_pre2, token_mask, d_xd, d_xm, d_x_add, d_out,
                          layer_scalar, d_x, d_g_pre, d_g_pre2, ws, stream=None):
    """Backward pass of gemma4_pre_norms, plus d_x_add and layer_scalar * d_out.  The
    gradient of g_pre2 is d_g_pre2 plus moe_router_grad's d_pre_norm_gain: both calls
    overwrite, the sum is the caller's."""
    n, H, a, f32, dev = T * d.hidden, d.hidden, _act(d), torch.float32, _device()
    _check(_lib.gemma4_pre_norms_grad(
        ctypes.byref(d), T, _arg("x", x, a, n, dev), _arg("g_pre", g_pre, f32, H, dev),
        _arg("g_pre2", g_pre2, f32, H, dev), _arg("token_mask", token_mask, _MASK, T, dev, True),
        _arg("d_xd", d_xd, a, n, dev), _arg("d_xm", d_xm, a, n, dev),
        _arg("d_x_add", d_x_add, a, n, dev, True), _arg("d_out", d_out, a, n, dev, True),
        layer_scalar, _arg("d_x", d_x, a, n, dev), _arg("d_g_pre", d_g_pre, f32, H, dev),
        _arg("d_g_pre2", d_g_pre2, f32, H, dev), *_work(ws, dev), _stream(stream, dev)))


def gemma4_post_norms_grad(d, T, x, dn, moe_sum, g_post1, g_post2, g_post, layer_scalar,
                           token_mask, d_out, d_dn, d_moe, d_g_post1, d_g_post2, d_g_post,
                           d_layer_scalar, ws, stream=None):
    """Backward pass of gemma4_post_norms; x and d_layer_scalar may both be None."""
    n, H, a, f32, dev = T * d.hidden, d.hidden, _act(d), torch.float32, _device()
    _check(_lib.gemma4_post_norms_grad(
        ctypes.byref(d), T, _arg("x", x, a, n, dev, True), _arg("dn", dn, _slot(d), n, dev),
        _arg("moe_sum", moe_sum, _slot(d), n, dev), _arg("g_post1", g_post1, f32, H, dev),
        _arg("g_post2", g_post2, f32, H, dev), _arg("g_post", g_post, f32, H, dev), layer_scalar,
        _arg("token_mask", token_mask, _MASK, T, dev, True), _arg("d_out", d_out, a, n, dev),
        _arg("d_dn", d_dn, a, n, dev), _arg("d_moe", d_moe, a, n, dev),
        _arg("d_g_post1", d_g_post1, f32, H, dev), _arg("d_g_post2", d_g_post2, f32, H, dev),
        _arg("d_g_post", d_g_post, f32, H, dev),
        _arg("d_layer_scalar", d_layer_scalar, f32, 1, dev, True), *_work(ws, dev),
        _stream(stream, dev)))


class GradList:
    """A list of gradients for moe_grad_norm and moe_grad_clip: made once, used as long
    as the tensors keep their memory (it holds them)."""

    def __init__(self, tensors):
        self.tensors = list(tensors)
        self.device = _device()
        spans = []
        for i, t in enumerate(self.tensors):
            _arg(f"tensor {i}", t, _FLOAT, 0, self.device)
            if t.numel():
                spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), i))
        spans.sort()
        for (_, end, i), (start, _, j) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError(f"tensors {i} and {j} overlap")
        self.spans = spans
        self.fits = None  # the list whose gradients it was found to be outputs of
        self.n = len(self.tensors)
        self.array = (MoeTensor * self.n)(*[
            (t.data_ptr(), t.numel(), MOE_BF16 if t.dtype == torch.bfloat16 else MOE_F32)
            for t in self.tensors])

    def _on(self, dev):
        if self.device != dev:
            raise ValueError("the list's tensors are not on the current GPU")
        return self.array


def grad_list(tensors) -> GradList:
    """The gradients (contiguous, fp32 or bf16, of any sizes, none overlapping another)
    that moe_grad_norm and moe_grad_clip take.  One that overlaps another, or is listed
    twice, is refused here, also in a list that is only measured, where the library's
    own call would count it twice."""
    return GradList(tensors)


def grad_norm_workspace(grads: GradList, device="cuda") -> torch.Tensor:
    """A uint8 device buffer of moe_grad_norm_workspace_size bytes."""
    n = _lib.moe_grad_norm_workspace_size(grads.n, grads.array)
    if n == 0:
        raise MoeError(MOE_ERR_UNSUPPORTED, last_error())
    return torch.empty(n, dtype=torch.uint8, device=device)


def moe_grad_norm(grads: GradList, max_norm, norm, ws, stream=None):
    """norm [2] = {global norm, factor that brings it to max_norm at most}."""
    dev = _device()
    _check(_lib.moe_grad_norm(grads.n, grads._on(dev), max_norm,
                              _arg("norm", norm, torch.float32, 2, dev), *_work(ws, dev),
                              _stream(stream, dev)))


def _check_out(grads: GradList, out: GradList):
    """out's tensors are their gradients or overlap none of them."""
    if out.n != grads.n:
        raise ValueError(f"out has {out.n} tensors, grads {grads.n}")
    a, b = grads.spans, out.spans
    if not a or not b or a[-1][1] <= b[0][0] or b[-1][1] <= a[0][0]:
        return
    i = j = 0
    while i < len(a) and j < len(b):  # both ascending, neither overlapping itself
        if a[i][0] < b[j][1] and b[j][0] < a[i][1] and not (
                a[i] == b[j] and grads.tensors[a[i][2]].dtype == out.tensors[b[j][2]].dtype):
            raise ValueError(f"out tensor {b[j][2]} overlaps gradient {a[i][2]}")
        if a[i][1] <= b[j][1]:
            i += 1
        else:
            j += 1


def moe_grad_clip(grads: GradList, norm, out: Optional[GradList] = None, stream=None):
    """out (None: grads themselves) = grads * norm[1]."""
    dev = _device()
    if out is not None and out is not grads and (out.fits is None or out.fits() is not grads):
        _check_out(grads, out)
        out.fits = weakref.ref(grads)
    _check(_lib.moe_grad_clip(grads.n, grads._on(dev),
                              _arg("norm", norm, torch.float32, 2, dev),
                              None if out is None else out._on(dev), _stream(stream, dev)))


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

"""Refusals of the layer's training calls: on the host, before any HIP call (CPU)."""
import ctypes

import pytest

lib = pytest.importorskip("sparse_moe_transformer_router_amd.lib", reason="libmoe.so not built")
L = lib.raw()
P, BAD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
BIG = 1 << 50


def D(**kw):
    base = dict(hidden=2816, num_experts=128, top_k=8, expert_inter=704, dense_inter=2112,
                eps=1e-6, act=lib.MOE_BF16)
    base.update(kw)
    return ctypes.byref(lib.dims(**base))


# name -> (arguments after dims and T, without the stream; indexes of required pointers;
# of optional ones; index of ws)
F32, BF16 = lib.MOE_F32, lib.MOE_BF16
CALLS = {
    "moe_expert_ffn_keep": ([P] * 9 + [BIG], range(0, 8), (), 8),
    "moe_expert_ffn_grad": ([P] * 11 + [BF16, P, P, P, BIG], (0, 1, 2, 3, 4, 5, 6, 8),
                            (7, 9, 10, 12, 13), 14),
    "gemma4_dense_mlp": ([P] * 7 + [BIG], (0, 1, 2, 3, 5), (4,), 6),
    "gemma4_dense_mlp_grad": ([P] * 8 + [BF16, P, P, P, P, BIG], (0, 1, 2, 3, 4, 6),
                              (5, 7, 11), 12),
    "gemma4_pre_norms": ([P] * 5, range(0, 5), (), None),
    "gemma4_post_norms": ([P] * 6 + [0.5, P, P, P], (0, 1, 2, 3, 4, 5, 7), (8, 9), None),
    "gemma4_pre_norms_grad": ([P] * 8 + [0.5, P, P, P, P, BIG], (0, 1, 2, 4, 5, 9, 10, 11),
                              (3, 6, 7), 12),
    "gemma4_post_norms_grad": ([P] * 6 + [0.5] + [P] * 9 + [BIG],
                               (0, 1, 2, 3, 4, 5, 8, 9, 10, 11, 12, 13), (7, 14), 15),
}


def call(name, args, d=None, T=4):
    return getattr(L, name)(d or D(), T, *args, None)


@pytest.mark.parametrize("name", CALLS)
def test_pointers(name):
    args, need, may, ws = CALLS[name]
    for i in need:
        for v in (None, BAD):
            a = list(args)
            a[i] = v
            assert call(name, a) == lib.MOE_ERR_ARG, (name, i, v)
            assert lib.last_error()
    for i in may:
        a = list(args)
        a[i] = BAD
        assert call(name, a) == lib.MOE_ERR_ARG, (name, i)
    if ws is not None:
        for v in (None, ctypes.c_void_p(0x10010)):
            a = list(args)
            a[ws] = v
            assert call(name, a) == lib.MOE_ERR_WORKSPACE, (name, v)
        a = list(args)
        a[ws + 1] = 100
        assert call(name, a) == lib.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("name", CALLS)
def test_dims_and_tokens(name):
    args = CALLS[name][0]
    assert call(name, args, T=-1) == lib.MOE_ERR_ARG
    assert call(name, args, T=65537) == lib.MOE_ERR_ARG
    for kw in (dict(hidden=100), dict(num_experts=300), dict(expert_inter=48),
               dict(dense_inter=16400)):
        assert call(name, args, D(**kw)) == lib.MOE_ERR_UNSUPPORTED, (name, kw)
    assert call(name, args, D(eps=0.0)) == lib.MOE_ERR_ARG
    if "dense" in name:
        assert call(name, args, D(dense_inter=0)) == lib.MOE_ERR_UNSUPPORTED


def test_slots_past_the_limit():
    args = CALLS["moe_expert_ffn_grad"][0]
    assert call("moe_expert_ffn_grad", args, D(top_k=128), T=8193) == lib.MOE_ERR_UNSUPPORTED


def test_weight_gradient_types():
    for name, at in (("moe_expert_ffn_grad", 11), ("gemma4_dense_mlp_grad", 8)):
        a = list(CALLS[name][0])
        a[at] = 7
        assert call(name, a) == lib.MOE_ERR_ARG
        a[at] = BF16
        assert call(name, a, D(act=F32)) == lib.MOE_ERR_UNSUPPORTED


def test_outputs_asked_for():
    a = list(CALLS["moe_expert_ffn_grad"][0])
    for i in (9, 10, 12, 13):
        a[i] = None
    assert call("moe_expert_ffn_grad", a) == lib.MOE_ERR_ARG and "NULL" in lib.last_error()
    a = list(CALLS["gemma4_dense_mlp_grad"][0])
    a[9] = None
    assert call("gemma4_dense_mlp_grad", a) == lib.MOE_ERR_ARG and "together" in lib.last_error()
    for i in (7, 9, 10, 11):
        a[i] = None
    assert call("gemma4_dense_mlp_grad", a) == lib.MOE_ERR_ARG


def test_forward_calls_take_no_tokens():
    for name in ("moe_expert_ffn_keep", "gemma4_dense_mlp", "gemma4_pre_norms",
                 "gemma4_post_norms"):
        a = [None if v is P else 0 if v == BIG else v for v in CALLS[name][0]]
        assert call(name, a, T=0) == lib.MOE_OK, name


def test_workspace_sizes():
    for f in ("moe_expert_ffn_grad_workspace_size", "gemma4_dense_mlp_grad_workspace_size",
              "gemma4_norms_grad_workspace_size"):
        f = getattr(L, f)
        sizes = [f(D(), t) for t in (0, 1, 7, 64, 513, 4096, 65536)]
        assert all(s > 0 for s in sizes) and sizes == sorted(sizes)
        assert f(D(hidden=100), 4) == 0 and f(D(), -1) == 0
    assert L.gemma4_dense_mlp_grad_workspace_size(D(dense_inter=0), 4) == 0


def tensors(*t):
    return (lib.MoeTensor * len(t))(*t)


def test_grad_lists():
    ok = tensors((0x10000, 10, F32), (0x20002, 5, BF16), (None, 0, F32))
    assert L.moe_grad_norm_workspace_size(3, ok) > 0
    assert L.moe_grad_norm(3, ok, 1.0, P, None, 0, None) == lib.MOE_ERR_WORKSPACE
    assert L.moe_grad_norm(3, ok, 1.0, P, P, 8, None) == lib.MOE_ERR_WORKSPACE
    assert L.moe_grad_norm(3, ok, 1.0, None, P, BIG, None) == lib.MOE_ERR_ARG
    for limit in (0.0, -1.0, float("nan")):
        assert L.moe_grad_norm(3, ok, limit, P, P, BIG, None) == lib.MOE_ERR_ARG
    assert L.moe_grad_clip(3, ok, None, None, None) == lib.MOE_ERR_ARG
    assert L.moe_grad_clip(0, None, None, None, None) == lib.MOE_OK
    for n, bad, code in ((-1, ok, lib.MOE_ERR_ARG), (70000, ok, lib.MOE_ERR_ARG),
                         (1, None, lib.MOE_ERR_ARG),
                         (1, tensors((None, 1, F32)), lib.MOE_ERR_ARG),
                         (1, tensors((0x10002, 1, F32)), lib.MOE_ERR_ARG),
                         (1, tensors((0x10001, 1, BF16)), lib.MOE_ERR_ARG),
                         (1, tensors((0x10000, 1, 2)), lib.MOE_ERR_ARG),
                         (1, tensors((0x10000, -1, F32)), lib.MOE_ERR_UNSUPPORTED),
                         (1, tensors((0x10000, (1 << 40) + 1, F32)), lib.MOE_ERR_UNSUPPORTED),
                         (2, tensors((0x10000, 1 << 40, F32), (0x10000, 1, F32)),
                          lib.MOE_ERR_UNSUPPORTED)):
        assert L.moe_grad_norm(n, bad, 1.0, P, P, BIG, None) == code
        assert L.moe_grad_clip(n, bad, P, None, None) == code
    out = tensors((0x10000, 10, BF16), (0x20002, 4, BF16), (None, 0, F32))
    assert L.moe_grad_clip(3, ok, P, out, None) == lib.MOE_ERR_ARG
    assert "out[1]" in lib.last_error()

"""Workspaces of the layer's backward passes by name: the binding's sizes are what the
calls ask for (before any HIP call, so the pointers are never dereferenced)."""
import ctypes

import pytest

lib = pytest.importorskip("sparse_moe_transformer_router_amd.lib", reason="libmoe.so not built")

from tests.test_layer_train_abi import BIG, CALLS  # noqa: E402
from tests.test_workspace import _needed  # noqa: E402

L = lib.raw()
NAMES = {"expert_ffn_grad": ("moe_expert_ffn_grad",),
         "dense_mlp_grad": ("gemma4_dense_mlp_grad",),
         "norms_grad": ("gemma4_pre_norms_grad", "gemma4_post_norms_grad"),
         "layer": ("moe_expert_ffn_keep", "gemma4_dense_mlp")}


def asks(call, d, T):
    args = list(CALLS[call][0])
    assert args[-1] == BIG
    args[-1] = 0
    return _needed(getattr(L, call)(ctypes.byref(d), T, *args, None))


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("sizes", [(2816, 128, 8, 704, 2112), (64, 4, 2, 32, 96)])
def test_named_sizes_are_what_the_calls_ask_for(name, sizes):
    d = lib.dims(*sizes)
    before = 0
    for T in (1, 63, 700, 4096, 65536):
        n = lib.workspace_size(d, T, (name,))
        assert all(asks(c, d, T) == n for c in NAMES[name]) and n >= before
        before = n


def test_a_workspace_for_a_whole_step():
    """One buffer of the largest size serves every call named; the default does not name
    the backward passes, and says so by its size."""
    d = lib.dims(2816, 128, 8, 704, 2112)
    step = ("layer", "balance_loss", "router_grad", "expert_ffn_grad", "dense_mlp_grad",
            "norms_grad")
    need = lib.workspace_size(d, 300, step)
    assert need == max(lib.workspace_size(d, 300, (c,)) for c in step)
    assert need >= max(asks(c, d, 300) for cs in NAMES.values() for c in cs)
    old = ("layer", "balance_loss", "router_grad", "expert_ffn_b128")
    assert lib.workspace_size(d, 300) == lib.workspace_size(d, 300, old)
    with pytest.raises(ValueError):
        lib.workspace_size(d, 300, ("grad_norm",))
    with pytest.raises(lib.MoeError):
        lib.workspace_size(lib.dims(64, 4, 2, 32, 0), 300, ("dense_mlp_grad",))

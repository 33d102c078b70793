"""Workspace sizes, as the calls' refusals name them (before any HIP call, so the
pointers are never dereferenced).  The figures of the layer's calls are those of
the library before the training calls and the block-scaled experts came."""
import ctypes
import re

import pytest

lib = pytest.importorskip("sparse_moe_transformer_router_amd.lib", reason="libmoe.so not built")
L = lib.raw()
FAKE = ctypes.c_void_p(0x10000)


def _needed(rc):
    """Bytes that a call refused for want of them asks for."""
    assert rc == lib.MOE_ERR_WORKSPACE
    return int(re.search(r"(\d+) needed", lib.last_error()).group(1))


def _asks(d, T):
    """What each call asks for when it is given no byte."""
    p, r, f = ctypes.byref(d), lambda n: [FAKE] * n, (ctypes.c_float(0.1), ctypes.c_float(0.1))
    end = (FAKE, 0, None)
    return {
        "moe_router": _needed(L.moe_router(p, T, *r(7), *end)),
        "moe_route": _needed(L.moe_route(p, T, *r(10), *end)),
        "moe_router_logits": _needed(L.moe_router_logits(p, T, *r(8), *end)),
        "moe_dispatch": _needed(L.moe_dispatch(p, T, *r(4), *end)),
        "moe_expert_ffn": _needed(L.moe_expert_ffn(p, T, *r(7), *end)),
        "moe_balance_loss": _needed(L.moe_balance_loss(p, T, *r(2), None, *f, *r(3), *end)),
        "moe_router_grad": _needed(L.moe_router_grad(p, T, *r(15), *end)),
        "moe_expert_ffn_b128": _needed(L.moe_expert_ffn_b128(p, T, *r(9), *end)),
    }


LAYER = ("moe_router", "moe_route", "moe_router_logits", "moe_dispatch", "moe_expert_ffn")


@pytest.mark.parametrize("sizes,figures", [
    ((2816, 128, 8, 704, 2112), {1: 141312, 8: 1102592, 64: 8801280, 4096: 563168768}),
    ((8192, 256, 8, 704, 0), {1: 359424, 257: 91077632}),
    ((64, 4, 2, 32, 0), {1: 5376, 65536: 87821056})])
def test_the_layers_calls_ask_for_what_they_use(sizes, figures):
    """No call asks for another's scratch."""
    d = lib.dims(*sizes)
    for T, n in figures.items():
        asks = _asks(d, T)
        assert all(asks[c] == n for c in LAYER), (T, asks)
        assert L.moe_workspace_size(ctypes.byref(d), T) == n
        assert lib.workspace_size(d, T, ("layer",)) == n


@pytest.mark.parametrize("sizes", [(2816, 128, 8, 704, 2112), (64, 4, 2, 32, 0)])
def test_size_functions_are_what_the_calls_ask_for(sizes):
    d = lib.dims(*sizes)
    before = dict.fromkeys(("balance_loss", "router_grad", "expert_ffn_b128"), 0)
    for T in (1, 63, 256, 257, 700, 4096, 65536):
        asks = _asks(d, T)
        for c in before:
            n = lib.workspace_size(d, T, (c,))
            assert n == asks["moe_" + c] and n >= before[c]  # serves smaller batches
            before[c] = n
        # the default serves every call
        assert lib.workspace_size(d, T) == max(asks.values())


def test_training_scratch_does_not_contain_a_layers():
    """The balance loss: two values per expert and two more from each of at most 256
    blocks, whatever the layer around it."""
    a = lambda n: (n + 255) // 256 * 256  # noqa: E731
    want = 2 * a(4 * 256 * 128) + 2 * a(4 * 256)
    for sizes in ((2816, 128, 8, 704, 2112), (64, 128, 1, 32, 0), (8192, 128, 16, 8192, 0)):
        d = lib.dims(*sizes)
        assert lib.workspace_size(d, 65536, ("balance_loss",)) == want
        assert _asks(d, 65536)["moe_balance_loss"] == want
    # the router's backward does not know the experts' width
    assert len({lib.workspace_size(lib.dims(2816, 128, 8, i, 0), 4096, ("router_grad",))
                for i in (32, 704, 8192)}) == 1


@pytest.mark.parametrize("calls", [("layer",), ("balance_loss",), ("router_grad",),
                                   ("expert_ffn_b128",), tuple(lib._WS_SIZES)])
def test_no_tokens(calls):
    """An empty batch is a size like any other (0 bytes would say unsupported)."""
    d = lib.dims(64, 4, 2, 32)
    assert 0 < lib.workspace_size(d, 0, calls) <= lib.workspace_size(d, 1, calls)


def test_refusals():
    for f in lib._WS_SIZES.values():
        size = getattr(L, f)
        assert size(ctypes.byref(lib.dims(100, 4, 2, 32)), 8) == 0 and "hidden" in lib.last_error()
        assert size(ctypes.byref(lib.dims(64, 4, 2, 32)), 65537) == 0
        assert size(ctypes.byref(lib.dims(64, 4, 2, 32)), -1) == 0
    with pytest.raises(ValueError):
        lib.workspace_size(lib.dims(64, 4, 2, 32), 8, ("router",))
    with pytest.raises(lib.MoeError):
        lib.workspace_size(lib.dims(100, 4, 2, 32), 8)

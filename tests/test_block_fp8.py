"""Block-scaled E4M3 without a GPU: the reference quantizer's rules, and the
library's refusals (before any HIP call: the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from tests import b128_ref as ref

lib = pytest.importorskip("sparse_moe_transformer_router_amd.lib", reason="libmoe.so not built")
L = lib.raw()
FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
BIG = 1 << 40


@pytest.mark.parametrize("rows,cols,br", [(5, 16, 1), (3, 304, 1), (130, 272, 128), (128, 128, 128)])
def test_reference_codes_are_nearest(rows, cols, br):
    """Each code's value is within half a step of the input: 2^-4 relative, or
    half of 2^-9 scales below the smallest normal; the block maximum is exact
    to fp32."""
    g = torch.Generator().manual_seed(rows + cols)
    v = torch.randn(rows, cols, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))
    v[0, :16] = 0
    q, s = ref.quantize(v, br)
    assert s.shape == ((rows + br - 1) // br, ref.blocks(cols))
    val = ref.values(q, s, br)
    full = s.double().repeat_interleave(br, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    err = (val - v.double()).abs()
    assert torch.all(err <= torch.maximum(2.0 ** -4 * v.double().abs(), 2.0 ** -10 * full) * 1.0001)


def test_reference_bound_holds_its_own_value():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 64, generator=g).bfloat16().float()
    gu = ref.values(*ref.quantize(torch.randn(3, 64, 64, generator=g), 128), 128)
    dn = ref.values(*ref.quantize(torch.randn(3, 64, 32, generator=g), 128), 128)
    idx = torch.tensor([[0, 1], [1, 2], [2, 0], [1, 0]])
    y, err = ref.experts(x, gu, dn, idx, torch.ones(4, 2))
    assert torch.all(err > 0) and float((err / y.abs().mean()).median()) < 0.2


def _q(br=128, batch=1, rows=4, cols=32, w=FAKE, q=FAKE, s=FAKE):
    return L.moe_quantize_b128(br, batch, rows, cols, w, q, s, None)


def _dq(br=128, batch=1, rows=4, cols=32, q=FAKE, s=FAKE, o=FAKE):
    return L.moe_dequantize_b128(br, batch, rows, cols, q, s, o, None)


@pytest.mark.parametrize("f", [_q, _dq])
def test_quantize_refusals(f):
    assert f(br=64) == lib.MOE_ERR_ARG and f(br=0) == lib.MOE_ERR_ARG
    assert f(cols=8) == lib.MOE_ERR_ARG and f(cols=40) == lib.MOE_ERR_ARG
    assert f(cols=0) == lib.MOE_ERR_ARG and f(cols=65552) == lib.MOE_ERR_ARG
    assert f(rows=-1) == lib.MOE_ERR_ARG and f(batch=-1) == lib.MOE_ERR_ARG
    assert f(batch=1 << 30, rows=1 << 20) == lib.MOE_ERR_UNSUPPORTED
    # a launch's lanes are counted in 32 bits: 16 of them per row and 128 columns
    assert f(batch=1 << 8, rows=1 << 20, cols=16) == lib.MOE_ERR_UNSUPPORTED
    assert f(batch=1 << 7, rows=1 << 20, cols=256) == lib.MOE_ERR_UNSUPPORTED
    assert f(batch=0) == lib.MOE_OK and f(rows=0) == lib.MOE_OK
    for k in ("w", "q", "s", "o"):
        if k in f.__code__.co_varnames:
            assert f(**{k: None}) == lib.MOE_ERR_ARG and f(**{k: ODD}) == lib.MOE_ERR_ARG


def _lin(T=4, n=32, k=64, x=FAKE, q=FAKE, s=FAKE, y=FAKE, dt=1, ws=FAKE, nb=BIG):
    return L.moe_linear_b128(T, n, k, x, q, s, y, dt, ws, nb, None)


def test_linear_refusals():
    assert _lin(T=-1) == lib.MOE_ERR_ARG and _lin(T=65537) == lib.MOE_ERR_ARG
    assert _lin(n=0) == lib.MOE_ERR_UNSUPPORTED and _lin(n=(1 << 18) + 1) == lib.MOE_ERR_UNSUPPORTED
    for k in (0, 8, 40, 16400):
        assert _lin(k=k) == lib.MOE_ERR_UNSUPPORTED
        assert L.moe_linear_b128_workspace_size(4, k) == 0
    assert _lin(dt=2) == lib.MOE_ERR_ARG
    for a in ("x", "q", "s", "y"):
        assert _lin(**{a: None}) == lib.MOE_ERR_ARG and _lin(**{a: ODD}) == lib.MOE_ERR_ARG
    assert _lin(ws=None) == lib.MOE_ERR_WORKSPACE
    assert _lin(ws=ctypes.c_void_p(0x10010)) == lib.MOE_ERR_WORKSPACE
    need = L.moe_linear_b128_workspace_size(4, 64)
    assert _lin(nb=need - 1) == lib.MOE_ERR_WORKSPACE
    assert _lin(T=0, x=None, ws=None) == lib.MOE_OK
    sizes = [L.moe_linear_b128_workspace_size(t, 2816) for t in (0, 1, 64, 65536)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def _ffn(T=4, ws=FAKE, nb=BIG, act=None, **kw):
    d = lib.dims(kw.pop("hidden", 2816), 128, 8, 704,
                 act=lib.MOE_BF16 if act is None else act)
    a = {k: FAKE for k in ("x", "guq", "gus", "dnq", "dns", "w", "off", "srt", "y")}
    a.update(kw)
    return L.moe_expert_ffn_b128(ctypes.byref(d), T, *a.values(), ws, nb, None)


def test_experts_refusals():
    assert _ffn(act=lib.MOE_F32) == lib.MOE_ERR_UNSUPPORTED
    assert _ffn(hidden=100) == lib.MOE_ERR_UNSUPPORTED
    assert _ffn(T=-1) == lib.MOE_ERR_ARG
    for k in ("x", "guq", "gus", "dnq", "dns", "w", "off", "srt", "y"):
        assert _ffn(**{k: None}) == lib.MOE_ERR_ARG and _ffn(**{k: ODD}) == lib.MOE_ERR_ARG
    assert _ffn(ws=None) == lib.MOE_ERR_WORKSPACE and _ffn(nb=1000) == lib.MOE_ERR_WORKSPACE
    assert _ffn(T=0, x=None, ws=None) == lib.MOE_OK


def test_workspace_serves_smaller_batches():
    """Monotone in the tokens across the change of form at 256."""
    d = lib.dims(2816, 128, 8, 704)
    sizes = [lib.workspace_size(d, t) for t in (1, 255, 256, 257, 300, 512, 4096)]
    assert sizes == sorted(sizes)

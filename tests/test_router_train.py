"""The router's training calls without a GPU: the fp64 reference of the GPU
tests against central differences, and the library's refusals (which come
before any HIP call, so the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from tests import router_train_ref as ref

lib = pytest.importorskip("sparse_moe_transformer_router_amd.lib", reason="libmoe.so not built")
L = lib.raw()
FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10004)
BIG = 1 << 40


def _close(got, want, scale):
    # central differences of fp64: h = 1e-5 leaves h^2 * third derivative and
    # 2^-53 / h, both below 1e-9 of these O(1) functions
    assert abs(float(got) - float(want)) <= 1e-7 * scale


def test_balance_gradient_is_the_difference_quotient():
    g = torch.Generator().manual_seed(1)
    lg = torch.randn(9, 6, generator=g, dtype=torch.float64)
    idx = torch.stack([torch.randperm(6, generator=g)[:2] for _ in range(9)])
    mask = torch.tensor([1, 1, 0, 1, 1, 1, 0, 1, 1], dtype=torch.uint8)
    d, mag = ref.balance_grad(lg, idx, mask, 0.3, 0.2, 1.7)
    assert torch.all(d.abs() <= mag * (1 + 1e-12))
    h = 1e-5
    for t, e in ((0, 0), (3, 5), (2, 1), (8, 4)):
        up, dn = lg.clone(), lg.clone()
        up[t, e] += h
        dn[t, e] -= h
        q = 1.7 * (ref.balance(up, idx, mask, 0.3, 0.2)[0]
                   - ref.balance(dn, idx, mask, 0.3, 0.2)[0]) / (2 * h)
        _close(d[t, e], q, 1.0)


@pytest.mark.parametrize("pre", [False, True])
def test_router_gradient_is_the_difference_quotient(pre):
    g = torch.Generator().manual_seed(2)
    T, H, E, K = 5, 64, 6, 3
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    a = {"x": n(T, H), "W": n(E, H) * 0.2, "scale": 1 + 0.1 * n(H), "pes": 1 + 0.1 * n(E),
         "gain": 1 + 0.1 * n(H) if pre else None}
    idx = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)])
    idx[1, 2] = -1                                    # no slot
    mask = torch.tensor([1, 1, 1, 0, 1], dtype=torch.uint8)
    dw, dl = n(T, K), n(T, E)
    got, tol = ref.router_grad(*a.values(), idx, mask, dw, dl, 1e-6, 1)
    assert set(got) == {k for k, v in a.items() if v is not None}
    h = 1e-5
    for k, v in a.items():
        if v is None:
            continue
        step = n(*v.shape)
        f = lambda s: ref.router_objective(  # noqa: E731
            *{**a, k: v + s * h * step}.values(), idx, mask, dw, dl, 1e-6)
        _close((got[k] * step).sum(), (f(1) - f(-1)) / (2 * h), 10.0)


def dims(**kw):
    base = dict(hidden=2816, num_experts=128, top_k=8, expert_inter=704, act=lib.MOE_BF16)
    return lib.dims(**{**base, **kw})


def _balance(d, T=4, lg=FAKE, idx=FAKE, mask=None, loss=FAKE, cnt=FAKE, p=FAKE, ws=FAKE, n=BIG):
    return L.moe_balance_loss(ctypes.byref(d), T, lg, idx, mask, 0.1, 0.1, loss, cnt, p, ws, n,
                              None)


def _balance_grad(d, T=4, lg=FAKE, mask=None, cnt=FAKE, loss=FAKE, g=FAKE, out=FAKE):
    return L.moe_balance_loss_grad(ctypes.byref(d), T, lg, mask, cnt, loss, 0.1, 0.1, g, out,
                                   None)


def _grad(d, T=4, ws=FAKE, n=BIG, **kw):
    names = ("x", "W", "scale", "pes", "gain", "logits", "idx", "mask", "dw", "dl", "dx", "dW",
             "dscale", "dpes", "dgain")
    a = {k: FAKE for k in names}
    a.update(mask=None)
    a.update(kw)
    return L.moe_router_grad(ctypes.byref(d), T, *[a[k] for k in names], ws, n, None)


def test_balance_refusals():
    d = dims()
    assert _balance(dims(num_experts=300)) == lib.MOE_ERR_UNSUPPORTED
    assert _balance(d, T=-1) == lib.MOE_ERR_ARG and _balance(d, T=65537) == lib.MOE_ERR_ARG
    for k in ("lg", "idx", "loss", "cnt", "p"):
        assert _balance(d, **{k: None}) == lib.MOE_ERR_ARG
        assert _balance(d, **{k: ODD}) == lib.MOE_ERR_ARG
    assert _balance(d, mask=ODD) == lib.MOE_ERR_ARG
    assert _balance(d, ws=None) == lib.MOE_ERR_WORKSPACE
    assert _balance(d, n=100) == lib.MOE_ERR_WORKSPACE
    for k in ("lg", "cnt", "loss", "g", "out"):
        assert _balance_grad(d, **{k: None}) == lib.MOE_ERR_ARG
        assert _balance_grad(d, **{k: ODD}) == lib.MOE_ERR_ARG
    assert _balance_grad(d, T=0, lg=None, out=None) == lib.MOE_OK


def test_router_grad_refusals():
    d = dims()
    for k in ("x", "W", "scale", "pes", "logits", "idx", "dW", "dscale", "dpes", "dgain"):
        assert _grad(d, **{k: None}) == lib.MOE_ERR_ARG, k
        assert _grad(d, **{k: ODD}) == lib.MOE_ERR_ARG, k
    for k in ("mask", "dw", "dl", "dx"):
        assert _grad(d, **{k: ODD}) == lib.MOE_ERR_ARG, k
    assert _grad(d, dw=None, dl=None) == lib.MOE_ERR_ARG
    assert _grad(d, gain=None) == lib.MOE_ERR_ARG and "d_pre_norm_gain" in lib.last_error()
    assert _grad(d, ws=None) == lib.MOE_ERR_WORKSPACE
    assert _grad(d, n=1000) == lib.MOE_ERR_WORKSPACE
    assert _grad(dims(hidden=100)) == lib.MOE_ERR_UNSUPPORTED


def test_binding_checks_types_and_sizes():
    d = dims()
    cpu = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="not on the current GPU"):
        lib._arg("logits", cpu, torch.float32, 4, 0)
    with pytest.raises(TypeError, match="logits"):
        lib._arg("logits", cpu.double(), torch.float32, 4, 0)
    with pytest.raises(ValueError, match="needed"):
        lib._arg("logits", cpu, torch.float32, 4096, 0)
    with pytest.raises(ValueError, match="required"):
        lib._arg("logits", None, torch.float32, 4, 0)
    assert lib._arg("token_mask", None, lib._MASK, 4, 0, True) is None
    assert d.num_experts == 128

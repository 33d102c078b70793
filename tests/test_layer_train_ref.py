"""The fp64 reference of the layer's training step against central differences (CPU)."""
import torch

from tests import layer_train_ref as ref

torch.manual_seed(0)
EPS = 1e-6


def differences(f, v, step=1e-6):
    d = torch.zeros_like(v)
    flat, out = v.view(-1), d.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + step
        hi = f()
        flat[i] = keep - step
        lo = f()
        flat[i] = keep
        out[i] = (hi - lo) / (2 * step)
    return d


def near(a, b):
    return float((a - b).abs().max()) <= 1e-6 * max(1.0, float(b.abs().max()))


def test_slope():
    z = torch.linspace(-6, 6, 241, dtype=torch.float64)
    assert near(ref.slope(z), (ref.gelu(z + 1e-6) - ref.gelu(z - 1e-6)) / 2e-6)


def test_experts_grad():
    T, H, E, K, I = 5, 6, 3, 2, 4
    r = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    x, gu, dn, w, d = r(T, H), r(E, 2 * I, H), r(E, H, I), r(T, K), r(T, H)
    idx = torch.tensor([[0, 1], [2, 0], [1, -1], [0, 2], [1, 2]], dtype=torch.int32)
    mask = torch.tensor([1, 1, 1, 0, 1], dtype=torch.uint8)

    def rows():
        return [(e, t, k) for e in range(E) for t in range(T) for k in range(K)
                if int(idx[t, k]) == e]

    def value():
        total = 0.0
        for e, t, k in rows():
            if mask[t]:
                z = gu[e] @ x[t]
                total += w[t, k] * (d[t] @ (dn[e] @ (ref.gelu(z[:I]) * z[I:])))
        return float(total)

    kept = torch.zeros(T * K, 2 * I, dtype=torch.float64)
    for i, (e, t, _) in enumerate(rows()):
        kept[i] = gu[e] @ x[t]
    got = ref.experts_grad(x, gu, dn, w, idx, kept, mask, d, False, False)
    for name, leaf in (("d_x", x), ("d_w", w), ("d_gate_up", gu), ("d_down", dn)):
        assert near(got[name][0], differences(value, leaf)), name


def test_dense_grad():
    T, H, D = 4, 5, 3
    r = lambda *s: torch.randn(*s, dtype=torch.float64)  # noqa: E731
    x, g, u, dn, d = r(T, H), r(D, H), r(D, H), r(H, D), r(T, H)
    mask = torch.tensor([1, 0, 1, 1], dtype=torch.uint8)

    def value():
        y = (ref.gelu(x @ g.t()) * (x @ u.t())) @ dn.t()
        return float((y * d * mask[:, None]).sum())

    got = ref.dense_grad(x, g, u, dn, torch.cat([x @ g.t(), x @ u.t()], 1), mask, d, False, False)
    for name, leaf in (("d_x", x), ("d_gate", g), ("d_up", u), ("d_down", dn)):
        assert near(got[name][0], differences(value, leaf)), name

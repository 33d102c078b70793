"""The layer's norms and their backward passes on the GPU against fp64."""
import pytest
import torch

from tests import layer_train_ref as ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_moe_transformer_router_amd import lib
else:
    lib = None

EPS = 1e-6


def rel(got, want):
    """RMS error over RMS value, and the largest error over the larger of a value and
    the RMS."""
    got, want = got.double(), want.double()
    assert torch.isfinite(got).all()
    rms = float(want.square().mean().sqrt())
    e = (got - want).abs()
    if rms == 0:
        return float(e.max()), float(e.max())
    return float(e.square().mean().sqrt()) / rms, float((e / want.abs().clamp(min=rms)).max())


def holds(got, want, bf16, name):
    """One rounding to the stored type (bf16 2^-8, 2.3e-3 in the RMS) on top of fp32
    arithmetic: a norm's chain of sums over up to 8192 columns and its few products, and
    sums over tokens of values that cancel, within 1e-5 of the RMS and 1e-4 at worst."""
    r, m = rel(got, want)
    assert r <= (2.4e-3 if bf16 else 0) + 1e-5 and m <= (2.0 ** -8 if bf16 else 0) + 1e-4, \
        (name, r, m)


class Norms:
    def __init__(self, T, H, K=3, bf16=True, slot16=True, seed=0, pad=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        dt = torch.bfloat16 if bf16 else torch.float32
        st = torch.bfloat16 if bf16 and slot16 else torch.float32
        self.T, self.H, self.bf16, self.st = T, H, bf16, st
        self.d = lib.dims(H, max(K, 2), K, 32, 0, EPS, lib.MOE_BF16 if bf16 else lib.MOE_F32,
                          lib.MOE_BF16 if st == torch.bfloat16 else lib.MOE_F32)
        self.x = (3 * r(T, H)).to(dt)
        self.y, self.dn = r(T, K, H).to(st), (0.3 * r(T, H)).to(st)
        self.g = [1 + 0.2 * r(H) for _ in range(3)]
        self.scalar = 0.7
        self.mask = None
        if pad:
            self.mask = (torch.rand(T, generator=g, device="cuda") >= pad).to(torch.uint8)
        self.d_out = (r(T, H) + 0.3 * self.x.float()).to(dt)
        self.d_xd, self.d_xm, self.d_add = (r(T, H).to(dt) for _ in range(3))
        nan = lambda *s, t=dt: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        self.out, self.ffn, self.total = nan(T, H), nan(T, H, t=torch.float32), nan(T, H, t=st)
        self.xd, self.xm, self.d_x = nan(T, H), nan(T, H), nan(T, H)
        self.d_dn, self.d_moe = nan(T, H), nan(T, H)
        self.d_g = [nan(H, t=torch.float32) for _ in range(3)]
        self.d_pre = [nan(H, t=torch.float32) for _ in range(2)]
        self.d_s = nan(1, t=torch.float32)
        self.ws = lib.norms_grad_workspace(self.d, T)
        self.ws.fill_(255)

    def forward(self):
        lib.gemma4_pre_norms(self.d, self.T, self.x, self.g[0], self.g[1], self.xd, self.xm)
        lib.gemma4_post_norms(self.d, self.T, self.x, self.y, self.dn, *self.g, self.scalar,
                              self.out, self.total, self.ffn)

    def backward(self, stream=None):
        lib.gemma4_post_norms_grad(self.d, self.T, self.x, self.dn, self.total, *self.g,
                                   self.scalar, self.mask, self.d_out, self.d_dn, self.d_moe,
                                   *self.d_g, self.d_s, self.ws, stream)
        lib.gemma4_pre_norms_grad(self.d, self.T, self.x, self.g[0], self.g[1], self.mask,
                                  self.d_xd, self.d_xm, self.d_add, self.d_out, self.scalar,
                                  self.d_x, *self.d_pre, self.ws, stream)

    def results(self):
        return [self.d_dn, self.d_moe, self.d_x, *self.d_g, *self.d_pre, self.d_s]

    def want(self):
        on = (torch.arange(self.T, device="cuda") if self.mask is None
              else self.mask.nonzero()[:, 0])
        leaf = lambda t: ref.f64(t).requires_grad_(True)  # noqa: E731
        x, dn, total = leaf(self.x), leaf(self.dn), leaf(self.total)
        g = [leaf(t) for t in self.g]
        s = torch.tensor([self.scalar], dtype=torch.float32, device="cuda").double()
        s.requires_grad_(True)
        d = ref.f64(self.d_out)[on]
        out = ref.behind(ref.f64(self.x)[on], dn[on], total[on], *g, s, EPS)
        behind = torch.autograd.grad((out * d).sum(), [dn, total, *g, s])
        p = [leaf(t) for t in self.g[:2]]
        n = ref.norm(x[on], EPS)
        before = torch.autograd.grad(
            (n * p[0] * ref.f64(self.d_xd)[on] + n * p[1] * ref.f64(self.d_xm)[on]
             + x[on] * (ref.f64(self.d_add)[on] + s.detach() * d)).sum(), [x, *p])
        return [behind[0], behind[1], before[0], *behind[2:5], *before[1:], behind[5]]

    def check(self):
        names = ("d_dn", "d_moe", "d_x", "d_g1", "d_g2", "d_g3", "d_pre", "d_pre2", "d_scalar")
        for i, (n, a, b) in enumerate(zip(names, self.results(), self.want())):
            holds(a, b, self.bf16 and i < 3, n)


SIZES = [(1, 64), (1, 2816), (5, 8192), (37, 192), (333, 2816), (700, 512), (2100, 576)]


@pytest.mark.parametrize("kind", ["bf16", "bf16_f32slots", "f32"])
@pytest.mark.parametrize("T,H", SIZES)
def test_norms(T, H, kind):
    s = Norms(T, H, bf16=kind != "f32", slot16=kind == "bf16", seed=T + H,
              pad=0.3 if T in (37, 700) else 0.0)
    note(f"norms and their backward passes T={T} H={H} {kind}")
    s.forward()
    torch.cuda.synchronize()
    x = s.x.double()
    holds(s.xd, ref.norm(x, EPS) * s.g[0].double(), s.bf16, "xd")
    holds(s.xm, ref.norm(x, EPS) * s.g[1].double(), s.bf16, "xm")
    total = s.y.double().sum(1)
    out = ref.behind(x, s.dn.double(), total, *(g.double() for g in s.g), s.scalar, EPS)
    holds(s.out, out, s.bf16, "out")
    holds(s.ffn, out / s.scalar - x, False, "ffn_out")
    holds(s.total, total, s.st == torch.bfloat16, "moe_sum")
    s.backward()
    torch.cuda.synchronize()
    s.check()


def test_post_norms_is_the_layers_end():
    """The same bits with and without the optional outputs, one slot or many."""
    for K in (1, 3, 8):
        s = Norms(50, 320, K=K, seed=K)
        note(f"post norms K={K}")
        s.forward()
        out = torch.empty_like(s.out)
        lib.gemma4_post_norms(s.d, s.T, s.x, s.y, s.dn, *s.g, s.scalar, out, None, None)
        torch.cuda.synchronize()
        assert torch.equal(out, s.out)


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_masked_rows_may_hold_anything(bf16):
    s = Norms(120, 320, bf16=bf16, slot16=bf16, seed=5, pad=0.4)
    s.forward()
    torch.cuda.synchronize()
    want = s.want()
    off = s.mask == 0
    for v in (s.x, s.dn, s.total, s.d_out, s.d_xd, s.d_xm, s.d_add):
        v[off] = float("nan")
    note("norms' backward passes, NaN in masked rows")
    s.backward()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(s.results(), want)):
        holds(a, b, bf16 and i < 3, i)
    assert all((v[off] == 0).all() for v in (s.d_dn, s.d_moe, s.d_x))
    s.mask.zero_()
    s.backward()
    torch.cuda.synchronize()
    assert all((v == 0).all() for v in s.results())


def test_rows_of_zeros():
    """A row of zeros has a finite norm (eps) and finite gradients."""
    s = Norms(9, 192, bf16=False, seed=6)
    s.forward()
    for v in (s.x, s.dn, s.total):
        v[3] = 0
    note("rows of zeros")
    s.backward()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(s.results(), s.want())):
        holds(a, b, False, i)


def test_optional_inputs_and_in_place():
    s = Norms(40, 320, seed=7)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    d_x, pre = s.d_x.clone(), [v.clone() for v in s.d_pre]
    note("optional inputs of the norms' backward passes")
    g = [torch.empty_like(v) for v in s.d_g]
    a, b = torch.empty_like(s.d_dn), torch.empty_like(s.d_moe)
    lib.gemma4_post_norms_grad(s.d, s.T, None, s.dn, s.total, *s.g, s.scalar, None, s.d_out, a, b,
                               *g, None, s.ws)
    torch.cuda.synchronize()
    assert torch.equal(a, s.d_dn) and torch.equal(b, s.d_moe)
    assert all(torch.equal(u, v) for u, v in zip(g, s.d_g))
    # without the two addends: the norms' part alone
    part = torch.empty_like(s.d_x)
    lib.gemma4_pre_norms_grad(s.d, s.T, s.x, s.g[0], s.g[1], None, s.d_xd, s.d_xm, None, None,
                              s.scalar, part, *s.d_pre, s.ws)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(pre, s.d_pre))
    x = ref.f64(s.x).requires_grad_(True)
    n = ref.norm(x, EPS)
    want, = torch.autograd.grad((n * s.g[0].double() * s.d_xd.double()
                                 + n * s.g[1].double() * s.d_xm.double()).sum(), x)
    holds(part, want, True, "norms' part")
    # d_x in the place of each of its inputs
    for name in ("d_xd", "d_xm", "d_add", "d_out", "x"):
        v = {n: getattr(s, n).clone() for n in ("x", "d_xd", "d_xm", "d_add", "d_out")}
        lib.gemma4_pre_norms_grad(s.d, s.T, v["x"], s.g[0], s.g[1], None, v["d_xd"], v["d_xm"],
                                  v["d_add"], v["d_out"], s.scalar, v[name], *s.d_pre, s.ws)
        torch.cuda.synchronize()
        assert torch.equal(v[name], d_x), name


def test_no_tokens():
    s = Norms(1, 128, seed=8)
    note("norms' backward passes, no tokens")
    lib.gemma4_post_norms_grad(s.d, 0, s.x, s.dn, s.total, *s.g, s.scalar, None, s.d_out, s.d_dn,
                               s.d_moe, *s.d_g, s.d_s, None)
    lib.gemma4_pre_norms_grad(s.d, 0, s.x, s.g[0], s.g[1], None, s.d_xd, s.d_xm, None, None,
                              s.scalar, s.d_x, *s.d_pre, None)
    torch.cuda.synchronize()
    assert all((v == 0).all() for v in (*s.d_g, *s.d_pre, s.d_s))
    assert s.d_x.isnan().all() and s.d_dn.isnan().all()


def test_repeat_and_replay():
    s, other = Norms(600, 576, seed=9, pad=0.1), Norms(77, 192, seed=10)
    for v in (s, other):
        v.forward()
        v.backward()
    torch.cuda.synchronize()
    want = [v.clone() for v in s.results()]
    st = torch.cuda.Stream()

    def spoil():
        for v in s.results():
            v.fill_(float("nan"))
        s.ws.fill_(255)
        torch.cuda.synchronize()

    spoil()
    s.backward(st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, s.results()))
    gr = torch.cuda.CUDAGraph()
    note("capture the norms' backward passes")
    with torch.cuda.graph(gr, stream=st):
        s.backward()
    for _ in range(4):
        spoil()
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, s.results()))
        other.backward()
        torch.cuda.synchronize()

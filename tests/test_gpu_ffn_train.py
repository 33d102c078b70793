"""The gated block's training calls on the GPU: moe_expert_ffn_keep, moe_expert_ffn_grad,
gemma4_dense_mlp and gemma4_dense_mlp_grad against fp64, at their edges."""
import pytest
import torch

from tests import layer_train_ref as ref
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_moe_transformer_router_amd import lib
else:
    lib = None

# RMS of the error over the RMS of the value.  A bf16 rounding is off by at most
# 2^-8, evenly spread: 2^-8 / sqrt(3) = 2.3e-3 in the root mean square at most; d_x
# is rounded three times ([d_gate, d_up], the slots' parts, the sum), a weight's
# gradient twice: 3.9e-3 and 3.2e-3.  One lost row of 256 would be 6e-2.
RMS_BF16, RMS_F32 = 5e-3, 1e-5


def close(got, want, name, bf16):
    value, bound = want
    got = got.double().to(value.device)
    err = (got - value).abs()
    assert torch.isfinite(got).all(), name
    assert (err <= bound).all(), (name, float((err - bound).max()), float(err.max()))
    rms = float(value.square().mean().sqrt())
    if rms > 0:
        lim = RMS_BF16 if bf16 else RMS_F32
        assert float(err.square().mean().sqrt()) <= lim * rms, (name, float(
            err.square().mean().sqrt()) / rms)


class Experts:
    def __init__(self, T, H, E, K, I, bf16=True, seed=0, pad=0.0, drop=0.0, skew=False,
                 store=None, slot=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        dt = torch.bfloat16 if bf16 else torch.float32
        self.T, self.H, self.E, self.K, self.I, self.bf16 = T, H, E, K, I, bf16
        self.store = bf16 if store is None else store
        mt = lib.MOE_BF16 if bf16 else lib.MOE_F32
        self.d = lib.dims(H, E, K, I, 0, 1e-6, mt, lib.MOE_F32 if slot is None else slot)
        self.x = r(T, H).to(dt)
        self.gu = (r(E, 2 * I, H) / H ** 0.5).to(dt)
        self.dn = (r(E, H, I) / I ** 0.5).to(dt)
        score = r(T, E) + (torch.linspace(3, -3, E, device="cuda") if skew else 0)
        self.idx = torch.topk(score, K, -1).indices.to(torch.int32)
        if drop:
            gone = torch.rand(T, K, generator=g, device="cuda") < drop
            self.idx[gone] = -1
        self.w = torch.rand(T, K, generator=g, device="cuda") + 0.1
        self.mask = None
        if pad:
            self.mask = (torch.rand(T, generator=g, device="cuda") >= pad).to(torch.uint8)
        self.d_out = r(T, H).to(dt)
        i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.cnt, self.off, self.srt = i32(E), i32(E + 1), i32(T * K)
        self.ws = lib.workspace(self.d, T, calls=("layer",))
        nan = lambda *s, t=dt: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        wt = torch.bfloat16 if self.store else torch.float32
        self.kept = nan(T * K, 2 * I)
        self.y = nan(T, K, H, t=torch.bfloat16 if self.d.slot_dtype else torch.float32)
        self.d_x, self.d_w = nan(T, H), nan(T, K, t=torch.float32)
        self.d_gu, self.d_dn = nan(E, 2 * I, H, t=wt), nan(E, H, I, t=wt)
        self.gws = lib.expert_ffn_grad_workspace(self.d, T)
        self.gws.fill_(255)  # NaN and -1 wherever a kernel reads what none wrote
        lib.moe_dispatch(self.d, T, self.idx, self.cnt, self.off, self.srt, self.ws)

    def forward(self):
        lib.moe_expert_ffn_keep(self.d, self.T, self.x, self.gu, self.dn, self.w, self.off,
                                self.srt, self.kept, self.y, self.ws)

    def backward(self, stream=None):
        lib.moe_expert_ffn_grad(self.d, self.T, self.x, self.gu, self.dn, self.w, self.off,
                                self.srt, self.kept, self.mask, self.d_out, self.d_x, self.d_w,
                                self.d_gu, self.d_dn, self.gws, stream)

    def outputs(self):
        return {"d_x": self.d_x, "d_w": self.d_w, "d_gate_up": self.d_gu, "d_down": self.d_dn}

    def want(self):
        return ref.experts_grad(self.x, self.gu, self.dn, self.w, self.idx, self.kept, self.mask,
                                self.d_out, self.bf16, self.store)

    def check(self):
        want = self.want()
        for k, v in self.outputs().items():
            lowp = self.bf16 and k != "d_w"
            close(v, want[k], k, lowp)


SIZES = [  # T, H, E, K, I
    (1, 64, 1, 1, 32),        # the smallest
    (1, 2816, 8, 8, 704),     # one token at the layer's widths
    (7, 128, 5, 2, 96),
    (64, 2816, 16, 4, 704),   # column tiles that end inside the matrices
    (300, 320, 6, 3, 224),
    (257, 256, 1, 1, 256),    # one row past a tile, sizes of exactly one
    (700, 576, 3, 2, 288),
    (40, 192, 12, 12, 64),    # every expert takes every token
    (5000, 256, 2, 1, 64),    # rows past what a block looks up at a time
    (90, 8192, 2, 1, 32),     # the widest hidden size
    (33, 64, 3, 2, 8192),     # the widest experts
]


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_experts_grad(size, bf16):
    note(f"moe_expert_ffn_grad {size} bf16={bf16}")
    s = Experts(*size, bf16=bf16, seed=1)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    s.check()


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 150, 900])
def test_experts_keep(T, bf16):
    """y_slots bit for bit those of moe_expert_ffn; the projections within rounding."""
    for slot in ([lib.MOE_F32, lib.MOE_BF16] if bf16 else [lib.MOE_F32]):
        s = Experts(T, 320, 6, 3, 224, bf16=bf16, seed=2, drop=0.1, slot=slot)
        note(f"moe_expert_ffn_keep T={T} bf16={bf16} slot={slot}")
        s.forward()
        y = torch.full_like(s.y, float("nan"))
        lib.moe_expert_ffn(s.d, T, s.x, s.gu, s.dn, s.w, s.off, s.srt, y, s.ws)
        torch.cuda.synchronize()
        there = s.idx >= 0
        assert torch.equal(y[there], s.y[there])
        assert s.y[~there].isnan().all()  # a dropped slot's row is left alone
        n = int(s.off[-1])
        assert s.kept[n:].isnan().all()
        at = 0
        for e in range(s.E):
            t, _ = (s.idx == e).nonzero(as_tuple=True)
            x, g = s.x[t].double(), s.gu[e].double()
            value, mag = x @ g.t(), x.abs() @ g.abs().t()
            bound = ref.SUM * mag + (ref.BF16 * value.abs() if bf16 else 0)
            got = s.kept[at:at + t.numel()].double()
            assert ((got - value).abs() <= bound).all()
            at += t.numel()


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_experts_grad_dropped_masked_and_empty(bf16):
    """Slots that the dispatch dropped, tokens that do not count with NaN in their rows,
    experts without rows (zeros)."""
    s = Experts(200, 320, 24, 3, 96, bf16=bf16, seed=3, pad=0.3, drop=0.2, skew=True)
    note("moe_expert_ffn_grad dropped, masked, empty")
    s.forward()
    off = s.mask == 0
    want = s.want()
    s.x[off] = float("nan")
    s.d_out[off] = float("nan")
    s.w[off] = float("nan")
    rows = s.srt[:int(s.off[-1])].long() // s.K
    s.kept[:rows.numel()][off[rows]] = float("nan")
    s.backward()
    torch.cuda.synchronize()
    for k, v in s.outputs().items():
        close(v, want[k], k, s.bf16 and k != "d_w")
    assert (s.d_x[off] == 0).all() and (s.d_w[off] == 0).all() and (s.d_w[s.idx < 0] == 0).all()
    empty = s.cnt == 0
    assert empty.any() and (s.d_gu[empty] == 0).all() and (s.d_dn[empty] == 0).all()


def test_experts_grad_all_tokens_masked():
    s = Experts(50, 128, 4, 2, 64, seed=4)
    s.forward()
    s.mask = torch.zeros(50, dtype=torch.uint8, device="cuda")
    note("moe_expert_ffn_grad, no token counts")
    s.backward()
    torch.cuda.synchronize()
    assert all((v == 0).all() for v in s.outputs().values())


def test_experts_grad_fp32_weight_gradients_of_bf16():
    s = Experts(300, 320, 6, 3, 224, seed=5, store=False)
    note("moe_expert_ffn_grad, fp32 weight gradients")
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    s.check()
    t = Experts(300, 320, 6, 3, 224, seed=5)
    t.forward()
    t.backward()
    torch.cuda.synchronize()
    assert torch.equal(s.d_gu.bfloat16(), t.d_gu) and torch.equal(s.d_dn.bfloat16(), t.d_dn)


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_experts_grad_each_output_alone(bf16):
    s = Experts(120, 192, 5, 2, 96, bf16=bf16, seed=6, pad=0.2)
    s.forward()
    note("moe_expert_ffn_grad, one output at a time")
    s.backward()
    torch.cuda.synchronize()
    all_of = {k: v.clone() for k, v in s.outputs().items()}
    for name in ("d_x", "d_w", "d_gu", "d_dn"):
        keep = {n: getattr(s, n) for n in ("d_x", "d_w", "d_gu", "d_dn")}
        keep[name].fill_(float("nan"))
        for n in keep:
            if n != name:
                setattr(s, n, None)
        s.gws.fill_(255)
        s.backward()
        torch.cuda.synchronize()
        key = {"d_x": "d_x", "d_w": "d_w", "d_gu": "d_gate_up", "d_dn": "d_down"}[name]
        assert torch.equal(keep[name], all_of[key]), name
        for n, v in keep.items():
            setattr(s, n, v)


def test_experts_grad_extreme_projections():
    """Projections far out on both sides: the slope is 1 or 0 there, nothing overflows."""
    s = Experts(40, 128, 3, 1, 64, seed=7)
    s.forward()
    torch.cuda.synchronize()
    far = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 5.0, -5.0, 12.0, -12.0, 100.0, -100.0, 1e15,
                        -1e15], device="cuda").to(torch.bfloat16)
    s.kept[:, :12] = far
    want = s.want()
    note("moe_expert_ffn_grad, extreme projections")
    s.backward()
    torch.cuda.synchronize()
    for k, v in s.outputs().items():
        value, bound = want[k]
        assert torch.isfinite(v).all(), k
        # the slope is evaluated in fp32: where s and 1 - s meet it is off by the
        # magnitudes of its terms, not of itself
        assert ((v.double() - value).abs() <= bound + 1e-5 * value.abs().max()).all(), k


class Dense:
    def __init__(self, T, H, D, bf16=True, seed=0, pad=0.0, store=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        dt = torch.bfloat16 if bf16 else torch.float32
        self.T, self.H, self.D, self.bf16 = T, H, D, bf16
        self.store = bf16 if store is None else store
        self.d = lib.dims(H, 4, 2, 32, D, 1e-6, lib.MOE_BF16 if bf16 else lib.MOE_F32)
        self.x = r(T, H).to(dt)
        self.gate, self.up = (r(D, H) / H ** 0.5).to(dt), (r(D, H) / H ** 0.5).to(dt)
        self.down = (r(H, D) / D ** 0.5).to(dt)
        self.d_y = r(T, H).to(dt)
        self.mask = None
        if pad:
            self.mask = (torch.rand(T, generator=g, device="cuda") >= pad).to(torch.uint8)
        nan = lambda *s, t=dt: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
        wt = torch.bfloat16 if self.store else torch.float32
        self.kept, self.y = nan(T, 2 * D), nan(T, H, t=torch.float32)
        self.d_x, self.d_gate, self.d_up = nan(T, H), nan(D, H, t=wt), nan(D, H, t=wt)
        self.d_down = nan(H, D, t=wt)
        self.ws = lib.workspace(self.d, T, calls=("layer",))
        self.gws = lib.dense_mlp_grad_workspace(self.d, T)
        self.gws.fill_(255)

    def forward(self, kept=True):
        lib.gemma4_dense_mlp(self.d, self.T, self.x, self.gate, self.up, self.down,
                             self.kept if kept else None, self.y, self.ws)

    def backward(self, stream=None):
        lib.gemma4_dense_mlp_grad(self.d, self.T, self.x, self.gate, self.up, self.down,
                                  self.kept, self.mask, self.d_y, self.d_x, self.d_gate,
                                  self.d_up, self.d_down, self.gws, stream)

    def outputs(self):
        return {k: getattr(self, k) for k in ("d_x", "d_gate", "d_up", "d_down")}

    def check(self):
        want = ref.dense_grad(self.x, self.gate, self.up, self.down, self.kept, self.mask,
                              self.d_y, self.bf16, self.store)
        for k, v in self.outputs().items():
            close(v, want[k], k, self.bf16)


DENSE = [(1, 64, 32), (5, 128, 96), (301, 2816, 2112), (64, 320, 1056), (17, 64, 16384),
         (20, 8192, 64), (2500, 192, 160)]


@pytest.mark.parametrize("size", DENSE, ids=str)
@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_dense(size, bf16):
    """Forward with and without the projections kept, backward."""
    s = Dense(*size, bf16=bf16, seed=8)
    note(f"gemma4_dense_mlp and its backward pass {size} bf16={bf16}")
    s.forward(kept=False)
    torch.cuda.synchronize()
    y = s.y.clone()
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    assert torch.equal(y, s.y)
    x = s.x.double()
    a, b = x @ s.gate.double().t(), x @ s.up.double().t()
    mag = x.abs() @ torch.cat([s.gate, s.up]).double().abs().t()
    value = torch.cat([a, b], 1)
    bound = ref.SUM * mag + (ref.BF16 * value.abs() if bf16 else 0)
    assert ((s.kept.double() - value).abs() <= bound).all()
    h = ref.gelu(a) * b
    want = h @ s.down.double().t()
    # h is rounded to bf16 once; its own sums are off by SUM of their magnitudes,
    # times the other factor (|gelu'| <= 1.13)
    D = s.D
    e_h = ref.SUM * (1.13 * mag[:, :D] * b.abs() + ref.gelu(a).abs() * mag[:, D:] + h.abs())
    e_h = e_h + (ref.BF16 * h.abs() if bf16 else 0)
    assert ((s.y.double() - want).abs() <= (e_h + ref.SUM * h.abs()) @ s.down.double().abs().t()
            ).all()
    s.check()


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("store", [True, False], ids=["act", "f32grads"])
def test_dense_grad_masked(bf16, store):
    s = Dense(150, 192, 160, bf16=bf16, seed=9, pad=0.3, store=store and bf16)
    note("gemma4_dense_mlp_grad masked")
    s.forward()
    off = s.mask == 0
    want = ref.dense_grad(s.x, s.gate, s.up, s.down, s.kept, s.mask, s.d_y, s.bf16, s.store)
    for v in (s.x, s.kept, s.d_y):
        v[off] = float("nan")
    s.backward()
    torch.cuda.synchronize()
    for k, v in s.outputs().items():
        close(v, want[k], k, s.bf16)
    assert (s.d_x[off] == 0).all()


def test_no_tokens():
    """T = 0: the weights' gradients are written as zeros."""
    for bf16 in (True, False):
        s = Experts(1, 128, 3, 2, 64, bf16=bf16, seed=10)
        note("no tokens")
        lib.moe_expert_ffn_grad(s.d, 0, s.x, s.gu, s.dn, s.w, s.off, s.srt, s.kept, None, s.d_out,
                                s.d_x, s.d_w, s.d_gu, s.d_dn, None)
        m = Dense(1, 128, 64, bf16=bf16, seed=10)
        lib.gemma4_dense_mlp_grad(m.d, 0, m.x, m.gate, m.up, m.down, m.kept, None, m.d_y, m.d_x,
                                  m.d_gate, m.d_up, m.d_down, None)
        torch.cuda.synchronize()
        assert all((v == 0).all() for v in (s.d_gu, s.d_dn, m.d_gate, m.d_up, m.d_down))
        assert s.d_x.isnan().all() and m.d_x.isnan().all() and s.d_w.isnan().all()


def test_grads_repeat_and_replay():
    """The same bits again, on another stream, and from a graph that shares its
    workspace with nothing but its own replays, eager work between them."""
    s, other = Experts(333, 320, 6, 3, 224, seed=11), Experts(90, 320, 6, 3, 224, seed=12)
    m = Dense(333, 320, 288, seed=11)
    for v in (s, other, m):
        v.forward()
        v.backward()
    torch.cuda.synchronize()
    want = {**{"e" + k: v.clone() for k, v in s.outputs().items()},
            **{"d" + k: v.clone() for k, v in m.outputs().items()}}

    def same():
        torch.cuda.synchronize()
        now = {**{"e" + k: v for k, v in s.outputs().items()},
               **{"d" + k: v for k, v in m.outputs().items()}}
        return all(torch.equal(now[k], want[k]) for k in want)

    def spoil():
        for v in (*s.outputs().values(), *m.outputs().values()):
            v.fill_(float("nan"))
        s.gws.fill_(255)
        m.gws.fill_(255)
        torch.cuda.synchronize()

    st = torch.cuda.Stream()
    spoil()
    s.backward(st)
    m.backward(st)
    assert same()
    gr = torch.cuda.CUDAGraph()
    note("capture the gated block's backward passes")
    with torch.cuda.graph(gr, stream=st):
        s.backward()
        m.backward()
    for _ in range(4):
        spoil()
        gr.replay()
        assert same()
        other.backward()
        torch.cuda.synchronize()

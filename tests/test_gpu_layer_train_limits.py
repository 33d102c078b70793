"""The layer's training calls at their largest sizes: 65536 tokens, a million slots,
arrays past 2^32 bytes.  Results are held to fp64 at the ends, where an offset cut to 32
bits would land elsewhere."""
import pytest
import torch

from tests import layer_train_ref as ref
from tests.gpu_util import note
from tests.test_gpu_ffn_train import Dense, Experts, close
from tests.test_gpu_grad_norm import call
from tests.test_gpu_norms_train import Norms, holds

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_moe_transformer_router_amd import lib
else:
    lib = None

T = 65536


@pytest.mark.parametrize("slot16", [True, False], ids=["bf16slots", "f32slots"])
def test_experts(slot16):
    """2^20 slots of 2816 columns: 5.9 or 11.8 GB of the slots' parts of d_x."""
    note(f"moe_expert_ffn_grad of {T} tokens x 16, bf16 slots {slot16}")
    s = Experts(T, 2816, 32, 16, 96, seed=21, pad=0.1, drop=0.05,
                slot=lib.MOE_BF16 if slot16 else lib.MOE_F32)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    total = int(s.off[-1])
    at = torch.full((T * s.K,), -1, dtype=torch.int64, device="cuda")  # slot -> row
    at[s.srt[:total].long()] = torch.arange(total, device="cuda")
    rows = [0, 1, T // 2 + 1, T - 2, T - 1, *range(T - 300, T - 200)]
    t = torch.tensor(rows, device="cuda")
    on = s.mask[t].bool()
    v, b = (torch.zeros(len(rows), 2816, dtype=torch.float64, device="cuda") for _ in range(2))
    w, wb = (torch.zeros(len(rows), 16, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(s.E):
        i, k = ((s.idx[t] == e) & on[:, None]).nonzero(as_tuple=True)
        tok = t[i]
        got = ref.group_grad(ref.f64(s.x[tok]), ref.f64(s.gu[e]), ref.f64(s.dn[e]),
                             ref.f64(s.w[tok, k]), ref.f64(s.kept[at[tok * s.K + k]]),
                             ref.f64(s.d_out[tok]), True, True)
        v.index_add_(0, i, got["d_xs"][0])
        b.index_add_(0, i, got["d_xs"][1])
        w[i, k], wb[i, k] = got["d_w"]
    close(s.d_x[t], (v, b + ref.BF16 * (v.abs() + b)), "d_x", True)
    close(s.d_w[t], (w, wb), "d_w", False)
    for e in (0, s.E - 1):
        r = torch.arange(int(s.off[e]), int(s.off[e + 1]), device="cuda")
        slot = s.srt[r].long()
        live = s.mask[slot // s.K].bool()
        r, slot = r[live], slot[live]
        tok = slot // s.K
        got = ref.group_grad(ref.f64(s.x[tok]), ref.f64(s.gu[e]), ref.f64(s.dn[e]),
                             ref.f64(s.w.view(-1)[slot]), ref.f64(s.kept[r]),
                             ref.f64(s.d_out[tok]), True, True)
        close(s.d_gu[e], got["d_gate_up"], "d_gate_up", True)
        close(s.d_dn[e], got["d_down"], "d_down", True)


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_dense(bf16):
    """65536 rows of 32768 projections: 4.3 GB of bf16, 8.6 of fp32."""
    note(f"gemma4_dense_mlp_grad of {T} tokens, width 16384, bf16={bf16}")
    s = Dense(T, 64, 16384, bf16=bf16, seed=22, pad=0.1)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    on = s.mask.bool()
    t = on.nonzero()[:, 0]
    one = torch.ones(t.numel(), dtype=torch.float64, device="cuda")
    for c in (slice(0, 64), slice(16384 - 64, 16384)):
        both = torch.cat([s.kept[t, c], s.kept[t, 16384 + c.start:16384 + c.stop]], 1)
        got = ref.group_grad(ref.f64(s.x[t]), ref.f64(torch.cat([s.gate[c], s.up[c]])),
                             ref.f64(s.down[:, c]), one, ref.f64(both), ref.f64(s.d_y[t]), bf16,
                             bf16)
        close(s.d_gate[c], tuple(v[:64] for v in got["d_gate_up"]), "d_gate", bf16)
        close(s.d_up[c], tuple(v[64:] for v in got["d_gate_up"]), "d_up", bf16)
        close(s.d_down[:, c], got["d_down"], "d_down", bf16)
    t = t[-50:]
    got = ref.group_grad(ref.f64(s.x[t]), ref.f64(torch.cat([s.gate, s.up])), ref.f64(s.down),
                         one[:50], ref.f64(s.kept[t]), ref.f64(s.d_y[t]), bf16, bf16)
    close(s.d_x[t], got["d_xs"], "d_x", bf16)
    assert (s.d_x[~on] == 0).all()


@pytest.mark.parametrize("H", [2816, 4160])
def test_norms(H):
    """Many rows a group, in the place of an input as well."""
    note(f"norms' backward passes of {T} tokens of {H}")
    s = Norms(T, H, K=1, seed=23, pad=0.1)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    s.check()
    for name in ("x", "d_out"):
        v = {n: getattr(s, n).clone() for n in ("x", "d_xd", "d_xm", "d_add", "d_out")}
        lib.gemma4_pre_norms_grad(s.d, T, v["x"], s.g[0], s.g[1], s.mask, v["d_xd"], v["d_xm"],
                                  v["d_add"], v["d_out"], s.scalar, v[name], *s.d_pre, s.ws)
        torch.cuda.synchronize()
        assert torch.equal(v[name], s.d_x), name
    holds(s.d_pre[0], s.want()[6], False, "d_pre")


def test_clip():
    """One gradient of 2^32 + 5 elements, a small one behind it."""
    note("clipping of 2^32 + 5 bf16 gradients")
    n = 2 ** 32 + 5
    a = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    a[-1] = 8.0
    b = torch.full((7,), 4.0, device="cuda")
    want = ((n - 1) * 0.25 + 64 + 7 * 16) ** 0.5
    norm = call([a, b], want / 4)
    assert abs(float(norm[0]) - want) <= 2.0 ** -23 * want
    assert abs(float(norm[1]) - 0.25) <= 2.0 ** -22
    # 0.125, 2 and 1 to one rounding of the factor and one of the product
    assert (a[:-1] - 0.125).abs().max() <= 0.125 * 2.0 ** -7 and abs(float(a[-1]) - 2) <= 2.0 ** -6
    assert ((b - 1).abs() <= 2.0 ** -21).all()


def test_clip_refuses_outputs_that_overlap():
    a = torch.ones(40, device="cuda")
    norm = torch.ones(2, device="cuda")
    plan = lib.grad_list([a[:16], a[24:]])
    for bad in ([a[4:20], torch.empty(16, device="cuda")], [a[24:], a[:16]],
                [a[:16], torch.empty(16, device="cuda", dtype=torch.bfloat16),
                 ], [a[16:32], torch.empty(16, device="cuda")],
                [a[:8].view(torch.bfloat16), torch.empty(16, device="cuda")]):
        out = lib.grad_list(bad)
        if bad[0].data_ptr() == a.data_ptr() and bad[0].dtype == a.dtype:
            lib.moe_grad_clip(plan, norm, out)  # the first in place, the second elsewhere
            continue
        with pytest.raises(ValueError):
            lib.moe_grad_clip(plan, norm, out)
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens", [100, 300, 1500])
def test_many_experts(tokens):
    """Few rows an expert and more, unevenly: one row tile of an expert or several, gradients
    that the caches do not hold (64 experts, 201 MB of them)."""
    note(f"moe_expert_ffn_grad of {tokens} tokens, 64 experts")
    s = Experts(tokens, 1024, 64, 4, 512, seed=24, pad=0.1, skew=True)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    assert int(s.cnt.max()) > (128 if tokens > 200 else 32)
    s.check()


def test_calls_at_once():
    """The same calls of two sizes on two streams at a time, each with its own workspace:
    the bits of one after another."""
    g = torch.Generator(device="cuda").manual_seed(25)
    sets = []
    for i, (n, st) in enumerate(((700, torch.cuda.Stream()), (90, torch.cuda.Stream()))):
        e, m, v = Experts(n, 320, 6, 3, 224, seed=i), Dense(n, 320, 288, seed=i), Norms(n, 320)
        for s in (e, m, v):
            s.forward()
        grads = [torch.randn(k, generator=g, device="cuda") for k in (5000 * n, 77, 12345)]
        plan, out = lib.grad_list(grads), [torch.empty_like(t) for t in grads]
        sets.append((st, e, m, v, plan, lib.grad_list(out), torch.empty(2, device="cuda"),
                     lib.grad_norm_workspace(plan)))

    def run(st, e, m, v, plan, to, norm, ws):
        for s in (e, m, v):
            s.backward(st)
        lib.moe_grad_norm(plan, 0.5, norm, ws, st)
        lib.moe_grad_clip(plan, norm, to, st)

    def results(st, e, m, v, plan, to, norm, ws):
        return [*e.outputs().values(), *m.outputs().values(), *v.results(), *to.tensors, norm]

    torch.cuda.synchronize()
    want = []
    for s in sets:
        run(*s)
        torch.cuda.synchronize()
        want.append([t.clone() for t in results(*s)])
    for _ in range(5):
        for s in sets:
            for t in results(*s):
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        note("training calls on two streams at once")
        for _ in range(3):
            for s in sets:
                run(*s)
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            assert all(torch.equal(a, b) for a, b in zip(results(*s), w))

"""Router backward over many tokens, by the root mean square of its error: the bound of
the other tests grows with the tokens as the gradient does not, and a chain that loses
a step of them stays inside it.  (tests/test_router_grad_rms.py shows that one step
lost exceeds this limit.)"""
import pytest

from tests import router_train_ref as ref
from tests import test_gpu_router_train as base
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,E,K", [(65536, 192, 16, 2), (65536, 64, 7, 2), (5000, 2816, 128, 8),
                                     (2003, 2816, 200, 8), (3001, 1408, 60, 4),
                                     (1000, 2816, 128, 8), (301, 512, 130, 8)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("kind", ["none", "some"])
def test_router_grad_rms(T, H, E, K, bf16, kind):
    c = base._router_case(T, H, E, K, bf16, True, True, True, kind, T + H)
    note(f"router grad, RMS, T={T} H={H} E={E} bf16={bf16} mask={kind}")
    got = base._run_router_grad(c, bf16, spoil=kind == "some")
    want, _ = ref.router_grad(*[ref.f64(c[k]) for k in ("x", "W", "scale", "pes", "gain")],
                              c["idx"], c["mask"], ref.f64(c["d_w"]), ref.f64(c["d_l"]), base.EPS,
                              1)
    for k, v in got.items():
        err = ref.rms_error(v, want[k])
        note(f"  {k} {err:.2e}")
        assert err <= (ref.GRAD_RMS_BF16 if bf16 and k == "x" else ref.GRAD_RMS), (k, err)

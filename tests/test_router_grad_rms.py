"""The limit that the GPU tests of the router's backward hold its RMS error to sees a
lost step of tokens.  On the CPU, in the 64-bit reference."""
import pytest
import torch

from tests import router_train_ref as ref
from tests import test_gpu_router_train as base


@pytest.mark.parametrize("T,H,E,K", [(65536, 192, 16, 2), (5000, 256, 60, 4)])
def test_a_lost_step_exceeds_the_limit(T, H, E, K):
    """32 tokens that add nothing, in one place or repeated from another."""
    c = base._router_case(T, H, E, K, True, True, True, True, "none", T + H)
    a = [ref.f64(c[k]) for k in ("x", "W", "scale", "pes", "gain")]

    def grads(mask):
        return ref.router_grad(*a, c["idx"], mask, ref.f64(c["d_w"]), ref.f64(c["d_l"]), base.EPS,
                               1)[0]
    want = grads(None)
    lost = torch.ones(T, dtype=torch.uint8)
    lost[-32:] = 0
    part = grads(lost)
    for k in ("W", "scale", "pes", "gain"):
        assert ref.rms_error(part[k], want[k]) > 100 * ref.GRAD_RMS, k
        twice = want[k] + (want[k] - part[k])
        assert ref.rms_error(twice, want[k]) > 100 * ref.GRAD_RMS, k
    # and a token's row of d_x
    x = want["x"].clone()
    x[T // 2] = 0
    assert ref.rms_error(x, want["x"]) > 100 * ref.GRAD_RMS

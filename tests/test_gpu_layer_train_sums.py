"""Sums of the layer's training step that one call alone does not show: the second
pre-norm's gain, whose gradient has two parts."""
import pytest
import torch

from tests.gpu_util import F32_TOL, note, rel_max_err
from tests.test_gpu_layer_step import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 150])
def test_second_pre_norms_gain_has_two_parts(T):
    """g_pre2 feeds the experts and the router: its gradient is gemma4_pre_norms_grad's
    d_g_pre2 plus moe_router_grad's d_pre_norm_gain, neither of them alone."""
    s = Layer(T, 50 + T, False)
    note(f"gradient of the second pre-norm's gain, T={T}")
    s.run()
    torch.cuda.synchronize()
    want = s.want()["g_pre2"].numpy()
    both = s.g["g_pre2"].cpu()
    router = s.g2_router.cpu()
    assert rel_max_err(both.numpy(), want) <= F32_TOL
    for part in (router, both - router):
        assert rel_max_err(part.numpy(), want) > 100 * F32_TOL

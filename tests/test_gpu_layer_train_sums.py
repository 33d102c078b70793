"""Sums of the layer's training step that one call alone does not show: the second
pre-norm's gain, whose gradient has two parts, the clipped gradients of a whole step, and a
gradient that a list names twice."""
import ctypes
import math

import pytest
import torch

from tests.gpu_util import F32_TOL, note, rel_max_err
from tests.test_gpu_layer_step import Layer

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_moe_transformer_router_amd import lib
else:
    lib = None


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


@pytest.mark.parametrize("bf16", [False, True], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [5, 150, 700])
def test_clipped_gradients_of_a_step(T, bf16):
    """Each clipped value against its gradient times the factor: off by half a step of its
    type and the product's rounding, relative to itself (below the smallest normal number
    half a step of the subnormal ones)."""
    s = Layer(T, T, bf16)
    note(f"clipped gradients of a step, T={T} bf16={bf16}")
    s.run()
    torch.cuda.synchronize()
    norm = math.sqrt(sum(float(v.double().square().sum()) for v in s.grads.tensors))
    coef = min(1.0, 1.0 / (norm + 1e-6))
    assert coef < 0.9  # it clips
    assert abs(float(s.norm[1]) - coef) <= 4 * 2.0 ** -24 * coef
    for a, b in zip(s.clipped, s.grads.tensors):
        e = b.double() * float(s.norm[1])
        half = torch.finfo(a.dtype).eps / 2
        assert ((a.double() - e).abs()
                <= (1.01 * half + 2.0 ** -24) * e.abs() + 2.0 ** -134).all()
    total = math.sqrt(sum(float(v.double().square().sum()) for v in s.clipped))
    # at most a rounding of the norm, the quotient and each value
    assert abs(total - 1.0) <= (2.0 ** -8 if bf16 else 1e-6)


def test_a_gradient_listed_twice_counts_twice():
    """moe_grad_norm itself takes such a list (the binding's lists hold a tensor once)."""
    a = torch.randn(5000, device="cuda")
    b = torch.randn(33, device="cuda").bfloat16()
    t = (lib.MoeTensor * 3)((a.data_ptr(), a.numel(), lib.MOE_F32),
                            (b.data_ptr(), b.numel(), lib.MOE_BF16),
                            (a.data_ptr(), a.numel(), lib.MOE_F32))
    L = lib.raw()
    norm = torch.empty(2, device="cuda")
    ws = torch.empty(L.moe_grad_norm_workspace_size(3, t), dtype=torch.uint8, device="cuda")
    note("norm of a list that names a gradient twice")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert L.moe_grad_norm(3, t, 1.0, norm.data_ptr(), ws.data_ptr(), ws.numel(),
                           stream) == lib.MOE_OK
    torch.cuda.synchronize()
    want = math.sqrt(2 * float(a.double().square().sum()) + float(b.double().square().sum()))
    assert abs(float(norm[0]) - want) <= 1.01 * 2.0 ** -24 * want

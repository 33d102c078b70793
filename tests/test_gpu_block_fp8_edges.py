"""Block-scaled E4M3 experts where a scale leaves the normal numbers."""
import pytest
import torch

from tests import b128_ref as ref
from tests import test_gpu_block_fp8 as base
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


def tiny_h_case(T, seed, H=128, I=96):
    """Experts whose h is exact in fp32 and whose scale 1/s would overflow in fp32:
    gate 32 everywhere (where GELU is the identity), up small multiples of 2^-133
    in columns 32 .. I - 1 and zero before that.  Value 0 of a row of x, which no
    weight reads, makes x's scale one; down's scales bring y back to about one.
    Returns x, gate_up and down codes and scales, and h in fp64."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(0, 2, (T, H), generator=g).float() * 2 - 1
    x[:, 0], x[:, 1] = 448.0, 1.0
    up = torch.randint(-2, 3, (2, I, H), generator=g).float() * 0.5
    up[..., :2] = 0
    up[:, :32] = 0
    gate = torch.zeros(2, I, H)
    gate[..., 1] = 32.0
    guq = torch.cat([gate, up], 1).to(torch.float8_e4m3fn).view(torch.uint8)
    gus = torch.ones(2, ref.blocks(2 * I), ref.blocks(H))
    gus[:, 1:] = 2.0 ** -132          # rows 128 on: up's from column 32 on
    dn = (torch.randn(2, H, I, generator=g) * 64).clamp(-448, 448)
    dnq = dn.to(torch.float8_e4m3fn).view(torch.uint8)
    dns = torch.full((2, ref.blocks(H), 1), 2.0 ** 110)
    return x, guq, gus, dnq, dns, up


@pytest.mark.parametrize("T", [3, 40, 300, 1000])
def test_tiny_h_is_quantized_by_the_rule(T):
    """h's largest magnitude in a block below 448 * 2^-128: its zeros keep code 0, the
    columns past the last among them, and the others the code nearest to the
    quotient, streamed (up to 256 tokens) and tiled."""
    x, guq, gus, dnq, dns, up = tiny_h_case(T, T)
    g = torch.Generator().manual_seed(T + 1)
    idx, w = torch.randint(0, 2, (T, 1), generator=g), torch.ones(T, 1)
    xv = ref.values(*ref.quantize(x, 1), 1)
    assert torch.equal(xv[:, 1:], x[:, 1:].double())
    u = torch.einsum("eih,th->tei", up.double(), xv) * 2.0 ** -132
    h = (32.0 * u)[torch.arange(T), idx[:, 0]]
    assert torch.equal(h.float().double(), h) and bool((h == 0).any())
    q, s = ref.quantize(h.float(), 1)
    assert torch.all((s > 0) & (s < 2.0 ** -128))
    hv = ref.values(q, s, 1)
    dv = ref.values(dnq, dns, 128)[idx[:, 0]]
    want = torch.einsum("thi,ti->th", dv, hv)
    mag = torch.einsum("thi,ti->th", dv.abs(), hv.abs())
    note(f"experts_b128, subnormal scales of h, T={T}")
    y, _ = base._experts(x, guq, gus, dnq, dns, idx, w)
    # one block: the down product's 128 terms, its scaling, nothing else
    tol = (ref.ACC_REL + 4 * 2.0 ** -24) * mag
    err = (y[:, 0].double() - want).abs()
    assert torch.all(err <= tol), float((err / tol.clamp(min=1e-300)).max())

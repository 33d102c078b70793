"""What the 8-bit matrix instruction makes of a block's 128 products, in the tiled
product: of every eight consecutive ones each is cut (toward zero) below 2^-13 of the
largest power of two that the exponents of the eight pairs of codes give, a code below
2^-6 counting as 2^-6; what is left adds up to fp32."""
import pytest
import torch

from tests import b128_ref as ref
from tests import test_gpu_block_fp8 as base
from tests.gpu_util import note

CUT = 13  # bits below the group's largest exponent that a product keeps


def cut_sums(xq, wq):
    """Codes [t, K], [n, K] -> per block of 128: the sums of the cut products, of the
    products, of their magnitudes, and the bound of what the cuts take, [t, n, KB]."""
    def parts(c):
        c = torch.nn.functional.pad(c, (0, ref.blocks(c.shape[1]) * 128 - c.shape[1]))
        e = ((c >> 3) & 15).clamp(min=1).double() - 7
        return c.view(torch.float8_e4m3fn).double(), e
    (xv, xe), (wv, we) = parts(xq), parts(wq)
    p = (xv[:, None] * wv[None]).unflatten(-1, (-1, 16, 8))
    e = (xe[:, None] + we[None]).unflatten(-1, (-1, 16, 8))
    e = torch.where(p == 0, torch.full_like(e, -60.0), e).amax(-1, keepdim=True)
    unit = torch.exp2(e - CUT)
    cut = torch.trunc(p / unit) * unit
    add = lambda v: v.sum((-1, -2))  # noqa: E731
    return add(cut), add(p), add(p.abs()), 7 * (unit * (e > -60)).sum((-1, -2))


def spread(g, rows, cols, sigma=2.0):
    """Values over many binades, both signs."""
    n = lambda: torch.randn(rows, cols, generator=g)  # noqa: E731
    return (n() * torch.exp(sigma * n())).bfloat16().float()


def test_the_cut_exceeds_2_to_minus_12_of_the_magnitudes():
    """On the CPU: no multiple of the magnitudes as small as that bounds the cuts."""
    g = torch.Generator().manual_seed(3)
    xq, wq = ref.quantize(spread(g, 256, 128), 1)[0], ref.quantize(spread(g, 256, 128), 128)[0]
    cut, exact, mag, bound = cut_sums(xq, wq)
    assert float(((cut - exact).abs() / mag).max()) > 2.0 ** -12
    assert torch.all((cut - exact).abs() <= bound)


# 128 x 128, 256 x 192 and 256 x 256 tiles
@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", [(1024, 2816, 704), (4096, 2816, 272), (4096, 4096, 512),
                                   (2048, 5632, 128)])
@pytest.mark.parametrize("sigma", [0.0, 2.0])
def test_tiled_sums(T, N, K, sigma):
    g = torch.Generator().manual_seed(T + N + K)
    x = spread(g, T, K, sigma)
    q, s = ref.quantize(spread(g, N, K, sigma), 128)
    note(f"linear_b128, cut sums, T={T} N={N} K={K} sigma={sigma}")
    y = base._linear(x, q, s, torch.float32)
    rows, cols = torch.randperm(T, generator=g)[:40], torch.randperm(N, generator=g)[:150]
    xq, xs = ref.quantize(x[rows], 1)
    cut, exact, mag, bound = cut_sums(xq, q[cols])
    sc = xs.double()[:, None] * s.double()[cols // 128][None]
    got = y[rows][:, cols].double()
    add = lambda v: (v * sc).sum(-1)  # noqa: E731
    # 16 groups added in fp32, each cut below 2^-23 of what is there; scaling and
    # adding the blocks
    fp32 = (2.0 ** -19 + (ref.blocks(K) + 4) * 2.0 ** -24) * add(mag)
    err = (got - add(cut)).abs()
    note(f"  against the cut sums 2^{float((err / add(mag)).max().log2()):.1f} of the magnitudes")
    assert torch.all(err <= fp32)
    assert torch.all((got - add(exact)).abs() <= add(bound) + fp32)


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", [(3, 300, 400), (12, 300, 1520), (60, 704, 2816)])
def test_streamed_sums(T, N, K):
    """Codes widened to bf16: to 2^-20 of the magnitudes, whatever their spread."""
    g = torch.Generator().manual_seed(T + N + K)
    x = spread(g, T, K)
    q, s = ref.quantize(spread(g, N, K), 128)
    note(f"linear_b128, streamed sums, T={T} N={N} K={K}")
    y = base._linear(x, q, s, torch.float32)
    xv, wv = ref.values(*ref.quantize(x, 1), 1), ref.values(q, s, 128)
    mag = xv.abs() @ wv.abs().t()
    err = (y.double() - xv @ wv.t()).abs()
    note(f"  2^{float((err / mag).max().log2()):.1f} of the magnitudes")
    assert torch.all(err <= (2.0 ** -20 + (ref.blocks(K) + 4) * 2.0 ** -24) * mag)

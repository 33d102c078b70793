"""Block-scaled experts by the root mean square of their error, in every form: the
bound of the other tests lets a whole step of h's codes go either way, so a scale that
is wrong by some per cent stays inside it.

Limit 5e-3 of the outputs' RMS: the output's rounding to bf16 and a bf16 slot's are at
most 2^-8, some 1.7e-3 in the root mean square, each; in the tiled form the 8-bit
instruction moves h by some 2e-5 of it, which takes about one code in 2000 to its
neighbour, 2^-3.5 away: 2e-3.  In all 3.2e-3.  A scale off by one per cent is outside."""
import pytest
import torch

from tests import b128_ref as ref
from tests import test_gpu_block_fp8 as base
from tests.gpu_util import note

pytestmark = pytest.mark.gpu


# streamed: quantizers inside and before the products; tiled: down's tiles of 128 rows
# below 192 rows an expert and of 256 from there, at this model's widths too
@pytest.mark.parametrize("T,H,E,K,I,skew", [
    (1, 256, 8, 8, 160, 0.8), (3, 2816, 4, 4, 704, 0.8), (5, 192, 16, 3, 96, 0.8),
    (37, 192, 16, 3, 96, 0.8), (90, 320, 2, 2, 160, 0.8), (200, 512, 128, 8, 64, 0.8),
    (256, 64, 256, 16, 32, 0.8), (4, 8192, 3, 2, 32, 0.8), (20, 64, 4, 2, 3200, 0.8),
    (200, 2816, 3, 3, 704, 0.8), (300, 256, 8, 2, 192, 0.8), (257, 64, 256, 4, 32, 0.8),
    (300, 64, 4, 2, 3200, 0.8), (520, 8192, 2, 1, 288, 0.8), (700, 192, 5, 1, 96, 0.8),
    (1100, 2816, 3, 2, 704, 0.8), (1500, 2816, 6, 2, 704, 2.0), (700, 2816, 8, 2, 704, 2.0)])
def test_experts_rms(T, H, E, K, I, skew):
    g = base._gen(T + H + I)
    x = base._x(g, T, H)
    guq, gus = base._weights(g, E, 2 * I, H, std=1.0 / H ** 0.5)
    dnq, dns = base._weights(g, E, H, I, std=1.0 / I ** 0.5)
    idx, w = base._routing(g, T, E, K, skew)
    for slot in (None, 1):
        note(f"experts_b128, RMS, T={T} H={H} E={E} K={K} I={I} slot={slot}")
        y, out = base._experts(x, guq, gus, dnq, dns, idx, w, slot)
        assert base._check_experts(x, guq, gus, dnq, dns, idx, w, y, out) <= 5e-3
        if slot is None:  # the slots themselves, before any bf16
            want, _ = ref.experts(x, ref.values(guq, gus, 128), ref.values(dnq, dns, 128), idx, w)
            d = y.double().sum(1) - want
            assert float((d ** 2).mean().sqrt() / (want ** 2).mean().sqrt()) <= 4e-3


@pytest.mark.parametrize("T,N,K", [(37, 1003, 1520), (300, 513, 6016), (4096, 2816, 2112),
                                   (1025, 130, 2944), (2500, 65, 64), (640, 2816, 704)])
def test_linear_rms(T, N, K):
    """The sums' own error: 2^-12 of the magnitudes at most is some 2^-16 of them in the
    root mean square, and random sums are at least 2^-5 of their magnitudes here."""
    g = base._gen(T + N + K)
    x = base._x(g, T, K)
    q, s = base._weights(g, N, K)
    note(f"linear_b128, RMS, T={T} N={N} K={K}")
    y = base._linear(x, q, s, torch.float32)
    xv, wv = ref.values(*ref.quantize(x, 1), 1), ref.values(q, s, 128)
    want = xv @ wv.t()
    d = y.double() - want
    err = float((d ** 2).mean().sqrt() / (want ** 2).mean().sqrt())
    note(f"  RMS err / RMS {err:.2e}")
    assert err <= 2.0 ** -11

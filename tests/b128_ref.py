"""E4M3 with one fp32 scale per block of 128, in torch on the CPU: the
quantizer bit for bit, the values, and the experts with the bound of the GPU
path's error."""
from __future__ import annotations

import math

import torch

E4M3_MAX = 448.0
INV_MAX = torch.tensor(1.0 / 448.0, dtype=torch.float32)  # a scale is max |v| times this
# Accumulation error of the 8-bit matrix instruction relative to the sum of the
# magnitudes of the 128 products it adds, for values like those of these tests
# (normal ones: at most 2^-16 of 131072 sums; values spread over many binades
# exceed it: test_gpu_block_fp8_sums.py has the rule).
ACC_REL = 2.0 ** -12
BF16 = 2.0 ** -8  # half a unit in the last place, relative


def blocks(n):
    return (n + 127) // 128


def _tiles(v, block_rows):
    """[..., rows, cols] padded to whole blocks, as [..., RB, block_rows, CB, 128]."""
    rows, cols = v.shape[-2:]
    rb = (rows + block_rows - 1) // block_rows
    p = torch.nn.functional.pad(v, (0, blocks(cols) * 128 - cols, 0, rb * block_rows - rows))
    return p.unflatten(-1, (blocks(cols), 128)).unflatten(-3, (rb, block_rows))


def quantize(v, block_rows):
    """(uint8 codes, fp32 scales) of fp32 v: the scale by the reciprocal of 448,
    the quotients by fp32 division, ties to even."""
    rows, cols = v.shape[-2:]
    t = _tiles(v.float(), block_rows)
    s = t.abs().amax((-3, -1)) * INV_MAX
    d = s[..., :, None, :, None]
    q = torch.where(d > 0, t / torch.where(d > 0, d, torch.ones_like(d)), torch.zeros_like(t))
    q = q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    q = q.view(torch.uint8).flatten(-2).flatten(-3, -2)[..., :rows, :cols].contiguous()
    return q, s.contiguous()


def values(q, s, block_rows):
    """fp64 values of codes."""
    rows, cols = q.shape[-2:]
    full = s.double().repeat_interleave(block_rows, -2)[..., :rows, :]
    full = full.repeat_interleave(128, -1)[..., :cols]
    return q.view(torch.float8_e4m3fn).double() * full


def _e4m3(v):
    return v.clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn).double()


def gelu(z):
    return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))


def experts(x, gu, dn, idx, w):
    """The layer on fp64 weight values gu [E, 2I, H], dn [E, H, I] and bf16 input
    x, and the GPU path's bound (before any rounding of the output).

    The codes of x agree on both sides.  The gate and up sums differ by the
    instruction's accumulation error, h by that and its fp32 evaluation; so an
    element of h lies in an interval [lo, hi], its block's scale in [s-, s+],
    and its quantized magnitude between Q(lo / s+) s- and Q(hi / s-) s+: the
    staircase Q is monotone.  y then moves by |W_d| times the largest distance
    from the exact side's value, plus the down product's accumulation error."""
    T, H = x.shape
    I = gu.shape[1] // 2
    xv = values(*quantize(x, 1), 1)
    out = torch.zeros(T, H, dtype=torch.float64)
    err = torch.zeros(T, H, dtype=torch.float64)
    for e in idx.unique().tolist():
        if not 0 <= e < gu.shape[0]:
            continue
        t, k = (idx == e).nonzero(as_tuple=True)
        a = xv[t]
        g, u = a @ gu[e, :I].t(), a @ gu[e, I:].t()
        ge = ACC_REL * (a.abs() @ gu[e, :I].abs().t()) + 2.0 ** -20 * g.abs()
        ue = ACC_REL * (a.abs() @ gu[e, I:].abs().t()) + 2.0 ** -20 * u.abs()
        h = gelu(g) * u
        # |gelu'| <= 1.13
        he = 1.13 * ge * (u.abs() + ue) + gelu(g).abs() * ue + 1e-6 * h.abs()
        pad = blocks(I) * 128 - I
        m = torch.nn.functional.pad(h.abs(), (0, pad)).unflatten(-1, (-1, 128))
        me = torch.nn.functional.pad(he, (0, pad)).unflatten(-1, (-1, 128))
        rep = lambda v: v.repeat_interleave(128, -1)[:, :I]  # noqa: E731
        s = rep((m.amax(-1).float() * INV_MAX).double())
        s_lo = rep((m - me).clamp(min=0).amax(-1)) / E4M3_MAX * (1 - 2.0 ** -22)
        s_hi = rep((m + me).amax(-1)) / E4M3_MAX * (1 + 2.0 ** -22)
        q = torch.where(s > 0, _e4m3(h / s.clamp(min=1e-300)) * s, torch.zeros_like(h))
        lo = (h.abs() - he).clamp(min=0)
        hi = h.abs() + he
        q_lo = _e4m3(lo / s_hi.clamp(min=1e-300) * (1 - 2.0 ** -22)) * s_lo
        q_hi = _e4m3(hi / s_lo.clamp(min=1e-300) * (1 + 2.0 ** -22)) * s_hi
        d = torch.maximum((q.abs() - q_lo).abs(), (q_hi - q.abs()).abs())
        # an element whose interval reaches 0 may change its sign
        d = torch.where(h.abs() <= he, torch.maximum(d, q.abs() + q_hi), d)
        wk = w[t, k].double()[:, None]
        out.index_add_(0, t, wk * (q @ dn[e].t()))
        err.index_add_(0, t, wk.abs() * (d @ dn[e].abs().t()
                                         + ACC_REL * (q.abs() @ dn[e].abs().t())))
    return out, err * 1.001 + 2.0 ** -18 * out.abs()

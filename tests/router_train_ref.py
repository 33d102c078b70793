"""The router's training step in fp64 torch on the CPU: the balance loss, the
router's outputs as a function of its inputs, and their gradients, with the
magnitudes that bound an fp32 evaluation's error.  Used by the GPU tests and
checked against central differences by the CPU tests."""
from __future__ import annotations

import torch

U32 = 2.0 ** -24  # half a unit in the last place of fp32, relative


def f64(t):
    return None if t is None else t.detach().cpu().double()


def balance(logits, idx, mask, a, b):
    """(total, balance, z, N, counts, mean_p) of fp64 logits; -inf allowed."""
    T, E = logits.shape
    K = idx.shape[1]
    keep = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    rows, ids = logits[keep], idx[keep].long()
    n = rows.shape[0]
    counts = torch.stack([(ids == e).sum() for e in range(E)])
    if n == 0:
        z = torch.zeros((), dtype=torch.float64)
        return z, z, z, 0, counts, torch.zeros(E, dtype=torch.float64)
    some = (rows > -torch.inf).any(-1, keepdim=True)
    safe = torch.where(some, rows, torch.zeros_like(rows))
    p = torch.softmax(safe, -1) * some
    lse = torch.logsumexp(safe, -1, keepdim=True) * some
    mean_p = p.sum(0) / n
    bal = E * (counts.double() / (n * K) * mean_p).sum()
    z = (lse ** 2).sum() / n
    return a * bal + b * z, bal, z, n, counts, mean_p


def balance_grad(logits, idx, mask, a, b, g):
    """Gradient of g * total by differentiation, and sum_j of the magnitudes of
    the terms that each element adds."""
    lg = logits.clone().requires_grad_(True)
    total = balance(lg, idx, mask, a, b)[0]
    d = torch.zeros_like(logits)
    if total.requires_grad:
        d, = torch.autograd.grad(g * total, lg)
        d = torch.nan_to_num(d, nan=0.0)
    _, _, _, n, counts, _ = balance(logits, idx, mask, a, b)
    E, K = logits.shape[1], idx.shape[1]
    keep = torch.ones(len(logits), 1) if mask is None else mask.double()[:, None]
    rows = torch.where(keep.bool().expand_as(logits), logits, torch.zeros_like(logits))
    some = (rows > -torch.inf).any(-1, keepdim=True)
    rows = torch.where(some, rows, torch.zeros_like(rows))
    p = torch.softmax(rows, -1) * keep * some
    f = counts.double() / max(1, n * K)
    lse = torch.logsumexp(rows, -1, keepdim=True).abs()
    mag = p * abs(g) / max(1, n) * (abs(a) * E * (f + (p * f).sum(-1, keepdim=True))
                                    + 2 * abs(b) * lse)
    return torch.where(keep.bool(), d, torch.zeros_like(d)), mag


def router_outputs(x, W, scale, pes, gain, idx, eps):
    """Routing weights (of the given picks) and logits; a pick outside [0, E)
    takes part in nothing."""
    v = x
    if gain is not None:
        v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * gain
    v = v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * scale
    logits = v @ W.t()
    ids = idx.long()
    ok = (ids >= 0) & (ids < W.shape[0])
    safe = ids.clamp(0, W.shape[0] - 1)
    picked = torch.gather(logits, 1, safe).masked_fill(~ok, -torch.inf)
    none = ~ok.any(-1, keepdim=True)
    q = torch.softmax(picked.masked_fill(none, 0.0), -1) * ok
    return q * pes[safe], logits


def router_objective(x, W, scale, pes, gain, idx, mask, d_w, d_l, eps):
    w, logits = router_outputs(x, W, scale, pes, gain, idx, eps)
    on = 1.0 if mask is None else mask.double()[:, None]
    total = 0.0
    if d_w is not None:
        total = total + (w * d_w * on).sum()
    if d_l is not None:
        total = total + (logits * d_l * on).sum()
    return total


def router_grad(x, W, scale, pes, gain, idx, mask, d_w, d_l, eps, n_round):
    """Gradients by differentiation and, beside each, the bound of an fp32
    evaluation whose longest chain of roundings has n_round of them: n_round
    * 2^-24 times the sum of the magnitudes of what is added.  A softmax
    weight's gradient q_k (d_k - sum_j q_j d_j) counts as q_k (|d_k| + sum_j
    q_j |d_j|)."""
    leaf = {"x": x, "W": W, "scale": scale, "pes": pes, "gain": gain}
    leaf = {k: v.clone().requires_grad_(True) for k, v in leaf.items() if v is not None}
    total = router_objective(leaf["x"], leaf["W"], leaf["scale"], leaf["pes"], leaf.get("gain"),
                             idx, mask, d_w, d_l, eps)
    got = dict(zip(leaf, torch.autograd.grad(total, list(leaf.values()), allow_unused=True)))
    got = {k: torch.zeros_like(leaf[k]) if v is None else v for k, v in got.items()}
    # magnitudes
    T, H = x.shape
    E = W.shape[0]
    on = torch.ones(T, 1, dtype=torch.float64) if mask is None else mask.double()[:, None]
    one = torch.ones(H, dtype=torch.float64)
    g = one if gain is None else gain
    r0 = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) if gain is not None \
        else torch.ones(T, 1, dtype=torch.float64)
    v = x * r0 * g
    r = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    w, logits = router_outputs(x, W, scale, torch.ones(E, dtype=torch.float64), gain, idx, eps)
    dl = torch.zeros(T, E, dtype=torch.float64)
    pes_mag = torch.zeros(E, dtype=torch.float64)
    ids = idx.long()
    ok = (ids >= 0) & (ids < E)
    safe = ids.clamp(0, E - 1)
    if d_w is not None:
        d = (d_w * pes[safe]).abs()
        dl.scatter_add_(1, safe, w * (d + (w * d).sum(-1, keepdim=True)) * ok)
        pes_mag.scatter_add_(0, safe.reshape(-1), (w * d_w.abs() * on * ok).reshape(-1))
    if d_l is not None:
        dl = dl + d_l.abs()
    dl = dl * on * r0 * r
    beta = (r0 * r) * (dl * logits.abs()).sum(-1, keepdim=True) / H
    u = n_round * U32
    gmag = dl.t() @ x.abs()
    m = (W.abs() * gmag).sum(0)
    gc = (g * scale).abs()
    tol = {"x": u * (gc * (dl @ W.abs())
                     + x.abs() * beta * (1.0 if gain is None else g * g + eps)),
           "W": u * gmag * gc, "scale": u * g.abs() * m, "pes": u * pes_mag}
    if gain is not None:
        tol["gain"] = u * (scale.abs() * m + g.abs() * (x * x * beta).sum(0))
    return got, tol


def rms_error(got, want):
    """Root mean square of the error over that of the values."""
    want = want.double()
    return float(((got.double() - want) ** 2).mean().sqrt() / (want ** 2).mean().sqrt())


# Limit of rms_error for an fp32 result of the router's backward.  A token's factors
# (norms of H / 512 + 8 roundings each, softmax, D: at most 100 of them together, as
# if all pointed one way) move its terms by 100 * 2^-24 = 6e-6; sums over T tokens add
# their roundings with either sign: a chain of n terms of size s, whose partial sums
# grow as sqrt(k) s, ends with an error near 0.41 n 2^-24 s where the sum is sqrt(n) s,
# 0.41 sqrt(n) 2^-24 of it: for a wave's 512 tokens 6e-7, and the parts' sums add less.
GRAD_RMS = 1e-5
# and of d_x rounded to bf16: half a step, as if every value lost all of it
GRAD_RMS_BF16 = 2.0 ** -8

"""The layer's training step in fp64 torch: the gated block's backward pass from kept
projections, the norms' and the layer's forward pass, the clipping of gradients, with
the magnitudes that bound the kernels' errors.  Used by the GPU tests and checked
against central differences by the CPU tests."""
from __future__ import annotations

import math

import torch

BF16 = 2.0 ** -8   # half a step of bf16, relative
# fp32 sums and function values, relative to the magnitudes that they add up:
# random-sign rounding over a few thousand terms stays below 3e-6 of them
SUM = 1e-5
C = math.sqrt(2.0 / math.pi)


def f64(t):
    return None if t is None else t.detach().double()


def gelu(z):
    return 0.5 * z * (1.0 + torch.tanh(C * (z + 0.044715 * z ** 3)))


def slope(z):
    t = torch.tanh(C * (z + 0.044715 * z ** 3))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * C * (1.0 + 3 * 0.044715 * z * z)


def group_grad(x, gate_up, down, w, kept, d, bf16, store):
    """One group's rows.  x [n,H], gate_up [2I,H], down [H,I], w [n], kept [n,2I],
    d [n,H]: {name: (value, bound)} of d_xs (rows), d_w, d_gate_up, d_down; `store`:
    the weights' gradients are stored in bf16."""
    r = BF16 if bf16 else 0.0
    I = down.shape[1]
    g, u = kept[:, :I], kept[:, I:]
    v, vm = d @ down, d.abs() @ down.abs()
    h = gelu(g) * u
    a = torch.cat([u * slope(g), gelu(g)], -1) * w[:, None]
    d_gu = torch.cat([v, v], -1) * a
    e_gu = r * d_gu.abs() + SUM * torch.cat([vm, vm], -1) * a.abs()
    hw = h * w[:, None]
    out = {"d_w": ((v * h).sum(-1), SUM * (vm * h.abs()).sum(-1))}
    val = d_gu @ gate_up
    err = (e_gu + SUM * d_gu.abs()) @ gate_up.abs()
    out["d_xs"] = (val, err + r * (val.abs() + err))
    s = BF16 if store else 0.0
    val = d_gu.t() @ x
    err = (e_gu + SUM * d_gu.abs()).t() @ x.abs()
    out["d_gate_up"] = (val, err + s * (val.abs() + err) + 1e-30)
    val = d.t() @ hw
    err = d.abs().t() @ ((r + SUM) * hw.abs())
    out["d_down"] = (val, err + s * (val.abs() + err) + 1e-30)
    return out


def experts_grad(x, gate_up, down, w, idx, kept, mask, d_out, bf16, store):
    """All experts: {name: (value, bound)} of d_x, d_w, d_gate_up, d_down.  kept: rows
    in the dispatch's order (by expert, slots ascending); ids outside [0, E) dropped."""
    T, K = idx.shape
    E = gate_up.shape[0]
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device=x.device)  # noqa: E731
    out = {"d_x": [z(*x.shape), z(*x.shape)], "d_w": [z(T, K), z(T, K)],
           "d_gate_up": [z(*gate_up.shape), z(*gate_up.shape)],
           "d_down": [z(*down.shape), z(*down.shape)]}
    on = torch.ones(T, dtype=torch.bool, device=x.device) if mask is None else mask.bool()
    at = 0
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        n = t.numel()
        live = on[t]
        rows = torch.arange(at, at + n, device=x.device)[live]
        at += n
        t, k = t[live], k[live]
        got = group_grad(f64(x[t]), f64(gate_up[e]), f64(down[e]), f64(w[t, k]), f64(kept[rows]),
                         f64(d_out[t]), bf16, store)
        for i in range(2):
            out["d_x"][i].index_add_(0, t, got["d_xs"][i])
            out["d_w"][i][t, k] = got["d_w"][i]
            out["d_gate_up"][i][e] = got["d_gate_up"][i]
            out["d_down"][i][e] = got["d_down"][i]
    if bf16:
        v, b = out["d_x"]
        out["d_x"][1] = b + BF16 * (v.abs() + b)
    return {k: tuple(v) for k, v in out.items()}


def dense_grad(x, gate, up, down, kept, mask, d_y, bf16, store):
    """The dense MLP: {name: (value, bound)} of d_x, d_gate, d_up, d_down."""
    T, H = x.shape
    on = torch.ones(T, dtype=torch.bool, device=x.device) if mask is None else mask.bool()
    t = on.nonzero()[:, 0]
    one = torch.ones(t.numel(), dtype=torch.float64, device=x.device)
    got = group_grad(f64(x[t]), torch.cat([f64(gate), f64(up)]), f64(down), one, f64(kept[t]),
                     f64(d_y[t]), bf16, store)
    out = {}
    out["d_x"] = tuple(torch.zeros(T, H, dtype=torch.float64, device=x.device).index_copy_(
        0, t, v) for v in got["d_xs"])
    D = gate.shape[0]
    out["d_gate"] = tuple(v[:D] for v in got["d_gate_up"])
    out["d_up"] = tuple(v[D:] for v in got["d_gate_up"])
    out["d_down"] = got["d_down"]
    return out


def norm(v, eps):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)


def behind(x, dn, total, g1, g2, g3, scalar, eps):
    return (norm(norm(dn, eps) * g1 + norm(total, eps) * g2, eps) * g3 + x) * scalar


def layer(x, p, idx, eps):
    """The whole dual-path layer with the picks given: (out, logits, weights).  p: a dict
    of fp64 leaves named as the layer's parameters."""
    xd, xm = norm(x, eps) * p["g_pre"], norm(x, eps) * p["g_pre2"]
    logits = (norm(xm, eps) * p["router_scale"]) @ p["router_w"].t()
    ids = idx.long()
    w = torch.softmax(torch.gather(logits, 1, ids), -1) * p["pes"][ids]
    moe = torch.zeros_like(x)
    for e in range(p["gate_up"].shape[0]):
        t, k = (idx == e).nonzero(as_tuple=True)
        z = xm[t] @ p["gate_up"][e].t()
        I = z.shape[1] // 2
        y = (gelu(z[:, :I]) * z[:, I:]) @ p["down"][e].t()
        moe = moe.index_add(0, t, y * w[t, k][:, None])
    dn = (gelu(xd @ p["gate"].t()) * (xd @ p["up"].t())) @ p["dense_down"].t()
    out = behind(x, dn, moe, p["g_post1"], p["g_post2"], p["g_post"], p["scalar"], eps)
    return out, logits, w

"""Router backward where logits are -inf: an expert switched off for a token has
probability and gradient 0."""
import numpy as np
import pytest
import torch

from tests import router_train_ref as ref
from tests import test_gpu_router_train as base
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_moe_transformer_router_amd import lib
else:
    lib = None


def _run(c, lg, bf16):
    """moe_router_grad with the logits given; every gradient, on the CPU."""
    T, H = c["x"].shape
    E, K = c["W"].shape[0], c["idx"].shape[1]
    d = lib.dims(H, E, K, 32, 0, base.EPS, lib.MOE_BF16 if bf16 else lib.MOE_F32)
    ws = lib.workspace(d, T)
    ws.fill_(0xFF)
    dt = torch.bfloat16 if bf16 else torch.float32
    dev = {k: None if v is None else v.cuda() for k, v in c.items()}
    new = lambda *s, t=torch.float32: torch.full(s, np.nan, dtype=t, device="cuda")  # noqa: E731
    out = dict(x=new(T, H, t=dt), W=new(E, H), scale=new(H), pes=new(E),
               gain=new(H) if c["gain"] is not None else None)
    lib.moe_router_grad(d, T, dev["x"].to(dt), dev["W"], dev["scale"], dev["pes"], dev["gain"],
                        lg.cuda(), dev["idx"], dev["mask"], dev["d_w"], dev["d_l"], *out.values(),
                        ws)
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in out.items() if v is not None}


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("T,H,E,K,pre", [(70, 128, 24, 4, True), (70, 128, 24, 4, False),
                                         (300, 704, 130, 8, True)])
@pytest.mark.parametrize("fill", [3.0, float("nan")])
def test_router_grad_switched_off_experts(T, H, E, K, pre, bf16, fill):
    """Logits of -inf at picked and other experts, at every pick of a token, and in a
    whole row; d_logits and d_topk_w hold something there.  As if the gradient there were 0 and
    the picks took part in nothing."""
    c = base._router_case(T, H, E, K, bf16, pre, True, True, "some" if T > 100 else "none", T + pre)
    lg = base._logits(c)
    off = torch.rand(T, E, generator=torch.Generator().manual_seed(T)) < 0.2
    off[3] = False
    off[3, c["idx"][3, 0].long()] = True              # a token's first pick
    off[4] = False
    off[4, c["idx"][4].long()] = True                 # all of its picks
    off[5] = True                                     # every expert
    off[6] = False
    lg[off] = -torch.inf
    want = dict(c)
    picked_off = torch.gather(off, 1, c["idx"].long())
    want["idx"] = torch.where(picked_off, torch.full_like(c["idx"], -1), c["idx"])
    want["d_l"] = torch.where(off, torch.zeros_like(c["d_l"]), c["d_l"])
    want["d_w"] = c["d_w"].clone()
    c["d_l"] = torch.where(off, torch.full_like(c["d_l"], fill), c["d_l"])
    c["d_w"] = torch.where(picked_off, torch.full_like(c["d_w"], fill), c["d_w"])
    note(f"router grad, experts off, T={T} H={H} E={E} bf16={bf16} pre={pre} fill={fill}")
    got = _run(c, lg, bf16)
    assert all(v.isfinite().all() for v in got.values())
    base._check_router_grad(want, got, bf16)
    # a token without experts
    assert not got["x"][5].any()

"""The router's training calls at their largest sizes: of 65536 tokens a few scattered
ones count, so a reference on those alone tells every offset."""
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


@pytest.mark.parametrize("T,H,E,K", [(65536, 8192, 256, 16), (65536, 8192, 128, 16),
                                     (32767, 8192, 255, 32), (1, 8192, 256, 32)])
@pytest.mark.parametrize("bf16", [False, True])
def test_router_grad_at_the_limits(T, H, E, K, bf16):
    note(f"router grad at the limits T={T} H={H} E={E} K={K} bf16={bf16}")
    n = min(T, 60)
    c = base._router_case(n, H, E, K, bf16, True, True, True, "none", T + E)
    g = torch.Generator().manual_seed(T)
    at = torch.randperm(T, generator=g)[:n]
    if T > 1:
        at[0], at[1] = T - 1, T - 2
        at = at.unique()
        n = len(at)
        for k in ("x", "idx", "d_w", "d_l"):
            c[k] = c[k][:n]
    dt = torch.bfloat16 if bf16 else torch.float32
    d = lib.dims(H, E, K, 32, 0, base.EPS, lib.MOE_BF16 if bf16 else lib.MOE_F32)
    ws = lib.workspace(d, T, calls=("router_grad",))
    ws.fill_(0xFF)

    def spread(t, dtype, fill):  # the counted tokens' rows among others'
        out = torch.full((T, t.shape[1]), fill, dtype=dtype, device="cuda")
        out[at.cuda()] = t.to(dtype).cuda()
        return out
    nan = float("nan")
    x, lg = spread(c["x"], dt, nan), spread(base._logits(c), torch.float32, nan)
    idx = spread(c["idx"], torch.int32, 0)
    d_w, d_l = spread(c["d_w"], torch.float32, nan), spread(c["d_l"], torch.float32, nan)
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    mask[at.cuda()] = 1
    new = lambda *s, t=torch.float32: torch.full(s, np.nan, dtype=t, device="cuda")  # noqa: E731
    out = dict(x=new(T, H, t=dt), W=new(E, H), scale=new(H), pes=new(E), gain=new(H))
    p = [c[k].cuda() for k in ("W", "scale", "pes", "gain")]
    lib.moe_router_grad(d, T, x, *p, lg, idx, mask, d_w, d_l, *out.values(), ws)
    torch.cuda.synchronize()
    got = {k: v.cpu() for k, v in out.items() if k != "x"}
    got["x"] = out["x"][at.cuda()].cpu()
    out["x"][at.cuda()] = 0
    assert not out["x"].any()  # NaN counts as true
    base._check_router_grad(c, got, bf16)
    want, _ = ref.router_grad(*[ref.f64(c[k]) for k in ("x", "W", "scale", "pes", "gain")],
                              c["idx"], None, ref.f64(c["d_w"]), ref.f64(c["d_l"]), base.EPS, 1)
    for k, v in got.items():
        err = ref.rms_error(v, want[k])
        assert err <= (ref.GRAD_RMS_BF16 if bf16 and k == "x" else ref.GRAD_RMS), (k, err)


@pytest.mark.parametrize("T,E,K", [(65536, 256, 16), (32768, 255, 32), (16400, 130, 8)])
def test_balance_at_the_limits(T, E, K):
    g = torch.Generator().manual_seed(T)
    lg = (2.0 * torch.randn(T, E, generator=g)).double().float().double()
    idx = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    mask = base._mask(g, T, "some")
    note(f"balance at the limits T={T} E={E} K={K}")
    base._check_balance(lg, idx, mask, base._run_balance(lg, idx, mask, E, K))

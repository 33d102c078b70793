"""moe_router_logits in every form of the router's logits kernels: the logits are the
oracle's bit for bit, the routing is moe_router's."""
import numpy as np
import pytest
import torch

import oracle
from tests.gpu_util import note

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_moe_transformer_router_amd import lib
else:
    lib = None


# one to four tokens a block, four and eight experts (up to 448 tokens); blocks of 16
# tokens, of 32 with four wave groups and with two (E a multiple of 4, by the number of
# blocks); the kernel for other E; a hidden size past the small kernels' limit
@pytest.mark.parametrize("T,H,E,K", [(1, 192, 7, 3), (7, 256, 60, 4), (30, 192, 130, 8),
                                     (448, 320, 128, 8), (449, 320, 128, 8), (2048, 192, 128, 8),
                                     (2049, 192, 128, 8), (4096, 64, 128, 8), (4100, 128, 128, 8),
                                     (65536, 64, 8, 2), (500, 192, 130, 5), (3000, 64, 7, 3),
                                     (3, 8192, 16, 2), (600, 4096, 33, 4)])
@pytest.mark.parametrize("bf16,pre", [(True, True), (True, False), (False, True)])
def test_logits(T, H, E, K, bf16, pre):
    g = torch.Generator().manual_seed(T + H + E)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, W = n(T, H), n(E, H) * (1.5 / H ** 0.5)
    x = x.bfloat16().float() if bf16 else x
    scale, pes, gain = 1 + 0.1 * n(H), 1 + 0.1 * n(E), 1 + 0.1 * n(H) if pre else None
    note(f"router logits T={T} H={H} E={E} bf16={bf16} pre={pre}")
    d = lib.dims(H, E, K, 32, 0, 1e-6, lib.MOE_BF16 if bf16 else lib.MOE_F32)
    ws = lib.workspace(d, T, calls=("layer",))
    ws.fill_(0xFF)
    xd = x.cuda().to(torch.bfloat16 if bf16 else torch.float32)
    args = [None if t is None else t.cuda() for t in (W, scale, pes, gain)]
    idx = [torch.full((T, K), -1, dtype=torch.int32, device="cuda") for _ in range(2)]
    w = [torch.full((T, K), np.nan, device="cuda") for _ in range(2)]
    lg = torch.full((T + 1, E), np.nan, device="cuda")
    lib.moe_router(d, T, xd, *args, idx[0], w[0], ws)
    lib.moe_router_logits(d, T, xd, *args, idx[1], w[1], lg, ws)
    torch.cuda.synchronize()
    assert torch.equal(idx[0], idx[1]) and torch.equal(w[0], w[1])
    oi, _, ol = oracle.router(x.numpy(), W.numpy(), scale.numpy(), pes.numpy(), K, 1e-6,
                              pre_gain=None if gain is None else gain.numpy(), want_logits=True)
    got = lg.cpu().numpy()
    assert np.isnan(got[T]).all()
    assert np.array_equal(got[:T].view(np.uint32), ol.view(np.uint32))
    assert np.array_equal(idx[1].cpu().numpy(), oi)

"""Forms of the gated block's backward pass that its sizes and types choose: fp32 weight
gradients of bf16 weights where a block goes through many large tiles, bf16 slots in every
tile, many experts; against fp64, at the bounds of tests/test_gpu_ffn_train.py."""
import ctypes

import pytest
import torch

from tests.gpu_util import note
from tests.test_gpu_ffn_train import Experts, close

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from sparse_moe_transformer_router_amd import lib
else:
    lib = None

# T, H, E, K, I: more large tiles of the weights' gradients than CUs, of either or both
MANY_TILES = [
    (300, 320, 200, 4, 64),    # 400 of each, partial, 49 MB of fp32
    (700, 576, 50, 3, 160),    # 300 and 150, 55 MB
    (300, 1024, 64, 4, 512),   # 1024 and 512, 402 MB: past the caches
    (1500, 1024, 64, 4, 512),
]


def run(s):
    s.forward()
    s.backward()
    torch.cuda.synchronize()


@pytest.mark.parametrize("size", MANY_TILES, ids=str)
def test_fp32_weight_gradients_of_many_tiles(size):
    """Experts without rows, with a few and with several k-tiles in one block's stream; the
    fp32 sums are those that the bf16 store rounds, bit for bit."""
    note(f"moe_expert_ffn_grad, fp32 weight gradients {size}")
    s = Experts(*size, seed=31, pad=0.1, skew=True, store=False)
    run(s)
    s.check()
    t = Experts(*size, seed=31, pad=0.1, skew=True)
    run(t)
    assert torch.equal(s.d_gu.bfloat16(), t.d_gu) and torch.equal(s.d_dn.bfloat16(), t.d_dn)
    assert torch.equal(s.d_x, t.d_x) and torch.equal(s.d_w, t.d_w)


@pytest.mark.parametrize("size", [
    (1, 64, 1, 1, 32),
    (1, 2816, 8, 8, 704),
    (64, 2816, 16, 4, 704),    # large tiles, up to 32 rows an expert: weights read once
    (300, 320, 6, 3, 224),     # small tiles
    (700, 576, 3, 2, 288),
    (900, 2816, 3, 2, 704),    # large tiles, many rows an expert
    (40, 192, 12, 12, 64),
    (33, 64, 3, 2, 8192),
    (40, 8192, 4, 2, 160),
], ids=str)
def test_bf16_slots(size):
    note(f"moe_expert_ffn_grad, bf16 slots {size}")
    s = Experts(*size, seed=32, slot=lib.MOE_BF16)
    run(s)
    s.check()


@pytest.mark.parametrize("tokens", [100, 300, 1500])
def test_bf16_slots_of_many_experts(tokens):
    note(f"moe_expert_ffn_grad, bf16 slots, {tokens} tokens, 64 experts")
    s = Experts(tokens, 1024, 64, 4, 512, seed=33, pad=0.1, skew=True, slot=lib.MOE_BF16)
    run(s)
    s.check()


@pytest.mark.parametrize("size", [(200, 320, 24, 3, 96), (200, 2816, 24, 3, 96),
                                  (1100, 2816, 24, 3, 96)], ids=str)
@pytest.mark.parametrize("slot16", [True, False], ids=["bf16slots", "f32slots"])
def test_slots_dropped_masked_and_empty(size, slot16):
    """Slots that the dispatch dropped, tokens that do not count with NaN in their rows,
    experts without rows: in small tiles, in large ones that read the weights once and in
    those that keep them."""
    note(f"moe_expert_ffn_grad dropped, masked, empty {size} bf16 slots {slot16}")
    s = Experts(*size, seed=34, pad=0.3, drop=0.2, skew=True,
                slot=lib.MOE_BF16 if slot16 else lib.MOE_F32)
    # the last experts are nobody's
    s.idx[s.idx >= s.E - 3] = -1
    lib.moe_dispatch(s.d, s.T, s.idx, s.cnt, s.off, s.srt, s.ws)
    s.forward()
    off = s.mask == 0
    want = s.want()
    s.x[off] = float("nan")
    s.d_out[off] = float("nan")
    s.w[off] = float("nan")
    rows = s.srt[:int(s.off[-1])].long() // s.K
    s.kept[:rows.numel()][off[rows]] = float("nan")
    s.backward()
    torch.cuda.synchronize()
    for k, v in s.outputs().items():
        close(v, want[k], k, k != "d_w")
    assert (s.d_x[off] == 0).all() and (s.d_w[off] == 0).all() and (s.d_w[s.idx < 0] == 0).all()
    assert (s.d_gu[-3:] == 0).all() and (s.d_dn[-3:] == 0).all()


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
@pytest.mark.parametrize("E", [65, 129, 256])
def test_experts_past_a_wave(E, bf16):
    """More experts than a wave has lanes: two to four to a lane in the kernels' scans."""
    note(f"moe_expert_ffn_grad, {E} experts, bf16={bf16}")
    s = Experts(150, 128, E, 5, 32, bf16=bf16, seed=E, pad=0.1, skew=True)
    run(s)
    assert int((s.cnt == 0).sum()) > 0
    s.check()


def test_the_same_bits_again():
    """Every form of the weights' gradients and of d_x, ten times over."""
    for size, kw in (((300, 1024, 64, 4, 512), dict(store=False)),
                     ((100, 1024, 64, 4, 512), dict(slot=1)),
                     ((1500, 1024, 64, 4, 512), dict(slot=1)),
                     ((300, 320, 6, 3, 224), dict(slot=1))):
        s = Experts(*size, seed=35, pad=0.1, skew=True, **kw)
        note(f"moe_expert_ffn_grad again {size} {kw}")
        run(s)
        want = {k: v.clone() for k, v in s.outputs().items()}
        for _ in range(10):
            for v in s.outputs().values():
                v.fill_(float("nan"))
            s.gws.fill_(255)
            s.backward()
            torch.cuda.synchronize()
            assert all(torch.equal(v, want[k]) for k, v in s.outputs().items())


@pytest.mark.parametrize("bf16", [True, False], ids=["bf16", "f32"])
def test_no_tokens_and_no_inputs(bf16):
    """T = 0 through the library's own calls, every input NULL: the gradients of what sums
    over tokens are zeros."""
    L, t = lib.raw(), lib.MOE_BF16 if bf16 else lib.MOE_F32
    d = ctypes.byref(lib.dims(128, 5, 2, 96, 64, 1e-6, t, lib.MOE_F32))
    nan = lambda *s: torch.full(s, float("nan"), device="cuda")  # noqa: E731
    gu, dn, gate, up, down = nan(5, 192, 128), nan(5, 128, 96), nan(64, 128), nan(64, 128), \
        nan(128, 64)
    g = [nan(128) for _ in range(5)]
    scalar = nan(1)
    p = lambda v: v.data_ptr()  # noqa: E731
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    note(f"no tokens, no inputs, bf16={bf16}")
    assert L.moe_expert_ffn_grad(d, 0, *[None] * 11, lib.MOE_F32, p(gu), p(dn), None, 0,
                                 stream) == lib.MOE_OK
    assert L.gemma4_dense_mlp_grad(d, 0, *[None] * 8, lib.MOE_F32, p(gate), p(up), p(down), None,
                                   0, stream) == lib.MOE_OK
    assert L.gemma4_post_norms_grad(d, 0, *[None] * 6, 0.5, *[None] * 4, p(g[0]), p(g[1]), p(g[2]),
                                    p(scalar), None, 0, stream) == lib.MOE_OK
    assert L.gemma4_pre_norms_grad(d, 0, *[None] * 8, 0.5, None, p(g[3]), p(g[4]), None, 0,
                                   stream) == lib.MOE_OK
    torch.cuda.synchronize()
    assert all((v == 0).all() for v in (gu, dn, gate, up, down, *g, scalar))

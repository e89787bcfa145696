"""Waits of the router's product that give up, without a GPU fault: with the bound far
below what they take (W4A16_WAIT_TIMEOUT_CYCLES) they run out, the kernel ends
behind its copies and MMAs, and logits that waited are NaN."""

import pytest
import torch

from helpers import Guarded
from w4a16_int4_moe_gb300 import ops

pytestmark = pytest.mark.gpu

# (tokens, experts, hidden): pairs of CTAs, alone and with the columns split, and single CTAs
SIZES = [(8192, 384, 7168), (4096, 384, 7168), (8192, 256, 2048), (2000, 128, 7168),
         (777, 384, 7168), (777, 60, 2088), (300, 256, 1024), (100, 384, 7168), (2000, 17, 520)]


@pytest.mark.parametrize("tokens,experts,hidden", SIZES)
def test_waits_that_give_up(cuda_dev, monkeypatch, tokens, experts, hidden):
    gen = torch.Generator(device=cuda_dev).manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=gen, device=cuda_dev).to(torch.bfloat16)
    w = torch.randn(experts, hidden, generator=gen, device=cuda_dev).to(torch.bfloat16)
    want = ops.w4a16_router_logits(x, w)
    other = ops.w4a16_router_logits(-2 * x, w)
    out = Guarded((tokens, experts), torch.float32, cuda_dev)
    for limit in (1, 500, 3000, 10000):
        out.t.copy_(other)
        monkeypatch.setenv("W4A16_WAIT_TIMEOUT_CYCLES", str(limit))
        ops.w4a16_router_logits(x, w, out=out.t)
        monkeypatch.delenv("W4A16_WAIT_TIMEOUT_CYCLES")
        again = ops.w4a16_router_logits(x, w)   # right behind it, on the same SMs
        out.check(f"limit {limit}")
        gone = torch.isnan(out.t)
        assert not (~gone & (out.t != want)).any(), (limit, int(gone.sum()))
        assert torch.equal(again, want)
        # (a wait is suspended for up to some thousand cycles before the bound counts, so
        # that in a small product, whose operands are in L2, all may come in time)
        if limit == 1 and tokens * hidden >= 1 << 22:
            assert gone.any()

"""Waits of the products' kernels that give up, without a GPU fault.

Every wait on a copy, an accumulator or a slot is bounded. With the bound far below
the time that such a wait takes (W4A16_WAIT_TIMEOUT_CYCLES) it runs out: the kernel
leaves out the rest of its work, lets the copies and MMAs that it has in flight
finish and ends, and the next call runs as if nothing had been."""

import pytest
import torch

from helpers import Guarded
from test_gpu_products import Dense, Int4, _rows

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# (kind, tokens, n, k, gated, f32): CTA pairs that go over several tiles each, with one
# and with several accumulators a tile; clusters that split the columns; the packed
# weight's tcgen05 kernel, with blocks that come round again.
CASES = [(Dense, 8192, 7168, 2048, False, True), (Dense, 8192, 4096, 1096, True, False),
         (Dense, 5000, 7168, 64, False, False),
         (Dense, 100, 2002, 2088, True, False), (Dense, 200, 1000, 7168, False, True),
         (Int4, 20, 20001, 1568, False, True), (Int4, 32, 39168, 1056, True, False)]


def _case(dev, kind, tokens, n, k, gated, f32):
    weight = kind(dev, n, k, gated)
    weight.w = weight.loose = None   # (not compared with the 64-bit form here)
    x = _rows(torch.Generator(device=dev).manual_seed(1), tokens, k, 0, dev)
    dtype = F32 if f32 else BF
    out = Guarded((tokens, n // 2 if gated else n), dtype, dev)
    return weight, x, weight(x, out_dtype=dtype), out


@pytest.mark.parametrize("kind,tokens,n,k,gated,f32", CASES)
def test_waits_that_give_up_end_the_call_in_order(cuda_dev, monkeypatch, kind, tokens, n, k, gated,
                                                  f32):
    weight, x, want, out = _case(cuda_dev, kind, tokens, n, k, gated, f32)
    for limit in (1, 500, 3000, 10000):
        monkeypatch.setenv("W4A16_WAIT_TIMEOUT_CYCLES", str(limit))
        weight(x, out=out.t)
        monkeypatch.delenv("W4A16_WAIT_TIMEOUT_CYCLES")
        again = weight(x, out_dtype=want.dtype)   # right behind it, on the same SMs
        out.check(f"limit {limit}")
        assert torch.equal(again, want)


@pytest.mark.parametrize("kind,tokens,n,k,gated,f32", CASES)
def test_outputs_are_nan_once_a_wait_gave_up(cuda_dev, monkeypatch, kind, tokens, n, k, gated, f32):
    # (the accumulators hold sums of other calls by then, which must not come out)
    weight, x, want, out = _case(cuda_dev, kind, tokens, n, k, gated, f32)
    other = weight(-2 * x, out_dtype=want.dtype)
    for limit in (1, 500, 3000, 10000):
        out.t.copy_(other)
        monkeypatch.setenv("W4A16_WAIT_TIMEOUT_CYCLES", str(limit))
        weight(x, out=out.t)
        monkeypatch.delenv("W4A16_WAIT_TIMEOUT_CYCLES")
        gone = torch.isnan(out.t)
        wrong = ~gone & (out.t != want)
        assert not wrong.any(), (limit, int(wrong.sum()), int(gone.sum()), out.t.numel())
        if limit == 1:
            assert gone.any()

"""How far the products' sums are off, as a whole: bounds of single outputs allow for
every rounding in the same direction, which hides a mechanism that has stopped
working (a weight rounded to BF16, a tensor core's sum that is never taken over).

A sum that a tensor core keeps is cut off at every addition, by half a step of 2^-24
on average: after A additions in a row that is about 1e-8 A of the result."""

import math

import pytest
import torch

import product_reference as ref
from test_gpu_products import Dense, Int4, _rows

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


# BF16 results: an FP32 error e moves an output over a border between two BF16 numbers with
# the probability |e| / step, by a step, at most 2^-7 of it: off by sqrt(0.8 * 2^-7 * e)
# (0.8: a normal error's mean size). 4e-6 is a product of 1024 columns' accumulators
# (64 additions, 6e-7), thrice for silu(gate) * up, with half of it to spare; one
# accumulator for all of 7168 columns is 5e-6 a factor, for 65536 5e-5.
@pytest.mark.parametrize("tokens,n,k,gated", [(64, 4096, 7168, True), (576, 4096, 7168, True),
                                              (2048, 4096, 7168, True), (576, 512, 65536, False),
                                              (100, 512, 65536, False)])
def test_bf16_results_are_the_rounded_sums(cuda_dev, tokens, n, k, gated):
    weight = Dense(cuda_dev, n, k, gated, 3)
    x = _rows(torch.Generator(device=cuda_dev).manual_seed(4), tokens, k, 0, cuda_dev)
    if not gated:   # all of one sign: the cut-off parts add up
        weight.bits, x = weight.bits.abs(), x.abs()
        weight.w = weight.bits.double()
    want = ref.product(x, weight.w, None, gated, None)[0].float().to(BF).double()
    assert _off(weight(x), want) < math.sqrt(0.8 * 2.0 ** -7 * 4e-6)


# FP32 results. Up to 32 tokens a step's 64 columns, INT4 a group's 32, are four or two
# additions in the tensor core, 4e-8; their sums are rounded FP32 additions, at most 128
# in a row here, 3e-8 sqrt(128) / 2 = 1.7e-7. Left in the tensor core the 56 additions of
# a warp's share of 7168 columns are 6e-7 and more.
@pytest.mark.parametrize("kind", [Dense, Int4])
@pytest.mark.parametrize("tokens,n,k", [(1, 4096, 7168), (8, 7168, 2048), (16, 4096, 7168),
                                        (32, 4096, 7168), (32, 512, 65536), (3, 512, 65536),
                                        (32, 16384, 7168)])
def test_fp32_results_of_few_tokens(cuda_dev, kind, tokens, n, k):
    weight = kind(cuda_dev, n, k, False, 5)
    x = _rows(torch.Generator(device=cuda_dev).manual_seed(6), tokens, k, 0, cuda_dev)
    assert _off(weight(x, out_dtype=F32), x.double() @ weight.w.t()) < 4e-7


# More tokens: 32 additions in the tensor core, 3e-7, and half as much again for the sums
# of 512 columns each; 128 and more in a row would be 1.5e-6 and more.
@pytest.mark.parametrize("tokens,n,k", [(64, 4096, 7168), (200, 1000, 2048), (576, 7168, 2048),
                                        (576, 4096, 7168), (4096, 7168, 2048), (100, 512, 65536)])
def test_fp32_results_of_many_tokens(cuda_dev, tokens, n, k):
    weight = Dense(cuda_dev, n, k, False, 7)
    x = _rows(torch.Generator(device=cuda_dev).manual_seed(8), tokens, k, 0, cuda_dev)
    assert _off(weight(x, out_dtype=F32), x.double() @ weight.w.t()) < 1e-6


def test_a_rounded_weight_would_be_seen(cuda_dev):
    # the limit against the mistake: the INT4 weight's products rounded to BF16
    weight = Int4(cuda_dev, 512, 7168, False, 9)
    x = _rows(torch.Generator(device=cuda_dev).manual_seed(10), 32, 7168, 0, cuda_dev).double()
    assert _off(x @ weight.w.to(BF).double().t(), x @ weight.w.t()) > 1e-4

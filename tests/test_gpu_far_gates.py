"""Gated products whose gates are as far out as FP32's exponential, with ups so large
that the result is not small: silu(g) is -1e-36 where e^-g is past FP32's range."""

import pytest
import torch

import product_reference as ref
from w4a16_int4_moe_gb300 import ops

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
GLU = ops.W4A16_LAYOUT_KTILE64_GLU16


def _gates_and_ups(dev, columns):
    gate = torch.cat([torch.linspace(-89.5, -86.5, columns // 2, device=dev),
                      torch.linspace(-115, 20, columns - columns // 2, device=dev)]).to(BF)
    up = (2.0 ** (40 + torch.arange(columns, device=dev) % 32)).to(BF)
    return gate, up


def _check(out, gate, up):
    # Steps of 2^-23, from the units in the last place that CUDA states for each
    # operation: the exponential 1; its square, one more and the sum 1.75; the division
    # 2; gate and up times the exponential 1.5 each; the last product 0.5. A result
    # below FP32's normal range is off by a step of its own besides. Where the result is
    # rounded to BF16 and the gate is at least -80, 2^-16: the exponent is at most 116
    # and rounded once, and its factor to 2^-26: 116 * (2^-24 + 2^-26) * ln 2 = 2^-17.3;
    # exponential, sum, reciprocal and two products take 2^-21.
    g, u = gate.double(), up.double()
    want = (g * torch.sigmoid(g) * u).expand(out.shape[0], -1)
    bound = 8 * ref.STEP * want.abs() + 2.0 ** -149
    if out.dtype is BF:
        bound = torch.where(g < -80, bound, 2.0 ** -16 * want.abs())
        # (below its normal range BF16's steps are 2^-133, and a rounding half of one)
        bound = bound + (want.abs() + bound) * ref.BF16_HALF + 2.0 ** -134
    ref.assert_within(out, want, bound)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens,columns", [(1, 300), (32, 300), (33, 300), (200, 1001), (600, 4096),
                                            (4096, 4096)])
def test_dense(cuda_dev, dtype, tokens, columns):
    gate, up = _gates_and_ups(cuda_dev, columns)
    weight = torch.zeros(2 * columns, 72, dtype=BF, device=cuda_dev)
    weight[:columns, 3], weight[columns:, 3] = gate, up
    x = torch.zeros(tokens, 72, dtype=BF, device=cuda_dev)
    x[:, 3] = 1
    _check(ops.w4a16_dense(x, weight, gated=True, out_dtype=dtype), gate, up)


def test_whole_tiles_of_near_and_of_far_gates(cuda_dev):
    # each 64 columns in another range, so that some warps have no far gate and some only such
    columns = 4096
    gate = torch.cat([torch.linspace(a, a + 16, 64, device=cuda_dev)
                      for a in range(-140, 116, 4)]).to(BF)
    up = (2.0 ** (20 + torch.arange(columns, device=cuda_dev) % 32)).to(BF)
    weight = torch.zeros(2 * columns, 72, dtype=BF, device=cuda_dev)
    weight[:columns, 3], weight[columns:, 3] = gate, up
    x = torch.zeros(1000, 72, dtype=BF, device=cuda_dev)
    x[:, 3] = 1
    for dtype in (BF, F32):
        _check(ops.w4a16_dense(x, weight, gated=True, out_dtype=dtype), gate, up)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("tokens,columns", [(1, 320), (12, 4096), (32, 320), (32, 4992)])
def test_int4(cuda_dev, dtype, tokens, columns):
    # code 9 is one, code 8 nothing: the scale is the weight, code 7 its negative
    gate, up = _gates_and_ups(cuda_dev, columns)
    q = torch.full((1, 2 * columns, 32), 0x88, dtype=torch.uint8, device=cuda_dev)
    q[0, :, 1] = 0x89
    q[0, :columns, 1] = torch.where(gate < 0, 0x87, 0x89).to(torch.uint8)
    s = torch.ones(1, 2 * columns, 2, dtype=BF, device=cuda_dev)
    s[0, :columns, 0], s[0, columns:, 0] = gate.abs(), up
    packed = ops.w4a16_prepack(q, s, layout=GLU)
    x = torch.zeros(tokens, 64, dtype=BF, device=cuda_dev)
    x[:, 2] = 1
    out = ops.w4a16_linear_few_tokens(x, packed, 2 * columns, layout=GLU, out_dtype=dtype)
    _check(out, gate, up)

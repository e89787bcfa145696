"""BF16 products through every kernel, width and split that w4a16_dense has, at sizes
that take them on this device, against 64-bit forms within bounds that count
roundings."""

import pytest
import torch

import dense_sizes
from test_gpu_products import Dense, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gated,dtype", dense_sizes.KINDS)
@pytest.mark.parametrize("shape", dense_sizes.SHAPES)
def test_dense(cuda_dev, shape, gated, dtype):
    tokens, n, k = dense_sizes.sizes()[shape, gated, dtype]
    weight = Dense(cuda_dev, n, k, gated, tokens)
    f32 = dtype is torch.float32
    _run(weight, cuda_dev, tokens, 0, add=not gated, f32=f32)
    _run(weight, cuda_dev, tokens, k + 8, add=False, f32=f32)

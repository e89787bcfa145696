"""BF16 products at sizes that take tiles of every width, against 64-bit forms within
bounds that count roundings."""

import pytest

from test_gpu_products import Dense, _run

pytestmark = pytest.mark.gpu

# On 152 SMs tiles of 96, 160 and 224 weight rows (twice each), then 64, 128, 192, 256
# and sizes between; columns that are no multiple of four, and one step of 64.
SIZES = [(300, 3222, 512, False), (300, 3326, 520, True), (520, 3906, 512, False),
         (520, 3856, 512, True), (2100, 1542, 512, False), (700, 4802, 512, True),
         (1024, 4096, 2088, True), (2048, 4094, 1024, True), (700, 7168, 2088, False),
         (1000, 8999, 1024, False), (610, 4096, 2048, True), (2049, 4096, 512, False),
         (1300, 2000, 64, True), (400, 5001, 72, False), (257, 9728, 264, False)]


@pytest.mark.parametrize("tokens,n,k,gated", SIZES)
def test_dense(cuda_dev, tokens, n, k, gated):
    weight = Dense(cuda_dev, n, k, gated, tokens)
    _run(weight, cuda_dev, tokens, 0, add=not gated, f32=not gated)
    _run(weight, cuda_dev, tokens, k + 8, add=False, f32=gated)

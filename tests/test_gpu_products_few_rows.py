"""Products of few weight rows and many columns, which a cluster of up to eight CTAs
shares, against 64-bit forms within bounds that count roundings."""

import pytest

from test_gpu_products import Dense, Int4, _run

pytestmark = pytest.mark.gpu

# rows of one cluster, up to the most that eights are taken for, and past it
ROWS = [1, 40, 129, 256, 300, 544, 1216]


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("tokens", [1, 7, 12, 32])
@pytest.mark.parametrize("k", [4104, 7168, 16392])
def test_dense(cuda_dev, n, tokens, k):
    _run(Dense(cuda_dev, n, k, False, n), cuda_dev, tokens, k + 24, add=tokens == 7, f32=tokens > 8)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("tokens", [1, 7, 12, 32])
@pytest.mark.parametrize("k", [4128, 7168, 16416])
def test_int4(cuda_dev, n, tokens, k):
    _run(Int4(cuda_dev, n, k, False, n), cuda_dev, tokens, k + 24, add=tokens == 7, f32=tokens > 8)


@pytest.mark.parametrize("kind,n", [(Dense, 2), (Dense, 310), (Int4, 128), (Int4, 384)])
@pytest.mark.parametrize("tokens", [1, 16, 30])
def test_gated(cuda_dev, kind, n, tokens):
    _run(kind(cuda_dev, n, 7168, True, n), cuda_dev, tokens, 0, add=False, f32=tokens > 1)

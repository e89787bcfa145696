"""A token's gated result does not depend on the tokens beside it, whatever their
gates, nor on what earlier calls have left behind."""

import pytest
import torch

from test_gpu_products import Dense, _rows

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("tokens,n,k", [(2048, 4096, 512), (600, 9728, 264), (5000, 130, 520),
                                        (300, 4096, 1024), (20, 4096, 512)])
@pytest.mark.parametrize("value", [3000.0, float("inf"), float("nan")])
def test_rows_beside_far_gates(cuda_dev, tokens, n, k, value):
    weight = Dense(cuda_dev, n, k, True, 11)
    x = _rows(torch.Generator(device=cuda_dev).manual_seed(12), tokens, k, 0, cuda_dev)
    clean = weight(x)
    far = torch.arange(tokens, device=cuda_dev) % 32 == 5
    x[far, 7] = value     # gates of either sign, past any exponential
    out = weight(x)
    assert not torch.equal(out[far], clean[far])
    assert torch.equal(out[~far], clean[~far])


@pytest.mark.parametrize("tokens,n,k", [(5000, 30, 520), (5000, 60, 264), (520, 9730, 512),
                                        (129, 5002, 512), (8192, 514, 64)])
def test_the_same_bits_behind_other_calls(cuda_dev, tokens, n, k):
    # tiles of few columns lie beside columns of the tensor memory that they do not use
    weight, other = Dense(cuda_dev, n, k, True, 13), Dense(cuda_dev, 4096, 512, True, 14)
    gen = torch.Generator(device=cuda_dev).manual_seed(15)
    x = _rows(gen, tokens, k, 0, cuda_dev)
    far = _rows(gen, 8192, 512, 0, cuda_dev) * 1000
    want = weight(x)
    for sign in (1, -1):
        other(sign * far)
        assert torch.equal(weight(x), want)

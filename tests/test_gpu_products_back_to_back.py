"""Products that follow one another closely: a kernel may ask for its weights before
the kernel in front of it has ended, and must not use them before."""

import pytest
import torch

import product_reference as ref
from w4a16_int4_moe_gb300 import ops

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _chain(x, first, last, tokens, out):
    # the first product's output, [n, k], is the second's weight
    w = ops.w4a16_dense(last, first)
    return w, ops.w4a16_dense(x[:tokens], w, out=out)


@pytest.mark.parametrize("rows", [24, 200, 1000])       # of the weight that is made
@pytest.mark.parametrize("tokens", [1, 12, 32, 64, 300])
def test_a_weight_of_the_product_before(cuda_dev, rows, tokens):
    k, inner = 1024, 512
    gen = torch.Generator(device=cuda_dev).manual_seed(rows + tokens)
    x = torch.randn(tokens, k, generator=gen, device=cuda_dev).to(BF)
    first = (torch.randn(k, inner, generator=gen, device=cuda_dev) / 700).to(BF)
    last = torch.randn(rows, inner, generator=gen, device=cuda_dev).to(BF)
    out = torch.empty(tokens, rows, dtype=BF, device=cuda_dev)
    _chain(x, first, last, tokens, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w, _ = _chain(x, first, last, tokens, out)
    for _ in range(5):
        last.copy_(torch.randn(rows, inner, generator=gen, device=cuda_dev))
        graph.replay()
        ref.check_product(w, last, first.double())
        ref.check_product(out, x, w.double())


@pytest.mark.parametrize("n,tokens", [(300, 1), (300, 20), (9900, 24), (9900, 5)])
def test_a_weight_packed_just_before(cuda_dev, n, tokens):
    k = 544
    gen = torch.Generator(device=cuda_dev).manual_seed(n + tokens)
    x = torch.randn(tokens, k, generator=gen, device=cuda_dev).to(BF)
    q = torch.zeros(1, n, k // 2, device=cuda_dev, dtype=torch.uint8)
    s = (torch.randn(1, n, k // 32, generator=gen, device=cuda_dev) / 100).to(BF)
    packed = ops.w4a16_prepack(q, s)
    out = ops.w4a16_linear_few_tokens(x, packed, n, out_dtype=torch.float32)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        packed = ops.w4a16_prepack(q, s)
        ops.w4a16_linear_few_tokens(x, packed, n, out=out)
    for _ in range(5):
        q.copy_(torch.randint(0, 256, q.shape, generator=gen, device=cuda_dev, dtype=torch.uint8))
        graph.replay()
        weight, loose = ref.int4_weight(q[0], s[0])
        ref.check_product(out, x, weight, loose)

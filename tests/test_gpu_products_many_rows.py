"""INT4 products whose weight has more rows than 64 an SM, for 17 to 32 tokens (and,
beside them, for fewer), against 64-bit forms within bounds that count roundings."""

import pytest
import torch

import product_reference as ref
from w4a16_int4_moe_gb300 import ops
from helpers import Guarded
from test_gpu_products import Int4, _check, _rows, _run

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32

# One and two groups, whole and half steps, up to and past what the rings hold, and
# blocks that come round again (more than 128 rows an SM); ragged last blocks.
SHAPES = [(9760, 32, False), (9729, 64, False), (9900, 96, False), (9857, 416, False),
          (10001, 512, False), (12288, 1504, False), (9730, 1536, False), (9985, 1568, False),
          (19585, 160, False), (20480, 2080, False), (40003, 544, False), (16384, 7168, False),
          (9856, 32, True), (9984, 544, True), (19584, 96, True), (39168, 1056, True)]


@pytest.mark.parametrize("n,k,gated", SHAPES)
@pytest.mark.parametrize("tokens", [17, 24, 31, 32])
def test_int4(cuda_dev, n, k, gated, tokens):
    weight = Int4(cuda_dev, n, k, gated, n + k)
    _run(weight, cuda_dev, tokens, 0, add=not gated and tokens % 2 == 1, f32=tokens % 2 == 1)
    _run(weight, cuda_dev, tokens, k + 40, add=False, f32=tokens % 2 == 0)


@pytest.mark.parametrize("tokens", [1, 8, 9, 16])
def test_fewer_tokens(cuda_dev, tokens):
    _run(Int4(cuda_dev, 19585, 1056, False), cuda_dev, tokens, 0, add=True, f32=True)


KINDS = [(9900, 544, False), (19712, 96, True), (20001, 1568, False)]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("n,k,gated", KINDS)
def test_a_token_that_is_not_finite_stays_alone(cuda_dev, n, k, gated, value):
    weight = Int4(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(5)
    x = _rows(gen, 20, k, 0, cuda_dev)
    clean = weight(x)
    x[3, k - 1] = value
    out = weight(x)
    keep = [t for t in range(20) if t != 3]
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("n,k,gated", KINDS)
def test_a_scale_that_is_not_finite_stays_in_its_row(cuda_dev, n, k, gated):
    weight = Int4(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(6)
    x = _rows(gen, 19, k, 0, cuda_dev)
    clean = weight(x)
    weight.s[5, k // 32 - 1] = float("nan")
    weight.packed = ops.w4a16_prepack(weight.q[None], weight.s[None], layout=weight.layout)
    out = weight(x)
    assert torch.isnan(out[:, 5]).all()
    keep = [r for r in range(out.shape[1]) if r != 5]
    assert torch.equal(out[:, keep], clean[:, keep])


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,k,gated", KINDS)
def test_reads_its_rows_and_writes_its_output(cuda_dev, n, k, gated, f32):
    # rows of a wider buffer whose other columns, and the rows behind the last, are NaN
    weight = Int4(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(7)
    wide = torch.full((64, k + 72), float("nan"), dtype=BF, device=cuda_dev)
    x = wide[:21, :k]
    x.copy_(_rows(gen, 21, k, 0, cuda_dev))
    g = Guarded((21, n // 2 if gated else n), F32 if f32 else BF, cuda_dev)
    weight(x, out=g.t)
    g.check("out")
    _check(weight, x, g.t)


def test_every_code_and_position(cuda_dev):
    # weight row r has code r % 16 everywhere, every token picks one column
    n, k = 9800, 128
    code = torch.arange(n, device=cuda_dev, dtype=torch.uint8)[:, None] % 16
    q = (code | code << 4).repeat(1, k // 2)
    s = (1 + (torch.arange(n * 4, device=cuda_dev) % 640).view(n, 4) / 64.0).to(BF)
    packed = ops.w4a16_prepack(q[None].contiguous(), s[None])
    for c0 in range(0, k, 32):
        x = torch.zeros(32, k, dtype=BF, device=cuda_dev)
        x[torch.arange(32), c0 + torch.arange(32)] = 1
        out = ops.w4a16_linear_few_tokens(x, packed, n, out_dtype=F32)
        # (a code has four bits and a scale eight: their product is exact)
        want = (code.float() - 8) * s[:, c0 // 32, None].float()
        assert torch.equal(out, want.t().expand(32, n))


def test_the_addend_may_be_the_output(cuda_dev):
    weight = Int4(cuda_dev, 9900, 544, False)
    gen = torch.Generator(device=cuda_dev).manual_seed(9)
    x = _rows(gen, 18, 544, 0, cuda_dev)
    add = torch.randn(18, 9900, generator=gen, device=cuda_dev)
    want = weight(x, addend=add, out_dtype=F32)
    mine = add.clone()
    weight(x, addend=mine, out=mine)
    assert torch.equal(mine, want)


@pytest.mark.parametrize("n,k,gated", KINDS)
def test_in_a_graph_and_two_calls_at_once(cuda_dev, n, k, gated):
    weight = Int4(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(10)
    xs = [_rows(gen, 23, k, 0, cuda_dev) for _ in range(2)]
    want = [weight(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[weight(x, stream=s) for _ in range(20)] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(g, w) for g in got)
    x, out = xs[0].clone(), torch.zeros_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):  # one after the other, each before the last has ended
            weight(x, out=out)
    x.copy_(xs[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1])


def test_weights_past_32_bits(cuda_dev):
    n, k = 1 << 20, 8192
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    at = torch.cat([torch.arange(40), torch.arange(n - 40, n)]).to(cuda_dev)
    x = torch.randn(20, k, generator=gen, device=cuda_dev).to(BF)
    q = torch.randint(0, 256, (1, n, k // 2), generator=gen, device=cuda_dev, dtype=torch.uint8)
    s = torch.rand(1, n, k // 32, generator=gen, device=cuda_dev).to(BF) * 0.02
    packed = ops.w4a16_prepack(q, s)
    weight, loose = ref.int4_weight(q[0][at], s[0][at])
    del q, s
    out = ops.w4a16_linear_few_tokens(x, packed, n, out_dtype=F32)
    ref.check_product(out[:, at], x, weight, loose)


@pytest.mark.parametrize("n", [300, 9900])
@pytest.mark.parametrize("tokens", [1, 12, 32])
def test_large_inputs(cuda_dev, n, tokens):
    # a group's sum, before its scale, is at most 32 * 8 * 2^119 = 2^127
    weight = Int4(cuda_dev, n, 544, False)
    gen = torch.Generator(device=cuda_dev).manual_seed(12)
    x = _rows(gen, tokens, 544, 0, cuda_dev).sign() * 2.0 ** 119
    _check(weight, x, weight(x, out_dtype=F32))

"""Products with one weight (w4a16_linear_few_tokens, w4a16_dense) against
64-bit forms, within bounds that count roundings (product_reference)."""

import pytest
import torch

import product_reference as ref
from w4a16_int4_moe_gb300 import ops
from helpers import Guarded

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _rows(gen, tokens, k, pitch, dev):
    return torch.randn(tokens, pitch or k, generator=gen, device=dev).to(BF)[:, :k]


class Int4:
    def __init__(self, dev, n, k, gated, seed=0):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.n, self.k, self.gated = n, k, gated
        self.q = torch.randint(0, 256, (n, k // 2), generator=gen, device=dev, dtype=torch.uint8)
        self.s = (torch.randn(n, k // 32, generator=gen, device=dev) * (0.2 / k ** 0.5)).to(BF)
        self.layout = ops.W4A16_LAYOUT_KTILE64_GLU16 if gated else ops.W4A16_LAYOUT_KTILE64
        self.packed = ops.w4a16_prepack(self.q[None], self.s[None], layout=self.layout)
        self.w, self.loose = ref.int4_weight(self.q, self.s)

    def __call__(self, x, **kw):
        return ops.w4a16_linear_few_tokens(x, self.packed, self.n, layout=self.layout, **kw)


class Dense:
    def __init__(self, dev, n, k, gated, seed=0):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.n, self.k, self.gated, self.loose = n, k, gated, None
        self.bits = (torch.randn(n, k, generator=gen, device=dev) / k ** 0.5).to(BF)
        self.w = self.bits.double()

    def __call__(self, x, **kw):
        return ops.w4a16_dense(x, self.bits, gated=self.gated, **kw)


def _check(weight, x, out, addend=None, what=""):
    ref.check_product(out, x, weight.w, weight.loose, weight.gated, addend, what)


def _run(weight, dev, tokens, pitch, add, f32):
    gen = torch.Generator(device=dev).manual_seed(tokens + weight.n)
    x = _rows(gen, tokens, weight.k, pitch, dev)
    columns = weight.n // 2 if weight.gated else weight.n
    addend = torch.randn(tokens, columns, generator=gen, device=dev) if add else None
    out = weight(x, addend=addend, out_dtype=F32 if f32 else BF)
    assert out.dtype is (F32 if f32 else BF)
    _check(weight, x, out, addend)
    # the same bits again, and into a buffer of the caller's
    again = torch.empty_like(out)
    assert weight(x, addend=addend, out=again) is again
    assert torch.equal(out.view(torch.uint8), again.view(torch.uint8))


# (n, k, gated): one tile and less, ragged ones, an odd number of groups, the layer's own
INT4 = [(1, 32, False), (16, 64, False), (17, 96, False), (100, 2080, False), (130, 544, False),
        (384, 1024, False), (1000, 160, False), (7168, 2048, False), (2047, 7168, False),
        (128, 32, True), (128, 96, True), (384, 544, True), (512, 7168, True), (4096, 7168, True)]


@pytest.mark.parametrize("n,k,gated", INT4)
@pytest.mark.parametrize("tokens", [1, 2, 5, 8, 9, 16, 17, 24, 31, 32])
def test_int4(cuda_dev, n, k, gated, tokens):
    weight = Int4(cuda_dev, n, k, gated, n + k)
    _run(weight, cuda_dev, tokens, 0, add=not gated and tokens % 2 == 1, f32=tokens % 2 == 1)
    _run(weight, cuda_dev, tokens, k + 40, add=False, f32=tokens % 2 == 0)


DENSE = [(1, 8, False), (3, 72, False), (16, 64, False), (60, 2088, False), (129, 520, False),
         (257, 1024, False), (1000, 136, False), (7168, 2048, False), (2, 8, True), (6, 64, True),
         (126, 264, True), (512, 1024, True), (2002, 2088, True), (4096, 7168, True)]


@pytest.mark.parametrize("n,k,gated", DENSE)
@pytest.mark.parametrize("tokens", [1, 3, 8, 15, 16, 32, 33, 64, 100, 128, 129, 257, 600])
def test_dense(cuda_dev, n, k, gated, tokens):
    weight = Dense(cuda_dev, n, k, gated, n + k)
    _run(weight, cuda_dev, tokens, 0, add=not gated and tokens % 2 == 1, f32=tokens % 2 == 1)
    _run(weight, cuda_dev, tokens, k + 40, add=not gated, f32=tokens % 2 == 0)


@pytest.mark.parametrize("tokens,n,k,gated", [(8192, 512, 1024, True), (8192, 7168, 256, False),
                                              (4099, 4096, 72, True), (5000, 130, 2048, False),
                                              (2500, 4000, 4104, False), (1025, 8, 8, False)])
def test_dense_of_many_rows(cuda_dev, tokens, n, k, gated):
    weight = Dense(cuda_dev, n, k, gated, tokens)
    _run(weight, cuda_dev, tokens, 0, add=not gated, f32=not gated)
    _run(weight, cuda_dev, tokens, k + 8, add=False, f32=False)


KINDS = [(Int4, 300, 544, False, 7), (Int4, 384, 1056, True, 20), (Dense, 300, 520, False, 7),
         (Dense, 310, 520, True, 20), (Dense, 300, 520, False, 150), (Dense, 310, 520, True, 300)]


@pytest.mark.parametrize("kind,n,k,gated,tokens", KINDS)
def test_no_tokens(cuda_dev, kind, n, k, gated, tokens):
    weight = kind(cuda_dev, n, k, gated)
    out = weight(torch.empty(0, k, dtype=BF, device=cuda_dev))
    assert out.shape == (0, n // 2 if gated else n)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("kind,n,k,gated,tokens", KINDS)
def test_a_token_that_is_not_finite_stays_alone(cuda_dev, kind, n, k, gated, tokens, value):
    weight = kind(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(5)
    x = _rows(gen, tokens, k, 0, cuda_dev)
    clean = weight(x)
    x[3, k - 1] = value
    out = weight(x)
    keep = [t for t in range(tokens) if t != 3]
    assert torch.equal(out[keep], clean[keep])
    if not gated:
        # (an infinity times a weight of zero is NaN, and in INT4 it may be in any case)
        assert not torch.isfinite(out[3].float()).any()


@pytest.mark.parametrize("kind,n,k,gated,tokens", KINDS)
def test_what_lies_behind_the_rows_is_not_used(cuda_dev, kind, n, k, gated, tokens):
    # rows of a wider buffer whose other columns, and the rows behind the last, are NaN
    weight = kind(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(6)
    wide = torch.full((tokens + 40, k + 72), float("nan"), dtype=BF, device=cuda_dev)
    x = wide[:tokens, :k]
    x.copy_(_rows(gen, tokens, k, 0, cuda_dev))
    _check(weight, x, weight(x))


@pytest.mark.parametrize("kind,n,k,gated,tokens", KINDS)
def test_extreme_rows(cuda_dev, kind, n, k, gated, tokens):
    # every row of another size, and a column that is far larger than the others
    weight = kind(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(7)
    x = _rows(gen, tokens, k, 0, cuda_dev).float()
    x *= 2.0 ** torch.linspace(-30, 20, tokens, device=cuda_dev).round()[:, None]
    x[:, k // 2] *= 2.0 ** 10
    if gated:   # (gates beyond the exponential's range: silu is 0 or the gate)
        x = x.clamp(-2.0 ** 20, 2.0 ** 20)
    x = x.to(BF)
    x[tokens // 2] = 0
    out = weight(x, out_dtype=F32)
    assert (out[tokens // 2] == 0).all()
    _check(weight, x, out)


def test_every_code_and_position(cuda_dev):
    # weight row r has code r % 16 everywhere, every token picks one column
    n, k = 160, 128
    code = torch.arange(n, device=cuda_dev, dtype=torch.uint8)[:, None] % 16
    q = (code | code << 4).repeat(1, k // 2)
    s = (1 + torch.arange(n * 4, device=cuda_dev).view(n, 4) / 64.0).to(BF)
    packed = ops.w4a16_prepack(q[None].contiguous(), s[None])
    for c0 in range(0, k, 32):
        x = torch.zeros(32, k, dtype=BF, device=cuda_dev)
        x[torch.arange(32), c0 + torch.arange(32)] = 1
        out = ops.w4a16_linear_few_tokens(x, packed, n, out_dtype=F32)
        want = (code.float() - 8) * s[:, c0 // 32, None].float()
        assert torch.equal(out, want.t().expand(32, n))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind,n,k,gated,tokens",
                         KINDS + [(Dense, 301, 520, False, 33), (Int4, 301, 544, False, 32),
                                  (Dense, 302, 520, True, 200)])
def test_writes_only_its_output(cuda_dev, kind, n, k, gated, tokens, f32):
    weight = kind(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(8)
    x = _rows(gen, tokens, k, 0, cuda_dev)
    g = Guarded((tokens, n // 2 if gated else n), F32 if f32 else BF, cuda_dev)
    weight(x, out=g.t)
    g.check("out")
    _check(weight, x, g.t)


@pytest.mark.parametrize("kind,n,k,gated,tokens", [c for c in KINDS if not c[3]])
def test_the_addend_may_be_the_output(cuda_dev, kind, n, k, gated, tokens):
    weight = kind(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(9)
    x = _rows(gen, tokens, k, 0, cuda_dev)
    add = torch.randn(tokens, n, generator=gen, device=cuda_dev)
    want = weight(x, addend=add, out_dtype=F32)
    mine = add.clone()
    weight(x, addend=mine, out=mine)
    assert torch.equal(mine, want)


@pytest.mark.parametrize("kind,n,k,gated,tokens", KINDS)
def test_on_a_side_stream_and_in_a_graph(cuda_dev, kind, n, k, gated, tokens):
    weight = kind(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(10)
    x = _rows(gen, tokens, k, 0, cuda_dev)
    want = weight(x)
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        weight(x, out=out)
        side.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            weight(x, out=out)
    out.zero_()
    new = _rows(gen, tokens, k, 0, cuda_dev)
    x.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, weight(new))
    by_stream = weight(x, stream=side)
    side.synchronize()
    assert torch.equal(out, by_stream)


@pytest.mark.parametrize("kind,n,k,gated,tokens", KINDS)
def test_two_calls_at_once(cuda_dev, kind, n, k, gated, tokens):
    # nothing is shared between calls: two streams, the same weight
    weight = kind(cuda_dev, n, k, gated)
    gen = torch.Generator(device=cuda_dev).manual_seed(11)
    xs = [_rows(gen, tokens, k, 0, cuda_dev) for _ in range(2)]
    want = [weight(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[weight(x, stream=s) for _ in range(20)] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(g, w) for g in got)

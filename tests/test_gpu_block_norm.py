"""The norms after and before a block (w4a16_block_norm) against a 64-bit form.

An FP32 sum of at most 16384 squares over 64 or more threads is off by fewer
than 2^9 half steps, the root halves that, and a dozen products and roundings
follow: fewer than 2^10 half steps of each norm's factor. h is a sum of two
terms, so what its terms lose is relative to their magnitudes (`size`), and it
goes on into y through the row's second norm."""

import pytest
import torch

import product_reference as ref
from w4a16_int4_moe_gb300 import ops
from helpers import Guarded

pytestmark = pytest.mark.gpu

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
NORM = 2.0 ** 10 * 2.0 ** -24
E4M3_HALF = 2.0 ** -4


def _inputs(dev, tokens, hidden, x32=True, post=True, gate=0, residual=True, pitch=0, offset=False,
            seed=0):
    gen = torch.Generator(device=dev).manual_seed(seed + tokens + hidden)

    def rows(scale, dtype=BF):
        return (torch.randn(tokens, pitch or hidden, generator=gen, device=dev)
                * scale).to(dtype)[:, :hidden]

    def weight():
        return ((0.0 if offset else 1.0)
                + 0.2 * torch.randn(hidden, generator=gen, device=dev)).to(BF)
    kw = dict(post_weight=weight() if post else None, residual=rows(3.0) if residual else None)
    if gate:
        kw["gate"] = rows(1.0) if gate == 2 else torch.tanh(weight().float()).to(BF)
        kw["branch_scale"] = 0.75
    if offset:
        kw.update(weight_offset=1.0, residual_scale=1.5)
    return rows(0.5, F32 if x32 else BF), weight(), kw


def _check(x, pre, kw, out, fp8_group=0, eps=1e-6):
    y_got, h_got, y8, scales = out
    y, h, size = ref.block_norm(x, pre, eps, kw.get("post_weight"), kw.get("gate"),
                                kw.get("residual"), kw.get("branch_scale", 1.0),
                                kw.get("residual_scale", 1.0), kw.get("weight_offset", 0.0))
    h_err = size * 2 * NORM
    tiny = 2.0 ** -133   # half the lowest subnormal BF16
    if h_got is not None:
        ref.assert_within(h_got, h, h_err + (h.abs() + h_err) * ref.BF16_HALF + tiny, "h")
    if pre is None:
        return
    # y = h / rms(h): what h loses, at its own place and through the root
    root = torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    w = (pre.double() + kw.get("weight_offset", 0.0)).abs()
    lost = (h_err.square().mean(1, keepdim=True).sqrt() / root)
    y_err = h_err / root * w + y.abs() * (lost + 2 * NORM)
    if y_got is not None:
        ref.assert_within(y_got, y, y_err + (y.abs() + y_err) * ref.BF16_HALF + tiny, "y")
    if fp8_group:
        hidden = y.shape[1]
        width = hidden if fp8_group < 0 else fp8_group
        pad = torch.nn.functional.pad
        grouped = pad(y.abs(), (0, -hidden % width)).view(y.shape[0], -1, width)
        worst = pad(y_err, (0, -hidden % width)).view(y.shape[0], -1, width).amax(-1)
        s = grouped.amax(-1).clamp_min(1e-10) / 448
        ref.assert_within(scales, s, worst / 448 + s * 2.0 ** -22, "scales")
        full = s.repeat_interleave(width, 1)[:, :hidden]
        rel = (worst / 448 / s).repeat_interleave(width, 1)[:, :hidden]
        v = y / full
        half = torch.clamp(v.abs() * E4M3_HALF, min=2.0 ** -10)
        half = half + (y_err / full + v.abs() * (rel + 2.0 ** -20)) * (1 + E4M3_HALF)
        ref.assert_within(y8.float(), v, half, "codes")


SHAPES = [(1, 7168, 0), (1, 8, 0), (3, 8, 24), (2, 136, 0), (5, 1000, 1048), (7, 2088, 2400),
          (33, 512, 0), (4, 16384, 0), (3, 16376, 0), (300, 1024, 0), (1500, 4096, 0),
          (700, 7168, 7176), (160, 8192, 0), (153, 120, 0), (700, 2600, 0), (200, 5000, 0),
          (200, 10000, 10008), (170, 12280, 0), (170, 16000, 0)]


@pytest.mark.parametrize("fp8_group", [0, 128, -1])
@pytest.mark.parametrize("tokens,hidden,pitch", SHAPES)
@pytest.mark.parametrize("x32,post,gate,residual,offset", [
    (True, True, 0, True, False), (False, False, 1, True, True), (True, False, 2, True, False),
    (False, True, 2, False, True), (True, True, 1, True, True)])
def test_block_norm(cuda_dev, tokens, hidden, pitch, x32, post, gate, residual, offset, fp8_group):
    x, pre, kw = _inputs(cuda_dev, tokens, hidden, x32, post, gate, residual, pitch, offset)
    out = ops.w4a16_block_norm(x, pre, fp8_group=fp8_group, **kw)
    _check(x, pre, kw, out, fp8_group)
    if fp8_group:   # the 8-bit form alone: the same bits
        only = ops.w4a16_block_norm(x, pre, fp8_group=fp8_group, bf16_out=False, **kw)
        assert only[0] is None and torch.equal(only[1], out[1])
        assert torch.equal(only[2].view(torch.uint8), out[2].view(torch.uint8))
        assert torch.equal(only[3], out[3])
    else:           # no norm behind the residual, and no h
        alone = ops.w4a16_block_norm(x, None, **kw)
        assert alone[0] is None and torch.equal(alone[1], out[1])
        y = torch.empty_like(out[0])
        ops.w4a16_block_norm(x, pre, out=(y, None, None, None), **kw)
        assert torch.equal(y, out[0])


def test_as_the_norm_in_front_of_the_experts(cuda_dev):
    # BF16 rows, a residual and no norm before it: w4a16_add_rms_norm's formula
    x, pre, kw = _inputs(cuda_dev, 40, 7168, False, False)
    for fp8_group in (0, 128, -1):
        a = ops.w4a16_block_norm(x, pre, fp8_group=fp8_group, **kw)
        b = ops.w4a16_add_rms_norm(x, pre, residual=kw["residual"], fp8_group=fp8_group)
        assert torch.equal(a[1], b[1])
        _check(x, pre, kw, b, fp8_group)
        _check(x, pre, kw, a, fp8_group)


def test_zero_rows_and_no_rows(cuda_dev):
    x, pre, kw = _inputs(cuda_dev, 4, 256)
    x[1] = 0
    kw["residual"][1] = 0
    for eps in (1e-6, 0.0):
        y, h, y8, s = ops.w4a16_block_norm(x, pre, eps, fp8_group=128, **kw)
        if eps:   # eps 0 makes 0 * inf of a zero row
            assert h[1].abs().max() == 0 and y[1].abs().max() == 0
            assert y8[1].float().abs().max() == 0
        else:
            assert torch.isnan(y[1].float()).all() and torch.isnan(s[1]).all()
        for row in (0, 2, 3):
            assert torch.isfinite(y[row].float()).all()
    out = ops.w4a16_block_norm(x[:0], pre, residual=kw["residual"][:0], fp8_group=128)
    assert out[0].shape == (0, 256) and out[3].shape == (0, 2)


@pytest.mark.parametrize("where", ["x", "residual", "gate"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_row_that_is_not_finite_stays_alone(cuda_dev, value, where):
    x, pre, kw = _inputs(cuda_dev, 40, 640, gate=2)
    clean = ops.w4a16_block_norm(x, pre, fp8_group=128, **kw)
    t = x if where == "x" else kw[where]
    t[17, 300] = value
    out = ops.w4a16_block_norm(x, pre, fp8_group=128, **kw)
    keep = [r for r in range(40) if r != 17]
    for a, b in zip(out, clean):
        a, b = (v.view(torch.uint8) if v.dtype is F8 else v for v in (a, b))
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(out[0][17, 300].float())
    assert torch.isnan(out[3][17, 300 // 128])
    assert torch.isnan(out[2][17, 256:384].float()).all()


def test_tiny_and_huge_rows(cuda_dev):
    # eps 0: y does not depend on the block's scale; squares stay inside FP32
    x, pre, kw = _inputs(cuda_dev, 6, 512, residual=False)
    x = x * torch.tensor([2.0 ** e for e in (-50, -40, -1, 0, 40, 50)], device=cuda_dev)[:, None]
    _check(x, pre, kw, ops.w4a16_block_norm(x, pre, 0.0, fp8_group=128, **kw), 128, 0.0)


def test_the_residual_may_be_updated_in_place(cuda_dev):
    for tokens in (3, 300):
        x, pre, kw = _inputs(cuda_dev, tokens, 7168)
        y, h, _, _ = ops.w4a16_block_norm(x, pre, **kw)
        mine = kw.pop("residual").clone()
        y2 = torch.empty_like(y)
        ops.w4a16_block_norm(x, pre, residual=mine, out=(y2, mine, None, None), **kw)
        assert torch.equal(y, y2) and torch.equal(h, mine)


@pytest.mark.parametrize("tokens,hidden", [(3, 200), (170, 7168)])
def test_writes_only_its_outputs(cuda_dev, tokens, hidden):
    x, pre, kw = _inputs(cuda_dev, tokens, hidden, gate=2)
    g = [Guarded((tokens, hidden), BF, cuda_dev), Guarded((tokens, hidden), BF, cuda_dev),
         Guarded((tokens, hidden), F8, cuda_dev),
         Guarded((tokens, -(-hidden // 128)), F32, cuda_dev)]
    out = ops.w4a16_block_norm(x, pre, fp8_group=128, out=tuple(b.t for b in g), **kw)
    for b, what in zip(g, ("y", "h", "codes", "scales")):
        b.check(what)
    _check(x, pre, kw, out, 128)


def test_on_a_side_stream_and_in_a_graph(cuda_dev):
    x, pre, kw = _inputs(cuda_dev, 20, 1024, gate=1)
    want = ops.w4a16_block_norm(x, pre, fp8_group=-1, **kw)
    out = tuple(torch.zeros_like(t) for t in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.w4a16_block_norm(x, pre, fp8_group=-1, out=out, **kw)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ops.w4a16_block_norm(x, pre, fp8_group=-1, out=out, **kw)
    for t in out:
        t.view(torch.uint8).zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))

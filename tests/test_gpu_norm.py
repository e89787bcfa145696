"""The residual's addition with the RMS norm (w4a16_add_rms_norm) against a
64-bit form. A BF16 value is off by half a step, an e4m3 code by half a step
of the quotient (2^-10 below the smallest normal, 2^-6), plus what the FP32
steps before the rounding lose: fewer than 2^10 half steps (a sum of at most
16384 squares over 128 or more lanes, halved by the root, and four products)."""

import numpy as np
import pytest
import torch

import layer_reference as ref
from w4a16_int4_moe_gb300 import ops
from helpers import Guarded

pytestmark = pytest.mark.gpu

FP32_STEPS = 2.0 ** 10 * ref.U32


def _f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def _inputs(tokens, hidden, residual, dev, seed=0, pitch=0, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    def rows(scale):
        t = torch.randn(tokens, pitch or hidden, generator=gen) * scale
        return t.to(torch.bfloat16).to(dev)[:, :hidden]
    x = rows(spread)
    r = rows(3.0 * spread) if residual else None
    w = (1 + 0.2 * torch.randn(hidden, generator=gen)).to(torch.bfloat16).to(dev)
    return x, r, w


def _check(x, r, w, eps, out, fp8_group):
    y_got, r_got, y8, scales = out
    h, y = ref.norm(_f64(x), None if r is None else _f64(r), _f64(w), eps)
    if y_got is not None:
        ref.assert_within(_f64(y_got), y, np.abs(y) * (ref.BF16_HALF + 2 * FP32_STEPS), "y")
    if r is not None:
        ref.assert_within(_f64(r_got), h, np.abs(h) * (ref.BF16_HALF + 2 * ref.U32), "residual")
    if fp8_group:
        group = h.shape[1] if fp8_group < 0 else fp8_group
        s = ref.group_scales(y, group)
        ref.assert_within(_f64(scales), s, s * FP32_STEPS, "scales")
        v = y / np.repeat(s, group, axis=1)[:, :h.shape[1]]
        half = np.maximum(np.abs(v) * ref.E4M3_HALF, 2.0 ** -10) + np.abs(v) * 4 * FP32_STEPS
        codes = ref.e4m3(y8.view(torch.uint8).cpu().numpy())
        ref.assert_within(codes, v, half, "codes")
        assert np.abs(codes).max(initial=0) <= 448


@pytest.mark.parametrize("fp8_group", [0, 128, -1])
@pytest.mark.parametrize("tokens,hidden,residual,pitch", [
    (1, 7168, True, 0), (1, 8, False, 0), (3, 8, True, 16), (2, 136, True, 0),
    (5, 1000, False, 1048), (7, 2088, True, 2400), (33, 512, True, 0), (4, 16384, True, 0),
    (3, 16376, False, 0), (300, 1024, True, 0), (1500, 4096, True, 0), (700, 7168, False, 7176),
    (160, 8192, True, 0), (153, 120, True, 0),
])
def test_norm(cuda_dev, tokens, hidden, residual, pitch, fp8_group):
    x, r, w = _inputs(tokens, hidden, residual, cuda_dev, tokens + hidden, pitch)
    out = ops.w4a16_add_rms_norm(x, w, 1e-6, residual=r, fp8_group=fp8_group)
    _check(x, r, w, 1e-6, out, fp8_group)
    if fp8_group:   # the 8-bit form alone: the same bits
        only = ops.w4a16_add_rms_norm(x, w, 1e-6, residual=r, fp8_group=fp8_group, bf16_out=False)
        assert only[0] is None
        assert torch.equal(only[2].view(torch.uint8), out[2].view(torch.uint8))
        assert torch.equal(only[3], out[3])


def test_zero_rows_and_zero_tokens(cuda_dev):
    x, r, w = _inputs(4, 256, True, cuda_dev)
    x[1] = 0
    r[1] = 0
    for eps in (1e-6, 0.0):
        y, res, y8, s = ops.w4a16_add_rms_norm(x, w, eps, residual=r, fp8_group=128)
        assert res[1].abs().max() == 0
        if eps:   # eps 0 makes 0 * inf of a zero row
            assert y[1].abs().max() == 0 and y8[1].float().abs().max() == 0
            # one correctly rounded FP32 division
            assert np.all(s[1].cpu().numpy() == np.float32(1e-10) / np.float32(448))
        else:
            assert torch.isnan(y[1].float()).all() and torch.isnan(s[1]).all()
    for row in (0, 2, 3):
        assert torch.isfinite(y[row].float()).all()
    y, res, y8, s = ops.w4a16_add_rms_norm(x[:0], w, residual=r[:0], fp8_group=128)
    assert y.shape == (0, 256) and s.shape == (0, 2)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_a_row_that_is_not_finite_stays_alone(cuda_dev, value):
    x, r, w = _inputs(40, 640, True, cuda_dev, 5)
    clean = ops.w4a16_add_rms_norm(x, w, residual=r, fp8_group=128)
    x[17, 300] = value
    y, res, y8, s = ops.w4a16_add_rms_norm(x, w, residual=r, fp8_group=128)
    keep = [t for t in range(40) if t != 17]
    for a, b in zip((y, res, y8.view(torch.uint8), s),
                    (clean[0], clean[1], clean[2].view(torch.uint8), clean[3])):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(y[17, 300].float())           # inf * rsqrt(inf) = inf * 0
    assert torch.isnan(s[17, 300 // 128])
    assert torch.isnan(y8[17, 256:384].float()).all()


def test_tiny_and_huge_rows(cuda_dev):
    # eps 0: the norm does not depend on the row's scale, except for what BF16
    # cannot hold; sums of squares stay inside FP32 for |h| up to 2^56
    x, _, w = _inputs(6, 512, False, cuda_dev, 9)
    base = (x.float() * torch.tensor([2.0 ** e for e in (-56, -40, -1, 0, 40, 56)],
                                     device=cuda_dev)[:, None]).to(torch.bfloat16)
    out = ops.w4a16_add_rms_norm(base, w, 0.0, fp8_group=128)
    _check(base, None, w, 0.0, out, 128)


def test_the_residual_may_be_updated_in_place(cuda_dev):
    x, r, w = _inputs(65, 7168, True, cuda_dev, 3)
    y, res, _, _ = ops.w4a16_add_rms_norm(x, w, residual=r)
    mine = r.clone()
    y2 = torch.empty_like(y)
    ops.w4a16_add_rms_norm(x, w, residual=mine, out=(y2, mine, None, None))
    assert torch.equal(y, y2) and torch.equal(res, mine)


@pytest.mark.parametrize("tokens,hidden", [(3, 200), (170, 7168)])
def test_writes_only_its_outputs(cuda_dev, tokens, hidden):
    x, r, w = _inputs(tokens, hidden, True, cuda_dev, 8)
    g = [Guarded((tokens, hidden), torch.bfloat16, cuda_dev),
         Guarded((tokens, hidden), torch.bfloat16, cuda_dev),
         Guarded((tokens, hidden), torch.float8_e4m3fn, cuda_dev),
         Guarded((tokens, -(-hidden // 128)), torch.float32, cuda_dev)]
    out = ops.w4a16_add_rms_norm(x, w, residual=r, fp8_group=128, out=tuple(b.t for b in g))
    for b, what in zip(g, ("y", "residual", "codes", "scales")):
        b.check(what)
    _check(x, r, w, 1e-6, out, 128)


def test_on_a_side_stream_and_in_a_graph(cuda_dev):
    x, r, w = _inputs(20, 1024, True, cuda_dev, 4)
    want = ops.w4a16_add_rms_norm(x, w, residual=r, fp8_group=-1)
    out = tuple(torch.zeros_like(t) for t in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ops.w4a16_add_rms_norm(x, w, residual=r, fp8_group=-1, out=out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            ops.w4a16_add_rms_norm(x, w, residual=r, fp8_group=-1, out=out)
    for t in out:
        t.view(torch.uint8).zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("fp8_group", [0, 128, -1])
@pytest.mark.parametrize("tokens,hidden,residual,pitch", [
    # more rows than SMs, and than four times as many, at every division of a row
    (400, 2088, True, 0), (700, 2600, True, 0), (200, 3336, False, 3400), (200, 5000, True, 0),
    (200, 8000, True, 8008), (200, 10000, True, 0), (170, 12280, False, 0), (170, 16000, True, 0),
    (100, 10008, True, 0),
])
def test_norm_of_many_rows(cuda_dev, tokens, hidden, residual, pitch, fp8_group):
    test_norm(cuda_dev, tokens, hidden, residual, pitch, fp8_group)

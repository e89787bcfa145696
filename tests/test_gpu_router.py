"""The router's product (w4a16_router_logits) against a 64-bit product; the
bound counts the additions' roundings (layer_reference.sum_bound)."""

import numpy as np
import pytest
import torch

import layer_reference as ref
from w4a16_int4_moe_gb300 import ops
from helpers import Guarded

pytestmark = pytest.mark.gpu


def _inputs(tokens, hidden, experts, dev, pitch=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, pitch or hidden, generator=gen).to(torch.bfloat16).to(dev)[:, :hidden]
    w = (torch.randn(experts, hidden, generator=gen) / hidden ** 0.5).to(torch.bfloat16).to(dev)
    return x, w


def _check(got, x, w):
    xf, wf = x.double().cpu().numpy(), w.double().cpu().numpy()
    bound = ref.sum_bound(x.shape[1]) * (np.abs(xf) @ np.abs(wf).T)
    ref.assert_within(got.cpu().numpy(), xf @ wf.T, bound, "logits")


@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 31, 48, 64, 65, 128, 129, 200, 777])
@pytest.mark.parametrize("hidden,experts,pitch", [
    (7168, 384, 0), (2088, 60, 2400), (512, 8, 0),
])
def test_router(cuda_dev, tokens, hidden, experts, pitch):
    x, w = _inputs(tokens, hidden, experts, cuda_dev, pitch, tokens)
    _check(ops.w4a16_router_logits(x, w), x, w)


@pytest.mark.parametrize("tokens,hidden,experts", [
    (1, 8, 1), (3, 8, 1), (130, 8, 2), (5, 24, 3), (140, 40, 1), (33, 72, 17), (129, 200, 257),
    (257, 136, 1024), (2, 1000, 1024), (1, 14336, 129), (300, 14336, 100), (1025, 320, 383),
    (2049, 64, 16), (4100, 1024, 256), (8192, 7168, 384),
])
def test_router_odd_sizes(cuda_dev, tokens, hidden, experts):
    x, w = _inputs(tokens, hidden, experts, cuda_dev, seed=hidden)
    _check(ops.w4a16_router_logits(x, w), x, w)


@pytest.mark.parametrize("tokens", [0, 1, 20, 150])
def test_writes_only_its_output_and_repeats_bits(cuda_dev, tokens):
    x, w = _inputs(tokens, 328, 45, cuda_dev)
    g = Guarded((tokens, 45), torch.float32, cuda_dev)
    ops.w4a16_router_logits(x, w, out=g.t)
    g.check("logits")
    for _ in range(3):
        assert torch.equal(ops.w4a16_router_logits(x, w), g.t)


@pytest.mark.parametrize("tokens", [6, 200])
def test_a_token_that_is_not_finite_stays_alone(cuda_dev, tokens):
    x, w = _inputs(tokens, 512, 40, cuda_dev)
    clean = ops.w4a16_router_logits(x, w)
    x[3, 77] = float("nan")
    x[4, 511] = float("inf")
    got = ops.w4a16_router_logits(x, w)
    assert torch.isnan(got[3]).all() and not torch.isfinite(got[4]).any()
    keep = [t for t in range(tokens) if t not in (3, 4)]
    assert torch.equal(got[keep], clean[keep])


def test_in_a_graph_on_a_side_stream(cuda_dev):
    for tokens in (4, 300):
        x, w = _inputs(tokens, 1024, 96, cuda_dev)
        want = ops.w4a16_router_logits(x, w)
        out = torch.zeros_like(want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                ops.w4a16_router_logits(x, w, out=out)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


@pytest.mark.parametrize("tokens,hidden,experts,pitch", [
    # pairs of CTAs, their columns split by four, by two and not at all, with a
    # last pair of one CTA's tokens, a last step outside the columns, padding
    (1500, 7168, 384, 0), (1450, 2056, 250, 2064), (3000, 4104, 384, 0), (4096, 7168, 384, 0),
    (2100, 7168, 64, 0), (6000, 520, 383, 528), (8100, 136, 70, 0), (700, 7168, 384, 0),
])
def test_router_many_tokens(cuda_dev, tokens, hidden, experts, pitch):
    x, w = _inputs(tokens, hidden, experts, cuda_dev, pitch, tokens)
    g = Guarded((tokens, experts), torch.float32, cuda_dev)
    ops.w4a16_router_logits(x, w, out=g.t)
    g.check("logits")
    _check(g.t, x, w)
    assert torch.equal(ops.w4a16_router_logits(x, w), g.t)


@pytest.mark.parametrize("tokens,hidden,experts", [
    # both sides of one wave of the few-token kernel
    (400, 2088, 60), (640, 2088, 60), (1500, 128, 16), (1800, 128, 16), (500, 1024, 32),
    (384, 7168, 64), (420, 7168, 64), (33, 520, 1024), (16, 520, 1024), (8, 520, 1024),
])
def test_router_between_the_kernels(cuda_dev, tokens, hidden, experts):
    test_router_many_tokens(cuda_dev, tokens, hidden, experts, 0)


@pytest.mark.parametrize("tokens,hidden,experts", [
    # clusters of eight, four, two and one of the small kernel
    (300, 2088, 60), (777, 2088, 60), (1200, 2088, 60), (1600, 136, 16), (2500, 136, 16),
    (4000, 136, 16), (8100, 136, 16), (1900, 264, 64), (2000, 4096, 16),
])
def test_router_small_clusters(cuda_dev, tokens, hidden, experts):
    test_router_many_tokens(cuda_dev, tokens, hidden, experts, hidden + 8)


def test_router_widest_tiles(cuda_dev):
    # 256 experts a tile, steps of 64 columns
    test_router_many_tokens(cuda_dev, 10000, 264, 256, 0)

"""The routing front end on both sides of every number of experts at which a
lane holds more logits, masked rows and ties among them."""

import numpy as np
import pytest
import torch

import oracle
from w4a16_int4_moe_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("topk", [1, 2, 3, 8, 32])
@pytest.mark.parametrize("experts", [1, 2, 8, 31, 32, 33, 127, 128, 129, 511, 512, 513, 1023, 1024])
def test_top_k_of(cuda_dev, experts, topk, dtype):
    if topk > experts:
        return
    rng = np.random.default_rng(experts + topk)
    lg = np.round(rng.standard_normal((70, experts)) * 16) / 16
    lg[20:40][rng.random((20, experts)) < 0.8] = -np.inf
    lg[40:60][rng.random((20, experts)) < 0.8] = float(torch.finfo(dtype).min)
    t = torch.from_numpy(lg.astype(np.float32)).to(dtype).to(cuda_dev)
    rid, rw = oracle.topk_softmax(lg, topk, True, experts // 4, max(1, experts // 2))
    args = (topk, True, experts // 4, max(1, experts // 2))
    ids, w = ops.w4a16_topk_softmax(t, *args)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=1e-5, atol=1e-8)
    ids2, w2, *_ = ops.w4a16_moe_route_align(
        t, topk, 16, torch.zeros(1, dtype=torch.int32, device=cuda_dev), *args[1:])
    assert torch.equal(ids2, ids) and torch.equal(w2, w)

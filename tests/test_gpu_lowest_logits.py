"""Logits of a type's lowest finite value are chosen like any others (only
-inf masks an expert): rows padded with them, and rows of nothing else."""

import numpy as np
import pytest
import torch

import oracle
from w4a16_int4_moe_gb300 import ops
from w4a16_int4_moe_gb300 import workloads as wl
from helpers import bf16_tensor, dev
from test_gpu_moe_few import _close, _packed, _workspace

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16]


def _logits(tokens, experts, dtype, seed):
    """Row t keeps t % 7 experts, of the rest a third are -inf in every other row."""
    lowest = float(torch.finfo(dtype).min)
    rng = np.random.default_rng(seed)
    lg = np.full((tokens, experts), lowest)
    for t in range(tokens):
        if t % 2:
            lg[t, rng.choice(experts, size=experts // 3, replace=False)] = -np.inf
        keep = rng.choice(experts, size=min(experts, t % 7), replace=False)
        lg[t, keep] = np.round(rng.standard_normal(keep.size) * 8) / 8
    return lg, torch.from_numpy(lg.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("tokens,experts,topk", [(14, 9, 8), (40, 64, 8), (30, 384, 8), (9, 1024, 32)])
def test_topk_softmax_and_route_align(cuda_dev, tokens, experts, topk, renorm, dtype):
    lg, t = _logits(tokens, experts, dtype, experts)
    t = t.to(cuda_dev)
    rid, rw = oracle.topk_softmax(lg, topk, renorm)
    ids, w = ops.w4a16_topk_softmax(t, topk, renorm)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=1e-5, atol=1e-8)
    ids2, w2, *_ = ops.w4a16_moe_route_align(t, topk, 16, torch.zeros(1, dtype=torch.int32,
                                                                      device=cuda_dev), renorm)
    assert torch.equal(ids2, ids) and torch.equal(w2, w)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [1, 2, 14])
def test_few_tokens(cuda_dev, tokens, dtype):
    # (the first token's row holds nothing but the lowest value)
    p = wl.uniform_problem(tokens, 128, 64, 16, 1, seed=3)
    p.topk = 4
    lg, t = _logits(tokens, 16, dtype, tokens)
    ids = torch.empty(tokens, 4, dtype=torch.int32, device=cuda_dev)
    w = torch.empty(tokens, 4, device=cuda_dev)
    gu, dn = _packed(p, cuda_dev)
    out = ops.w4a16_moe_few_tokens(gu, dn, 16, p.hidden, p.inter, bf16_tensor(p.x, cuda_dev), ids,
                                   w, _workspace(p, cuda_dev), logits=t.to(cuda_dev))
    rid, rw = oracle.topk_softmax(lg, 4, True)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=1e-5, atol=1e-8)
    _close(out, oracle.bf16_bits_to_f64(p.x), rid, w.cpu().numpy(), p)

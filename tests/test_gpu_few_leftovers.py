"""The few-token layer's results do not depend on what its memory held before:
sizes whose last stage of 256 columns is not whole, after calls and fills that
leave NaN bits in the workspace and in the SMs' shared memory."""

import numpy as np
import pytest
import torch

import oracle
from w4a16_int4_moe_gb300 import ops
from w4a16_int4_moe_gb300 import workloads as wl
from helpers import bf16_tensor, dev
from test_gpu_moe_few import _close, _packed, _run, _workspace

pytestmark = pytest.mark.gpu

HEADER = 4096   # the status words and counters lie in a workspace's first bytes

SIZES = [  # hidden with an odd number of 128-column blocks, inter that is no multiple of 256
    (1056, 192), (544, 64), (2080, 320), (96, 64), (512, 192), (1056, 256), (7168, 1408),
]


@pytest.mark.parametrize("tokens", [1, 2, 3, 5, 20])
@pytest.mark.parametrize("hidden,inter", SIZES)
def test_a_workspace_of_any_bits(cuda_dev, tokens, hidden, inter):
    p = wl.uniform_problem(tokens, hidden, inter, 8, 3, seed=hidden + tokens)
    packed, ws = _packed(p, cuda_dev), _workspace(p, cuda_dev)
    ws[HEADER:] = 0xFF
    out = _run(p, cuda_dev, packed=packed, ws=ws)
    _close(out, oracle.bf16_bits_to_f64(p.x), p.topk_ids, p.topk_weights, p)


@pytest.mark.parametrize("tokens", [1, 2])
@pytest.mark.parametrize("hidden,inter", SIZES)
def test_shared_memory_of_any_bits(cuda_dev, tokens, hidden, inter):
    # three tokens on 96 experts whose packed bytes are all 0xFF: every SM's
    # ring is full of them when the tokens of interest follow
    size = [ops.w4a16_prepack_size(96, 2 * inter, hidden, 32, ops.W4A16_LAYOUT_KTILE64_GLU16),
            ops.w4a16_prepack_size(96, hidden, inter)]
    bad = [torch.full((n,), 0xFF, dtype=torch.uint8, device=cuda_dev) for n in size]
    q = wl.uniform_problem(3, hidden, inter, 1, 1, seed=1)
    ids = np.arange(96, dtype=np.int32).reshape(3, 32)
    bad_ws = torch.zeros(ops.w4a16_moe_few_tokens_workspace_size(3, 32, hidden, inter),
                         dtype=torch.uint8, device=cuda_dev)
    p = wl.uniform_problem(tokens, hidden, inter, 8, 3, seed=hidden + tokens)
    packed, ws = _packed(p, cuda_dev), _workspace(p, cuda_dev)
    for _ in range(5):
        ops.w4a16_moe_few_tokens(bad[0], bad[1], 96, hidden, inter, bf16_tensor(q.x, cuda_dev),
                                 dev(ids, cuda_dev), torch.ones(3, 32, device=cuda_dev), bad_ws)
        out = _run(p, cuda_dev, packed=packed, ws=ws)
        _close(out, oracle.bf16_bits_to_f64(p.x), p.topk_ids, p.topk_weights, p)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("tokens", [1, 2, 3, 11])
def test_after_a_call_that_was_not_finite(cuda_dev, tokens, value):
    # padding rows of a captured batch hold anything: what they leave in the
    # workspace does not reach a later call of another number of tokens
    p = wl.uniform_problem(20, 1056, 192, 12, 3, seed=4)
    packed, ws = _packed(p, cuda_dev), _workspace(p, cuda_dev)
    x = bf16_tensor(p.x, cuda_dev).clone()
    x[1::2] = value
    q = wl.uniform_problem(tokens, 1056, 192, 12, 3, seed=6)
    q.q_gu, q.s_gu, q.q_dn, q.s_dn = p.q_gu, p.s_gu, p.q_dn, p.s_dn
    for _ in range(5):
        _run(p, cuda_dev, packed=packed, ws=ws, x=x)
        out = _run(q, cuda_dev, packed=packed, ws=ws)
        _close(out, oracle.bf16_bits_to_f64(q.x), q.topk_ids, q.topk_weights, q)

"""A few-token call from logits whose wait for the other CTAs' routing gives up
(the host lowers the limit; nothing faults): CTAs may then have read what the
routing tensors held before, and disagree. The status says so, and the next
call on the same workspace is right."""

import numpy as np
import pytest
import torch

from w4a16_int4_moe_gb300 import ops
from w4a16_int4_moe_gb300 import workloads as wl
from helpers import bf16_tensor, dev
from test_gpu_moe_few import _packed, _workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("limit", ["1", "100", "2000"])
@pytest.mark.parametrize("stale", ["none local", "one local", "an earlier call's", "any bits"])
@pytest.mark.parametrize("tokens", [3, 9, 32])
def test_the_next_call_is_right(cuda_dev, monkeypatch, tokens, stale, limit):
    p = wl.uniform_problem(tokens, 1056, 512, 8, 2, seed=41)
    (gu, dn), ws, x = _packed(p, cuda_dev), _workspace(p, cuda_dev), bf16_tensor(p.x, cuda_dev)
    rng = np.random.default_rng(tokens)
    logits = [dev(rng.standard_normal((tokens, 16)).astype(np.float32), cuda_dev) for _ in range(2)]
    ids = torch.empty(tokens, 2, dtype=torch.int32, device=cuda_dev)
    w = torch.empty(tokens, 2, device=cuda_dev)

    def call(lg):
        return ops.w4a16_moe_few_tokens(gu, dn, 8, 1056, 512, x, ids, w, ws, logits=lg,
                                        expert_offset=4)

    want = [call(lg).clone() for lg in logits]
    routed = ids.clone()
    assert ops.w4a16_read_device_status(ws)[0] == ops.W4A16_OK
    for _ in range(4):
        ids.copy_({"none local": torch.full_like(ids, -1), "an earlier call's": routed,
                   "one local": torch.where(torch.arange(2 * tokens, device=cuda_dev)
                                            .view(tokens, 2) == 3, 5, -1).to(torch.int32),
                   "any bits": torch.full_like(ids, -0x5A5A5A5B)}[stale])
        torch.cuda.synchronize()
        monkeypatch.setenv("W4A16_WAIT_TIMEOUT_CYCLES", limit)
        call(logits[0])
        st, word = ops.w4a16_read_device_status(ws)
        monkeypatch.delenv("W4A16_WAIT_TIMEOUT_CYCLES")
        assert limit == "2000" or (st == ops.W4A16_ERR_TIMEOUT and 0x1021 <= word <= 0x1025), hex(word)
        # status words and counters
        assert not ws[:2048].any()
        for lg, right in zip(logits, want):
            assert torch.equal(call(lg), right)
        assert ops.w4a16_read_device_status(ws)[0] == ops.W4A16_OK

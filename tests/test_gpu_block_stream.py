"""MoEBlock.forward(stream=s): everything that it makes comes from s's share of
the allocator, and its bits are those of a call on the current stream, also
while the current stream takes and gives back memory of the same sizes."""

import pytest
import torch

from w4a16_int4_moe_gb300 import moe as moe_mod
from w4a16_int4_moe_gb300 import ops
from w4a16_int4_moe_gb300 import workloads as wl
from helpers import bf16_tensor
from test_gpu_moe_few import _packed

pytestmark = pytest.mark.gpu


def _block(p, dev, tokens, fp8):
    gu, dn = _packed(p, dev)
    layer = moe_mod.W4A16MoE(
        moe_mod.PackedExperts(gu, 8, 512, 512, ops.W4A16_LAYOUT_KTILE64_GLU16),
        moe_mod.PackedExperts(dn, 8, 512, 256), 2, tokens, deterministic=True, device=dev)
    gen = torch.Generator().manual_seed(3)
    nw = (1 + 0.1 * torch.randn(512, generator=gen)).to(torch.bfloat16).to(dev)
    rw = (torch.randn(16, 512, generator=gen) / 512 ** 0.5).to(torch.bfloat16).to(dev)
    res = torch.randn(tokens, 512, generator=gen).to(torch.bfloat16).to(dev)
    return moe_mod.MoEBlock(nw, rw, layer, expert_offset=4, fp8_rows=fp8), res


def _stream_of(t):
    """The stream whose part of the allocator t lies in."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not the allocator's")


@pytest.mark.parametrize("tokens", [4, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_block_on_a_stream_of_its_own(cuda_dev, monkeypatch, tokens, fp8):
    p = wl.uniform_problem(tokens, 512, 256, 8, 2, seed=21)
    block, res = _block(p, cuda_dev, tokens, fp8)
    x = bf16_tensor(p.x, cuda_dev)
    want = [t.clone() for t in block.forward(x, res)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    made = []
    for name in ("w4a16_add_rms_norm", "w4a16_router_logits"):
        def call(*args, real=getattr(ops, name), **kw):
            got = real(*args, **kw)
            made.extend(t for t in (got if isinstance(got, tuple) else (got,)) if t is not None)
            return got
        monkeypatch.setattr(ops, name, call)
    made.extend(block.forward(x, res, stream=side))
    side.synchronize()
    assert len(made) >= 4 and {_stream_of(t) for t in made} == {side.cuda_stream}
    made.clear()
    monkeypatch.undo()
    for _ in range(30):
        junk = [torch.full((tokens, n), float("nan"), device=cuda_dev) for n in (16, 128, 256, 512)]
        del junk
        got = block.forward(x, res, stream=side)
        junk = [torch.full((tokens, n), float("nan"), device=cuda_dev) for n in (16, 128, 256, 512)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))

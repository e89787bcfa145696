"""The MoE half of a decoder layer with a shared expert and the norms behind it:
norm, router, experts, shared expert (BF16 or INT4 weights), the norm of the sum
into the residual, the next block's norm. Each addition to the block is checked
against its 64-bit form on the block's own inputs to it."""

import numpy as np
import pytest
import torch

import product_reference as ref
from w4a16_int4_moe_gb300 import moe as moe_mod
from w4a16_int4_moe_gb300 import ops
from w4a16_int4_moe_gb300 import workloads as wl
from helpers import bf16_tensor, dev
from test_gpu_block_norm import _check as check_norm
from test_gpu_moe_few import _packed

pytestmark = pytest.mark.gpu

H, I = 512, 256
BF = torch.bfloat16


def _shared(kind, device, max_tokens):
    gen = torch.Generator(device=device).manual_seed(17)
    if kind == "bf16":
        gu = (torch.randn(2 * I, H, generator=gen, device=device) / H ** 0.5).to(BF)
        dn = (torch.randn(H, I, generator=gen, device=device) / I ** 0.5).to(BF)
        return moe_mod.SharedExpert(gu, dn), (gu.double(), None), (dn.double(), None)

    def codes(n, k):
        q = torch.randint(0, 256, (1, n, k // 2), generator=gen, device=device, dtype=torch.uint8)
        s = torch.randn(1, n, k // 32, generator=gen, device=device) * (0.2 / k ** 0.5)
        return q, s.to(BF)
    q_gu, s_gu = codes(2 * I, H)
    q_dn, s_dn = codes(H, I)
    gu = moe_mod.PackedExperts.from_checkpoint(q_gu, s_gu, layout=ops.W4A16_LAYOUT_KTILE64_GLU16)
    dn = moe_mod.PackedExperts.from_checkpoint(q_dn, s_dn)
    return (moe_mod.PackedSharedExpert(gu, dn, max_tokens), ref.int4_weight(q_gu[0], s_gu[0]),
            ref.int4_weight(q_dn[0], s_dn[0]))


def _shared64(x, gu, dn, rounded_weights):
    """(value, bound of |error|) of the shared expert on x: the activation is
    rounded to BF16 once (gate and up before it too where the GEMM path runs,
    which also rounds the scaled weights)."""
    half = ref.BF16_HALF
    act, err = ref.product(x, gu[0], gu[1], True, None)
    if rounded_weights:
        i = gu[0].shape[0] // 2
        size = x.double().abs() @ gu[0].abs().t()
        v = x.double() @ gu[0].t()
        loose = half * size + half * (v.abs() + half * size)
        g, u, ge, ue = v[:, :i], v[:, i:], loose[:, :i], loose[:, i:]
        err = err + 1.1 * ge * (u.abs() + ue) + (g * torch.sigmoid(g)).abs() * ue
    err = err + half * (act.abs() + err)
    w = dn[0].abs()
    bound = err @ w.t() + ref.sum_bound(I) * ((act.abs() + err) @ w.t())
    if dn[1] is not None:
        bound = bound + (act.abs() + err) @ dn[1].t()
    if rounded_weights:
        bound = bound + half * ((act.abs() + err) @ w.t())
    return act @ dn[0].t(), bound


def _block(p, device, tokens, shared=None, after=None):
    gu, dn = _packed(p, device)
    layer = moe_mod.W4A16MoE(
        moe_mod.PackedExperts(gu, 8, 2 * I, H, ops.W4A16_LAYOUT_KTILE64_GLU16),
        moe_mod.PackedExperts(dn, 8, H, I), 2, tokens, deterministic=True, device=device)
    gen = torch.Generator(device=device).manual_seed(3)
    nw = (1 + 0.1 * torch.randn(H, generator=gen, device=device)).to(BF)
    rw = (torch.randn(16, H, generator=gen, device=device) / H ** 0.5).to(BF)
    return moe_mod.MoEBlock(nw, rw, layer, expert_offset=4, shared=shared, after=after)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("tokens", [1, 4, 32, 33, 200])
def test_block_with_a_shared_expert(cuda_dev, kind, tokens):
    p = wl.uniform_problem(tokens, H, I, 8, 2, seed=23)
    x = bf16_tensor(p.x, cuda_dev)
    gen = torch.Generator(device=cuda_dev).manual_seed(4)
    res = torch.randn(tokens, H, generator=gen, device=cuda_dev).to(BF)

    def weight():
        return (1 + 0.1 * torch.randn(H, generator=gen, device=cuda_dev)).to(BF)
    shared, gu, dn = _shared(kind, cuda_dev, tokens)
    after = moe_mod.BlockNorm(weight(), post_weight=weight(), gate=weight(), branch_scale=0.5)
    plain = _block(p, cuda_dev, tokens)
    block = _block(p, cuda_dev, tokens, shared, after)
    experts, new_res = plain.forward(x, res)
    total, new_res2 = block.forward(x, res)
    assert torch.equal(new_res, new_res2)
    rows = ops.w4a16_add_rms_norm(x, block.norm_weight, block.eps, residual=res)[0]
    want, bound = _shared64(rows, gu, dn, kind == "int4" and tokens > 32)
    sum64 = experts.double() + want
    ref.assert_within(total, sum64, bound + ref.STEP * (sum64.abs() + bound), "sum")
    # behind the block
    y, h, y8, scales = block.forward_layer(x, res, fp8_group=ops.W4A16_FP8_GROUP)
    kw = dict(post_weight=after.post_weight, gate=after.gate, branch_scale=0.5, residual=new_res)
    check_norm(total, after.pre_weight, kw, (y, h, y8, scales), 128)
    # alone, and onto what is there
    alone = shared.forward(rows)
    ref.assert_within(alone, want, bound, "alone")
    onto = experts.clone()
    assert shared.forward(rows, out=onto, add=True) is onto
    assert torch.equal(onto, total)


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("tokens", [4, 40])
def test_the_layer_in_a_graph_and_on_a_stream(cuda_dev, kind, tokens):
    p = wl.uniform_problem(tokens, H, I, 8, 2, seed=29)
    x = bf16_tensor(p.x, cuda_dev)
    gen = torch.Generator(device=cuda_dev).manual_seed(5)
    res = torch.randn(tokens, H, generator=gen, device=cuda_dev).to(BF)
    ones = torch.ones(H, dtype=BF, device=cuda_dev)
    block = _block(p, cuda_dev, tokens, _shared(kind, cuda_dev, tokens)[0],
                   moe_mod.BlockNorm(ones, post_weight=ones))
    want = [t.clone() for t in block.forward_layer(x, res)[:2]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = block.forward_layer(x, res, stream=side)[:2]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = block.forward_layer(x, res)[:2]
    new = torch.randn(tokens, H, generator=gen, device=cuda_dev).to(BF)
    x.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    eager = block.forward_layer(x, res)[:2]
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
    assert not torch.equal(out[0], want[0])

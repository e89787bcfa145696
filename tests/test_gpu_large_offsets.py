"""Offsets that pass 32 bits, of elements or of bytes: outputs, inputs and weights of
more than 2^31 elements; rows at both ends are checked."""

import pytest
import torch

import product_reference as ref
from w4a16_int4_moe_gb300 import ops
from test_gpu_block_norm import _check as check_norm

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _ends(count, rows=40):
    return torch.cat([torch.arange(rows), torch.arange(count - rows, count)])


@pytest.mark.parametrize("gated", [False, True])
def test_dense_rows(cuda_dev, gated):
    tokens, n, k = 300_007, 8192, 64
    gen = torch.Generator(device=cuda_dev).manual_seed(1)
    x = torch.randn(tokens, k, generator=gen, device=cuda_dev).to(BF)
    w = (torch.randn(2 * n if gated else n, k, generator=gen, device=cuda_dev) / 8).to(BF)
    out = ops.w4a16_dense(x, w, gated=gated)
    at = _ends(tokens).to(cuda_dev)
    ref.check_product(out[at], x[at], w.double(), gated=gated)


def test_dense_addend(cuda_dev):
    tokens, n, k = 300_007, 7200, 64
    gen = torch.Generator(device=cuda_dev).manual_seed(2)
    x = torch.randn(tokens, k, generator=gen, device=cuda_dev).to(BF)
    w = (torch.randn(n, k, generator=gen, device=cuda_dev) / 8).to(BF)
    add = torch.randn(tokens, n, generator=gen, device=cuda_dev)
    at = _ends(tokens).to(cuda_dev)
    before = add[at].clone()
    ops.w4a16_dense(x, w, addend=add, out=add)
    ref.check_product(add[at], x[at], w.double(), addend=before)


def test_weights(cuda_dev):
    # 2^20 rows: the BF16 weight has 4 GB, the INT4 one 4.5 of them
    n = 1 << 20
    gen = torch.Generator(device=cuda_dev).manual_seed(3)
    at = _ends(n).to(cuda_dev)
    x = torch.randn(3, 2064, generator=gen, device=cuda_dev).to(BF)
    w = torch.empty(n, 2064, dtype=BF, device=cuda_dev).normal_(0, 0.02, generator=gen)
    for tokens in (3, 40):
        rows = x.repeat(20, 1)[:tokens]
        out = ops.w4a16_dense(rows, w, out_dtype=torch.float32)
        ref.check_product(out[:, at], rows, w[at].double())
    del w
    k = 8192
    x = torch.randn(3, k, generator=gen, device=cuda_dev).to(BF)
    q = torch.randint(0, 256, (1, n, k // 2), generator=gen, device=cuda_dev, dtype=torch.uint8)
    s = torch.rand(1, n, k // 32, generator=gen, device=cuda_dev).to(BF) * 0.02
    packed = ops.w4a16_prepack(q, s)
    weight, loose = ref.int4_weight(q[0][at], s[0][at])
    del q, s
    out = ops.w4a16_linear_few_tokens(x, packed, n, out_dtype=torch.float32)
    ref.check_product(out[:, at], x, weight, loose)


def test_block_norm_rows(cuda_dev):
    rows, hidden = 140_003, 16384
    gen = torch.Generator(device=cuda_dev).manual_seed(4)
    x = torch.randn(rows, hidden, generator=gen, device=cuda_dev).to(BF)
    res = torch.randn(rows, hidden, generator=gen, device=cuda_dev).to(BF)
    pre = torch.ones(hidden, dtype=BF, device=cuda_dev)
    out = ops.w4a16_block_norm(x, pre, post_weight=pre, residual=res, gate=res, fp8_group=128)
    at = _ends(rows, 4).to(cuda_dev)
    kw = dict(post_weight=pre, residual=res[at], gate=res[at])
    check_norm(x[at], pre, kw, tuple(t[at] for t in out), 128)

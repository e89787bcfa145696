"""Shared experts on rows that are a part of a wider buffer's."""

import pytest
import torch

from test_gpu_shared_block import BF, H, _shared, _shared64
import product_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("tokens", [1, 32, 33, 200])
def test_strided_rows(cuda_dev, kind, tokens):
    shared, gu, dn = _shared(kind, cuda_dev, 200)
    gen = torch.Generator(device=cuda_dev).manual_seed(31)
    wide = torch.randn(tokens, H + 40, generator=gen, device=cuda_dev).to(BF)
    x = wide[:, 16:16 + H]
    out = shared.forward(x)
    assert torch.equal(out, shared.forward(x.clone()))
    want, bound = _shared64(x, gu, dn, kind == "int4" and tokens > 32)
    ref.assert_within(out, want, bound)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = shared.forward(x, stream=side)
    side.synchronize()
    assert torch.equal(on_side, out)

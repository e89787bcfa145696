"""The 8-bit form of w4a16_add_rms_norm where its contract is exact: groups that
are not finite."""

import pytest
import torch

from w4a16_int4_moe_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8_group", [128, -1])
@pytest.mark.parametrize("kind", ["huge weight", "squares that underflow"])
def test_a_group_with_an_infinity_is_nan(cuda_dev, kind, fp8_group):
    # finite rows whose y is not: by the weight in one column, or by eps 0 and
    # a sum of squares of 0
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(5, 640, generator=gen)
    w = torch.ones(640)
    eps = 1e-6
    if kind == "huge weight":
        x[:, 300] = 30.0
        w[300] = 3e38
        bad = torch.zeros(5, 640, dtype=torch.bool)
        bad[:, 300] = True
    else:
        x[2] = 1e-30
        eps = 0.0
        bad = torch.zeros(5, 640, dtype=torch.bool)
        bad[2] = True
    y, _, y8, s = ops.w4a16_add_rms_norm(x.to(torch.bfloat16).to(cuda_dev),
                                         w.to(torch.bfloat16).to(cuda_dev), eps,
                                         fp8_group=fp8_group)
    assert torch.equal(torch.isinf(y.float()).cpu(), bad)
    group = 640 if fp8_group < 0 else fp8_group
    groups = bad.view(5, -1, group).any(-1)
    assert torch.equal(torch.isnan(s).cpu(), groups)
    assert torch.isfinite(s.cpu()[~groups]).all()
    assert torch.equal(torch.isnan(y8.float()).cpu(), groups.repeat_interleave(group, 1))

"""The norms around a block at the last row length of each count of threads and chunks
and at the first of the next, with few and with many rows."""

import pytest

from test_gpu_block_norm import _check, _inputs
from w4a16_int4_moe_gb300 import ops

pytestmark = pytest.mark.gpu

LAST = [256, 768, 1024, 1536, 2048, 2304, 4096, 5120, 6144, 7168, 8192, 10240, 12288]


@pytest.mark.parametrize("tokens", [2, 153, 620])
@pytest.mark.parametrize("hidden", LAST + [h + 8 for h in LAST])
def test_block_norm(cuda_dev, tokens, hidden):
    x32 = hidden % 16 == 0
    x, pre, kw = _inputs(cuda_dev, tokens, hidden, x32=x32, gate=1 + x32)
    for fp8_group in (0, 128, -1):
        _check(x, pre, kw, ops.w4a16_block_norm(x, pre, fp8_group=fp8_group, **kw), fp8_group)

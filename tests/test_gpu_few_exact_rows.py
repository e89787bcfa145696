"""How far below its 128-column block's largest a BF16 value is exact in the
few-token layer: down to 2^-27 of it, whichever column it stands in. The large
value meets codes of 8 (weight 0), so the output is the small one's alone, and a
rounding of its eighth bit would be 2^-8 of it (the bound is FP32's)."""

import numpy as np
import pytest

import oracle
from w4a16_int4_moe_gb300 import workloads as wl
from test_gpu_moe_few import _close, _run

pytestmark = pytest.mark.gpu


def _bits(v):
    return (np.asarray(v, np.float32).view(np.uint32) >> 16).astype(np.uint16)


@pytest.mark.parametrize("tokens", [1, 5])
@pytest.mark.parametrize("column", [32, 33, 34, 35, 63, 94, 126, 127])
@pytest.mark.parametrize("ratio,largest", [(-27, 1.0), (-27, 1.9921875), (-20, 1.0), (-27, 2.0 ** 40)])
def test_small_values_beside_a_large_one(cuda_dev, tokens, column, ratio, largest):
    p = wl.uniform_problem(tokens, 256, 64, 1, 1, seed=1)
    small = largest / (largest / 2 ** np.floor(np.log2(largest))) * 2.0 ** ratio * (1 + 2.0 ** -7)
    x = np.zeros((tokens, 256), np.float32)
    x[:, 0], x[:, column] = largest, small
    p.x = _bits(x)
    assert np.array_equal(oracle.bf16_bits_to_f64(p.x), x.astype(np.float64))
    p.q_gu = np.full_like(p.q_gu, 0x88)
    p.q_gu[..., column // 2] = 0x89 if column % 2 == 0 else 0x98
    # gate and up near 1: the scale is about 1 / small, a power of two
    p.s_gu = np.full_like(p.s_gu, _bits(2.0 ** -np.floor(np.log2(small))))
    out = _run(p, cuda_dev)
    _close(out, oracle.bf16_bits_to_f64(p.x), p.topk_ids, p.topk_weights, p)

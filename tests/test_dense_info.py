"""What w4a16_dense says of how it runs a product. No GPU needed: no call here reaches
a kernel."""

import ctypes

import pytest
import torch

import dense_sizes
from w4a16_int4_moe_gb300 import ops

OK, INV, UNS = ops.W4A16_OK, ops.W4A16_ERR_INVALID_ARG, ops.W4A16_ERR_UNSUPPORTED
# pairs, then clusters of 1, 2, 4 and 8 CTAs, of 152 SMs
WHOLE = (76, 152, 76, 36, 16)


def test_refusals(lib):
    info = ops.DenseInfo()

    def call(n=256, k=256, gated=0, tokens=64, dtype=ops.W4A16_DTYPE_F32, counts=WHOLE,
             out=ctypes.byref(info)):
        return lib.w4a16_dense_info(n, k, gated, tokens, dtype, (ctypes.c_int * 5)(*counts), out)
    assert call() == OK
    for bad in (dict(n=0), dict(k=0), dict(tokens=-1), dict(dtype=ops.W4A16_DTYPE_FP8),
                dict(out=None), dict(counts=(0, 1, 1, 1, 1)), dict(counts=(1, 1, 1, 1, 0))):
        assert call(**bad) == INV, bad
    for bad in (dict(k=252), dict(n=(1 << 20) + 1), dict(k=(1 << 20) + 8), dict(gated=1, n=255),
                dict(tokens=(1 << 24) + 1)):
        assert call(**bad) == UNS, bad


def test_few_tokens_and_runs(lib):
    i = ops.w4a16_dense_info(32, 4096, 7168, True, at_once=WHOLE)
    assert (i.kernel, i.tile_rows, i.split, i.run) == (0, 0, 0, 0)
    for tokens, n, k, gated in ((33, 64, 8, False), (200, 1000, 7168, False), (576, 4096, 7168, True),
                                (8192, 7168, 2048, False), (1 << 24, 1 << 20, 1 << 20, True)):
        assert 0 < ops.w4a16_dense_info(tokens, n, k, gated, torch.float32, WHOLE).run <= 512
        assert 0 < ops.w4a16_dense_info(tokens, n, k, gated, at_once=WHOLE).run <= 1024


@pytest.mark.parametrize("room", [WHOLE, (74, 148, 74, 34, 14)])
def test_every_kernel_width_and_split_is_taken_somewhere(lib, room):
    found = dense_sizes.sizes(room)
    assert set(found) == {(shape, *kind) for shape in dense_sizes.SHAPES
                          for kind in dense_sizes.KINDS}

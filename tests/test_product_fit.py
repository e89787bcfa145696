"""A packed weight and the rows that it is multiplied with have to fit. No GPU needed:
no call here reaches a kernel."""

import pytest
import torch

from w4a16_int4_moe_gb300 import ops
from test_product_refusals import GLU, INV, Placed, Entered

BF = torch.bfloat16


class Bytes(Placed):
    dtype = torch.uint8

    def numel(self):
        return self.shape[0]


@pytest.fixture
def on_device_0(lib, monkeypatch):
    def stream(d):
        raise Entered   # all checks of the binding are passed
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    monkeypatch.setattr(ops, "_current_stream", stream)


def _call(n, k, size, layout=0):
    columns = n // 2 if layout == GLU else n
    return ops.w4a16_linear_few_tokens(Placed(0, (4, k)), Bytes(0, (size,)), n, layout,
                                       out=Placed(0, (4, columns)))


def test_a_blob_of_another_weight_is_refused(on_device_0):
    # [300, 544] is three tiles of nine steps
    size = ops.w4a16_prepack_size(1, 300, 544)
    assert size == 3 * 9 * 4608
    with pytest.raises(Entered):
        _call(300, 544, size)
    with pytest.raises(Entered):
        _call(512, 1024, ops.w4a16_prepack_size(1, 512, 1024, layout=GLU), GLU)
    for n, k, blob, layout in ((300, 544, size - 4608, 0), (300, 544, size + 4608, 0),
                               (300, 544, 2 * size, 0),       # two experts
                               (300, 512, size, 0),           # rows with fewer columns
                               (300, 608, size, 0), (200, 544, size, 0), (0, 544, size, 0),
                               (-300, 544, size, 0), (256, 544, size, GLU)):
        with pytest.raises(ops.W4A16Error) as e:
            _call(n, k, blob, layout)
        assert e.value.status == INV, (n, k, blob)

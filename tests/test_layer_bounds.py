"""Refusals of the bindings and the layer on the host. CPU tensors stand for
device tensors; no call here reaches a kernel."""

import pytest
import torch

from w4a16_int4_moe_gb300 import ops


def test_scales_without_a_group_are_refused(lib, monkeypatch):
    monkeypatch.setattr(ops, "_rows", lambda fn, what, t: (t.data_ptr(), *t.shape, t.shape[1]))
    monkeypatch.setattr(ops, "_raw_stream", lambda t, stream: None)
    x, need = torch.zeros(4, 256, dtype=torch.bfloat16), ops._need
    monkeypatch.setattr(ops, "_need", lambda fn, what, t, *kind: need(fn, what, t, *kind)
                        if what == "scales" else t.data_ptr())
    for shape in ((4, 1), (4, 2)):
        with pytest.raises(ops.W4A16Error) as e:
            ops.w4a16_add_rms_norm(x, x[0], out=(torch.zeros_like(x), None, None,
                                                 torch.zeros(shape)))
        assert e.value.status == ops.W4A16_ERR_INVALID_ARG

"""Refusals of the bindings and the layer on the host. CPU tensors stand for
device tensors; no call here reaches a kernel."""

import pytest
import torch

from w4a16_int4_moe_gb300 import moe as moe_mod
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


@pytest.mark.parametrize("call", ["route", "route_align", "forward_from_logits", "few_tokens",
                                  "few_tokens_from_logits", "forward"])
def test_more_tokens_than_planned_are_refused(lib, monkeypatch, call):
    # the layer's own routing tensors have room for max_tokens rows
    def packed(n, k, layout):
        return moe_mod.PackedExperts(
            torch.zeros(ops.w4a16_prepack_size(8, n, k, 32, layout), dtype=torch.uint8), 8, n, k,
            layout)
    layer = moe_mod.W4A16MoE(packed(256, 256, ops.W4A16_LAYOUT_KTILE64_GLU16),
                             packed(256, 128, ops.W4A16_LAYOUT_KTILE64), 2, 4, device="cpu")
    x, w = torch.zeros(5, 256, dtype=torch.bfloat16), torch.zeros(5, 2)
    ids, logits = torch.zeros(5, 2, dtype=torch.int32), torch.zeros(5, 16)
    args = {"route": (logits,), "route_align": (logits,), "forward_from_logits": (x, logits),
            "few_tokens": (x, ids, w), "few_tokens_from_logits": (x, logits), "forward": (x, ids, w)}

    def launch(*a, **kw):
        raise AssertionError("launched")
    for name in ("w4a16_topk_softmax", "w4a16_moe_route_align", "w4a16_moe_align_block_size",
                 "w4a16_moe_few_tokens"):
        monkeypatch.setattr(ops, name, launch)
    with pytest.raises(ValueError):
        getattr(layer, call)(*args[call])

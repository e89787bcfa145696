"""Memory that a call makes for itself belongs to the stream that the call runs
on: results, temporaries, copies of strided arguments and a layer's own lazily
made buffers. (The caching allocator gives a block that another stream freed, or
takes back one that a call dropped, by the stream it was made on.)"""

import contextlib

import pytest
import torch

from w4a16_int4_moe_gb300 import moe as moe_mod
from w4a16_int4_moe_gb300 import ops


class Stream:
    cuda_stream = 17


class Library:
    """The host-only calls as they are; device calls succeed and do nothing."""

    def __init__(self, lib):
        self._lib = lib

    def __getattr__(self, name):
        if name in ("w4a16_plan", "w4a16_align_capacity", "w4a16_prepack_size",
                    "w4a16_workspace_size", "w4a16_layer_workspace_size",
                    "w4a16_moe_few_tokens_workspace_size"):
            return getattr(self._lib, name)
        return lambda *args: ops.W4A16_OK


@pytest.fixture
def made(lib, monkeypatch):
    """[(what, the stream it was made on)] of all memory made from here on."""
    log, current = [], [None]

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("empty", "zeros"):
        def make(*args, real=getattr(torch, name), name=name, **kw):
            log.append((name, current[0]))
            return real(*args, **kw)
        monkeypatch.setattr(torch, name, make)

    def contiguous(t, real=torch.Tensor.contiguous):
        if not t.is_contiguous():
            log.append(("contiguous", current[0]))
        return real(t)
    monkeypatch.setattr(torch.Tensor, "contiguous", contiguous)
    fake = Library(lib)
    monkeypatch.setattr(ops, "load_library", lambda *a: fake)
    # CPU tensors stand for device tensors
    monkeypatch.setattr(ops, "_need", lambda fn, what, t, dtype, shape: t.data_ptr())
    monkeypatch.setattr(ops, "_blob", lambda fn, what, t, size: t.data_ptr())
    monkeypatch.setattr(ops, "_rows", lambda fn, what, t: (t.data_ptr(), *t.shape, t.shape[1]))
    return log


def _on(made, stream):
    assert made and all(s is stream for _, s in made), made


BF = torch.bfloat16


def _layer(tokens, layout):
    def packed(n, k, layout):
        return moe_mod.PackedExperts(
            torch.full((ops.w4a16_prepack_size(8, n, k, 32, layout),), 0, dtype=torch.uint8), 8,
            n, k, layout)
    return moe_mod.W4A16MoE(packed(256, 256, layout), packed(256, 128, ops.W4A16_LAYOUT_KTILE64),
                            2, tokens, device="cpu")


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [4, 40])
@pytest.mark.parametrize("layout", [ops.W4A16_LAYOUT_KTILE64, ops.W4A16_LAYOUT_KTILE64_GLU16])
def test_block(made, tokens, layout, fp8, residual):
    block = moe_mod.MoEBlock(torch.ones(256, dtype=BF), torch.ones(16, 256, dtype=BF),
                             _layer(tokens, layout), fp8_rows=fp8)
    x = torch.ones(tokens, 256, dtype=BF)
    for _ in range(2):      # (the layer's routing buffers and counter come with the first call)
        made.clear()
        stream = Stream()
        block.forward(x, x.clone() if residual else None, stream=stream)
        _on(made, stream)


def test_layer(made):
    x, w = torch.ones(40, 256, dtype=BF), torch.ones(40, 2)
    ids, logits = torch.ones(40, 2, dtype=torch.int32), torch.ones(40, 16)
    for call in (lambda la, s: la.forward(x, ids, w, stream=s),
                 lambda la, s: la.experts(x, w, stream=s),
                 lambda la, s: la.route(logits, stream=s),
                 lambda la, s: la.route_align(logits, stream=s),
                 lambda la, s: la.forward_from_logits(x, logits, stream=s),
                 lambda la, s: la.few_tokens(x[:4], ids[:4], w[:4], stream=s),
                 lambda la, s: la.few_tokens_from_logits(x[:4], logits[:4], stream=s)):
        layer, stream = _layer(40, ops.W4A16_LAYOUT_KTILE64_GLU16), Stream()
        made.clear()
        call(layer, stream)
        _on(made, stream)


def test_calls(made):
    x, logits = torch.ones(8, 256, dtype=BF), torch.ones(16, 8).t()
    blob, ints = torch.full((1 << 20,), 0, dtype=torch.uint8), torch.ones(8, 2, dtype=torch.int32)
    w = torch.ones(8, 2)
    plan = ops.w4a16_plan(8, 2, 8, 256, 256)
    routing = (ints.view(-1), ints.view(-1), ints.view(-1))
    for call in (
            lambda s: ops.w4a16_add_rms_norm(x, x[0], residual=x, fp8_group=128, stream=s),
            lambda s: ops.w4a16_router_logits(x, x, stream=s),
            lambda s: ops.w4a16_moe_few_tokens(blob, blob, 8, 256, 128, x, ints, w, blob, stream=s),
            lambda s: ops.w4a16_topk_softmax(logits, 2, stream=s),
            lambda s: ops.w4a16_moe_route_align(logits, 2, 16, ints, stream=s),
            lambda s: ops.w4a16_moe_align_block_size(ints, 8, 16, stream=s),
            lambda s: ops.w4a16_prepack(blob[:8 * 64 * 32].view(8, 64, 32), blob, stream=s),
            lambda s: ops.w4a16_unpack(blob, 8, 64, 64, stream=s),
            lambda s: ops.w4a16_silu_and_mul(x, stream=s),
            lambda s: ops.w4a16_moe_layer(blob, blob, 8, 256, 128, x, 8, 2, *routing, plan, blob,
                                          w, stream=s),
            *(lambda s, mode=mode: ops.w4a16_moe_indexed_gemm(
                mode, blob, 8, 256, 256, x, 8, 2, *routing, plan, blob, stream=s)
              for mode in (ops.W4A16_GATE_UP, ops.W4A16_GATE_UP_SILU, ops.W4A16_DOWN)),
            lambda s: ops.w4a16_moe_indexed_gemm_noalloc(
                ops.W4A16_DOWN, blob, 8, 256, 256, x, 8, 2, *routing, plan, stream=s),
            lambda s: ops.w4a16_moe_grouped_gemm(ops.W4A16_GROUPED_CONTIGUOUS, blob, 8, 256, 256,
                                                 x, 8, ints, blob, plan, stream=s)):
        made.clear()
        stream = Stream()
        call(stream)
        _on(made, stream)

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


# Shared experts of 96 columns, of which 64 are as many steps of a blob, for 8 and (the
# GEMM path) for 40 tokens.

def _expert(max_tokens):
    from w4a16_int4_moe_gb300 import moe
    blob = torch.zeros(16, dtype=torch.uint8)
    expert = moe.PackedSharedExpert(moe.PackedExperts(blob, 1, 128, 96, GLU),
                                    moe.PackedExperts(blob, 1, 96, 64), min(max_tokens, 32))
    expert.max_tokens = max_tokens
    return expert


class Reached(Exception):
    pass


class Layer:
    """Stands for the routed experts' path."""
    def align(self, ids, stream=None):
        raise Reached


@pytest.mark.parametrize("tokens", [8, 40])
def test_rows_that_are_not_the_packed_shared_experts_are_refused(lib, monkeypatch, tokens):
    def product(*a, **kw):
        raise Reached
    monkeypatch.setattr(ops, "w4a16_linear_few_tokens", product)
    expert = _expert(tokens)
    expert.layer, expert.ids = Layer(), torch.zeros(tokens, 1, dtype=torch.int32)
    with pytest.raises(Reached):
        expert.forward(torch.zeros(tokens, 96, dtype=BF))
    rows = torch.zeros(tokens, 96, dtype=BF)
    for x in (rows[:, :64], rows.float(), rows[0], rows[:, None], torch.zeros(tokens, 128, dtype=BF)):
        with pytest.raises(ValueError):
            expert.forward(x)
    if tokens > ops.W4A16_FEW_TOKENS_MAX:   # (the few-token product checks its output itself)
        out = torch.zeros(tokens, 96)
        for o in (out[:, :64], out[1:], out.to(BF), torch.zeros(tokens, 192)[:, :96]):
            with pytest.raises(ValueError):
                expert.forward(rows, out=o)


def test_strided_rows_reach_the_gemm_path_as_rows_in_line(lib, monkeypatch):
    expert = _expert(40)
    seen = []

    class Seen(Layer):
        def align(self, ids, stream=None):
            pass

        def gate_up_act(self, x, tokens, stream=None):
            seen.append(x)
            raise Reached
    expert.layer, expert.ids = Seen(), torch.zeros(40, 1, dtype=torch.int32)
    wide = torch.randn(40, 200).to(BF)
    for x in (wide[:, 8:104], wide[:, :96], torch.randn(96, 40).to(BF).t()):
        with pytest.raises(Reached):
            expert.forward(x)
        assert seen[-1].is_contiguous() and torch.equal(seen[-1], x)


def test_the_gemm_path_runs_on_the_rows_device(lib, monkeypatch):
    current = [0]
    monkeypatch.setattr(ops, "_current_device", lambda: current[0])

    class device:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.before, current[0] = current[0], self.d

        def __exit__(self, *a):
            current[0] = self.before
    monkeypatch.setattr(torch.cuda, "device", device)
    expert = _expert(40)
    seen = []

    class Seen(Layer):
        def align(self, ids, stream=None):
            seen.append(current[0])
            raise Reached
    expert.layer, expert.ids = Seen(), torch.zeros(40, 1, dtype=torch.int32)
    expert.gate_up.packed = Bytes(1, (16,))
    x = Placed(1, (40, 96))
    with pytest.raises(Reached):
        expert.forward(x)
    assert seen == [1] and current == [0]
    expert.gate_up.packed = Bytes(0, (16,))     # the weights are elsewhere
    with pytest.raises(ValueError):
        expert.forward(x)
    assert seen == [1] and current == [0]

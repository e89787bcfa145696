"""Host-side refusals of the products with one weight and of the block's norms.
No GPU needed: no call here reaches a kernel."""

import contextlib

import pytest
import torch

from w4a16_int4_moe_gb300 import ops

OK, INV, UNS = ops.W4A16_OK, ops.W4A16_ERR_INVALID_ARG, ops.W4A16_ERR_UNSUPPORTED
P = 1 << 20    # never dereferenced: the checks fail first
BF16, F32, FP8 = ops.W4A16_DTYPE_BF16, ops.W4A16_DTYPE_F32, ops.W4A16_DTYPE_FP8
GLU = ops.W4A16_LAYOUT_KTILE64_GLU16


def test_linear_few_tokens_refusals(lib):
    base = dict(w=P, layout=0, n=256, k=256, x=P, xs=256, t=4, add=P, out=P + (1 << 19), dt=F32)

    def call(**kw):
        a = dict(base, **kw)
        return lib.w4a16_linear_few_tokens(a["w"], a["layout"], a["n"], a["k"], a["x"], a["xs"],
                                           a["t"], a["add"], a["out"], a["dt"], None)
    for bad in (dict(n=0), dict(n=-1), dict(k=0), dict(t=-1), dict(layout=2), dict(layout=-1),
                dict(w=None), dict(x=None), dict(out=None), dict(dt=FP8), dict(dt=7),
                dict(xs=248), dict(xs=260), dict(xs=1 << 31), dict(w=P + 8), dict(x=P + 2),
                dict(out=P + 4), dict(add=P + 4), dict(layout=GLU), dict(add=P, out=P, dt=BF16),
                dict(out=P), dict(w=2 * P, out=P), dict(x=2 * P, out=P)):
        assert call(**bad) == INV, bad
    for bad in (dict(k=240), dict(k=8), dict(t=33), dict(n=(1 << 20) + 1),
                dict(k=(1 << 20) + 32, xs=1 << 21), dict(layout=GLU, n=192, add=None)):
        assert call(**bad) == UNS, bad
    assert call(t=0, x=None, add=None, out=None) == OK
    assert call(t=0, w=None) == INV


def test_dense_refusals(lib):
    base = dict(w=P, n=256, k=256, gated=0, x=P, xs=256, t=4, add=P, out=P + (1 << 19), dt=F32)

    def call(**kw):
        a = dict(base, **kw)
        return lib.w4a16_dense(a["w"], a["n"], a["k"], a["gated"], a["x"], a["xs"], a["t"],
                               a["add"], a["out"], a["dt"], None)
    for bad in (dict(n=0), dict(k=0), dict(k=-8), dict(t=-1), dict(w=None), dict(x=None),
                dict(out=None), dict(dt=FP8), dict(xs=248), dict(xs=257), dict(xs=1 << 31),
                dict(w=P + 2), dict(x=P + 8), dict(out=P + 8), dict(add=P + 4), dict(gated=1),
                dict(add=P, out=P, dt=BF16), dict(w=2 * P, out=P), dict(x=2 * P, out=P)):
        assert call(**bad) == INV, bad
    for bad in (dict(k=252), dict(n=(1 << 20) + 1), dict(k=(1 << 20) + 8, xs=1 << 21),
                dict(t=(1 << 24) + 1), dict(gated=1, n=255, add=None)):
        assert call(**bad) == UNS, bad
    assert call(t=0, x=None, add=None, out=None) == OK


def test_block_norm_refusals(lib):
    base = dict(x=P, xt=F32, xs=256, post=P, g=P, gs=256, r=P, rs=256, pre=P, off=0.0, b=1.0,
                s=1.0, eps=1e-6, rows=4, hidden=256, out=P, h=P, o8=P, sc=P, group=128)

    def call(**kw):
        a = dict(base, **kw)
        return lib.w4a16_block_norm(
            a["x"], a["xt"], a["xs"], a["post"], a["g"], a["gs"], a["r"], a["rs"], a["pre"],
            a["off"], a["b"], a["s"], a["eps"], a["rows"], a["hidden"], a["out"], a["h"], a["o8"],
            a["sc"], a["group"], None)
    inf, nan = float("inf"), float("nan")
    for bad in (dict(rows=-1), dict(hidden=0), dict(eps=-1.0), dict(eps=nan), dict(eps=inf),
                dict(off=nan), dict(b=inf), dict(s=nan), dict(xt=FP8), dict(x=None),
                dict(pre=None), dict(o8=None), dict(sc=None), dict(group=0), dict(xs=248),
                dict(xs=260), dict(rs=248), dict(rs=260), dict(gs=248), dict(gs=260), dict(gs=-8),
                dict(x=P + 8), dict(post=P + 2), dict(g=P + 8), dict(r=P + 8), dict(pre=P + 2),
                dict(out=P + 8), dict(h=P + 4), dict(o8=P + 4), dict(sc=P + 2),
                dict(out=None, o8=None, sc=None, group=0),                       # a weight, no norm
                dict(out=None, o8=None, sc=None, group=0, pre=None, h=None),     # nothing to write
                dict(rs=264)):                                                   # h is the residual
        assert call(**bad) == INV, bad
    for bad in (dict(hidden=252), dict(hidden=16392, xs=16392, rs=16392, gs=16392),
                dict(group=64)):
        assert call(**bad) == UNS, bad
    assert call(rows=0, x=None, r=None, g=None, pre=None, out=None, h=None, o8=None,
                sc=None) == OK


def test_tensors_of_the_wrong_kind_are_refused(lib):
    # CPU tensors never reach the library, nor do wrong types, shapes or strides
    bf = torch.bfloat16
    x, w = torch.zeros(4, 256, dtype=bf), torch.zeros(8, 256, dtype=bf)
    blob = torch.zeros(128 * 256, dtype=torch.uint8)
    for args in ((x, w), (x.float(), w), (x.t(), w), (x, w[:, :128]), (x, w[0]), (x, w.float())):
        with pytest.raises(ops.W4A16Error) as e:
            ops.w4a16_dense(*args)
        assert e.value.status == INV
    for args in ((x, blob, 8), (x[0], blob, 8), (x, blob[:16], 8), (x, blob.float(), 8)):
        with pytest.raises(ops.W4A16Error) as e:
            ops.w4a16_linear_few_tokens(*args)
        assert e.value.status == INV
    v = torch.zeros(256, dtype=bf)
    for args, kw in (((x, v), {}), ((x.double(), v), {}), ((x.float(), v[:128]), {}),
                     ((x, v), dict(gate=v)), ((x, None), {})):
        with pytest.raises(ops.W4A16Error) as e:
            ops.w4a16_block_norm(*args, **kw)
        assert e.value.status == INV


class Placed:
    """Stands for a matrix on a device."""
    dtype = torch.bfloat16

    def __init__(self, device, shape=(4, 256)):
        self.index, self.device, self.shape = device, f"cuda:{device}", torch.Size(shape)

    def get_device(self):
        return self.index

    def dim(self):
        return len(self.shape)

    is_cuda = True

    def is_contiguous(self):
        return True

    def stride(self):
        return (self.shape[-1], 1)

    def data_ptr(self):
        return P


class Entered(Exception):
    pass


def test_the_tensors_device_is_made_current(lib, monkeypatch):
    current = [0]
    monkeypatch.setattr(ops, "_current_device", lambda: current[0])

    @contextlib.contextmanager
    def device(d):
        before, current[0] = current[0], d
        try:
            yield
        finally:
            current[0] = before
    monkeypatch.setattr(torch.cuda, "device", device)

    def stream(d):
        assert current[0] == d == 1
        raise Entered
    monkeypatch.setattr(ops, "_current_stream", stream)
    x, w, v = Placed(1), Placed(1, (8, 256)), Placed(1, (256,))
    with pytest.raises(Entered):
        ops.w4a16_dense(x, w, out=Placed(1, (4, 8)))
    with pytest.raises(Entered):
        ops.w4a16_block_norm(x, v, out=(Placed(1), Placed(1), None, None))
    assert current == [0]
    # on two devices: refused
    for call in (lambda: ops.w4a16_dense(x, Placed(0, (8, 256)), out=Placed(1, (4, 8))),
                 lambda: ops.w4a16_dense(x, w, out=Placed(0, (4, 8))),
                 lambda: ops.w4a16_block_norm(x, Placed(0, (256,)), out=(x, x, None, None)),
                 lambda: ops.w4a16_block_norm(x, v, residual=Placed(2), out=(x, x, None, None))):
        with pytest.raises(ops.W4A16Error) as e:
            call()
        assert e.value.status == INV


def test_shared_experts_that_do_not_fit_are_refused(lib):
    from w4a16_int4_moe_gb300 import moe
    bf = torch.bfloat16
    gu, dn = torch.zeros(128, 96, dtype=bf), torch.zeros(96, 64, dtype=bf)
    assert moe.SharedExpert(gu, dn).hidden == 96
    for bad in ((gu, dn.t()), (gu[:64], dn), (gu[:, :64], dn), (gu[0], dn)):
        with pytest.raises(ValueError):
            moe.SharedExpert(*bad)
    blob = torch.zeros(16, dtype=torch.uint8)
    glu = moe.PackedExperts(blob, 1, 128, 96, GLU)
    packed = moe.PackedExperts(blob, 1, 96, 64)
    expert = moe.PackedSharedExpert(glu, packed, 8)
    with pytest.raises(ValueError):
        expert.forward(torch.zeros(9, 96, dtype=bf))
    for e in (expert, moe.SharedExpert(gu, dn)):   # nothing to add to
        with pytest.raises(ValueError):
            e.forward(torch.zeros(1, 96, dtype=bf), add=True)
    for bad in ((moe.PackedExperts(blob, 1, 128, 96), packed),
                (glu, moe.PackedExperts(blob, 1, 96, 96)),
                (moe.PackedExperts(blob, 2, 128, 96, GLU), packed),
                (glu, moe.PackedExperts(blob, 2, 96, 64))):
        with pytest.raises(ValueError):
            moe.PackedSharedExpert(*bad, 8)

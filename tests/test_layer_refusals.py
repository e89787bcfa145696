"""Host-side refusals of the norm, the router's product and the few-token
layer. No GPU needed: no call here reaches a kernel."""

import pytest
import torch

from w4a16_int4_moe_gb300 import ops

OK, INV, UNS, WS = (ops.W4A16_OK, ops.W4A16_ERR_INVALID_ARG, ops.W4A16_ERR_UNSUPPORTED,
                    ops.W4A16_ERR_WORKSPACE)
P = 1 << 20    # never dereferenced: the checks fail first


def test_norm_refusals(lib):
    base = dict(x=P, xs=256, r=P, rs=256, w=P, eps=1e-6, rows=4, hidden=256, out=P, ro=P, o8=P,
                sc=P, group=128)

    def call(**kw):
        a = dict(base, **kw)
        return lib.w4a16_add_rms_norm(a["x"], a["xs"], a["r"], a["rs"], a["w"], a["eps"],
                                      a["rows"], a["hidden"], a["out"], a["ro"], a["o8"], a["sc"],
                                      a["group"], None)
    for bad in (dict(rows=-1), dict(hidden=0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(x=None), dict(w=None), dict(r=None), dict(ro=None),
                dict(o8=None), dict(sc=None), dict(group=0), dict(xs=248), dict(xs=260),
                dict(rs=248), dict(rs=260), dict(x=P + 2), dict(r=P + 8), dict(w=P + 2),
                dict(out=P + 8), dict(ro=P + 4), dict(o8=P + 4), dict(sc=P + 2),
                dict(out=None, o8=None, sc=None, group=0),
                dict(ro=P, rs=264)):
        assert call(**bad) == INV, bad
    for bad in (dict(hidden=252), dict(hidden=16392, xs=16392, rs=16392), dict(group=64)):
        assert call(**bad) == UNS, bad
    assert call(rows=0, x=None, r=None, ro=None, w=None, out=None, o8=None, sc=None) == OK


def test_router_refusals(lib):
    base = dict(x=P, xs=256, w=P, t=4, h=256, e=8, out=P)

    def call(**kw):
        a = dict(base, **kw)
        return lib.w4a16_router_logits(a["x"], a["xs"], a["w"], a["t"], a["h"], a["e"], a["out"],
                                       None)
    for bad in (dict(t=-1), dict(h=0), dict(e=0), dict(x=None), dict(w=None), dict(out=None),
                dict(xs=248), dict(xs=257), dict(x=P + 8), dict(w=P + 2), dict(out=P + 2)):
        assert call(**bad) == INV, bad
    for bad in (dict(h=252), dict(e=1025)):
        assert call(**bad) == UNS, bad
    assert call(t=0, x=None, out=None) == OK


def test_few_tokens_refusals(lib):
    need = ops.w4a16_moe_few_tokens_workspace_size(4, 2, 256, 128)
    base = dict(gu=P, dn=P, E=8, H=256, I=128, x=P, xt=ops.W4A16_DTYPE_BF16, xs=None, t=4, k=2,
                lg=P, lt=ops.W4A16_DTYPE_F32, eg=16, ids=P, w=P, out=P, flags=0, ws=P, wsb=need)

    def call(**kw):
        a = dict(base, **kw)
        return lib.w4a16_moe_few_tokens(
            a["gu"], a["dn"], a["E"], a["H"], a["I"], a["x"], a["xt"], a["xs"], a["t"], a["k"],
            a["lg"], a["lt"], a["eg"], 1, 0, a["ids"], a["w"], a["out"], a["flags"], a["ws"],
            a["wsb"], None)
    for bad in (dict(E=0), dict(H=0), dict(I=-1), dict(t=-1), dict(k=0), dict(gu=None),
                dict(dn=None), dict(x=None), dict(ids=None), dict(w=None), dict(out=None),
                dict(xt=ops.W4A16_DTYPE_F32), dict(xt=ops.W4A16_DTYPE_FP8), dict(xs=P),
                dict(lt=ops.W4A16_DTYPE_FP8), dict(eg=0), dict(flags=1), dict(flags=8),
                dict(gu=P + 8), dict(dn=P + 4), dict(x=P + 2), dict(out=P + 4), dict(ws=P + 8)):
        assert call(**bad) == INV, bad
    for bad in (dict(H=240), dict(I=96), dict(t=33), dict(k=33), dict(E=1025), dict(eg=1025),
                dict(eg=1), dict(H=1 << 21), dict(I=1 << 21)):
        assert call(**bad) == UNS, bad
    assert call(ws=None) == WS and call(wsb=need - 1) == WS
    assert call(t=0, x=None, ids=None, w=None, out=None, ws=None, wsb=0) == OK
    assert ops.w4a16_moe_few_tokens_workspace_size(-1, 2, 256, 128) == 0
    assert ops.w4a16_moe_few_tokens_workspace_size(1, 2, 0, 128) == 0
    # a workspace for more tokens serves fewer
    sizes = [ops.w4a16_moe_few_tokens_workspace_size(t, 8, 7168, 2048) for t in range(1, 33)]
    assert sizes == sorted(sizes)


def test_tensors_of_the_wrong_kind_are_refused(lib):
    # CPU tensors never reach the library, nor do wrong types, shapes or strides
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    x, w = torch.zeros(4, 256, dtype=bf), torch.zeros(256, dtype=bf)
    for args in ((x, w), (x.float(), w), (x.t(), w), (x, w[:128]), (x, w.float())):
        with pytest.raises(ops.W4A16Error) as e:
            ops.w4a16_add_rms_norm(*args)
        assert e.value.status == INV
    with pytest.raises(ops.W4A16Error):
        ops.w4a16_router_logits(x, torch.zeros(8, 256, dtype=bf))
    ids, wt = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    blob = torch.zeros(16, dtype=torch.uint8)
    for x_, kw in ((x, {}), (x.to(f8), {}), (x, dict(x_scales=torch.zeros(4, 2))),
                   (x[:3], {}), (x, dict(logits=torch.zeros(4, 8)))):
        with pytest.raises(ops.W4A16Error):
            ops.w4a16_moe_few_tokens(blob, blob, 8, 256, 128, x_, ids, wt, blob, **kw)


def test_few_tokens_alignment(lib):
    need = ops.w4a16_moe_few_tokens_workspace_size(4, 2, 256, 128)
    base = dict(xt=ops.W4A16_DTYPE_FP8, xs=P, lg=P, lt=ops.W4A16_DTYPE_F32, ids=P, w=P)
    for bad in (dict(xs=P + 2), dict(lg=P + 2), dict(lg=P + 1, lt=ops.W4A16_DTYPE_BF16),
                dict(ids=P + 1), dict(w=P + 2)):
        a = dict(base, **bad)
        assert lib.w4a16_moe_few_tokens(P, P, 8, 256, 128, P, a["xt"], a["xs"], 4, 2, a["lg"],
                                        a["lt"], 16, 1, 0, a["ids"], a["w"], P, 0, P, need,
                                        None) == INV, bad

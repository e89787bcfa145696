"""The whole layer for a few tokens (w4a16_moe_few_tokens) against the 64-bit
layer. Two bounds hold: every element within the counted roundings of its own
sums (layer_reference.few_layer), and the whole output within a relative L2 of
2^-16: a sum of n terms with independent roundings loses about sqrt(n / 16)
half steps, under 2^6 of them for the sizes here, and the three chained steps
(two products and the activation) at most 2^2 times that."""

import numpy as np
import pytest
import torch

import layer_reference as ref
import oracle
from w4a16_int4_moe_gb300 import moe as moe_mod
from w4a16_int4_moe_gb300 import ops
from w4a16_int4_moe_gb300 import workloads as wl
from helpers import Guarded, bf16_tensor, dev

pytestmark = pytest.mark.gpu

REL_L2 = 2.0 ** -16


def _packed(p, device):
    gu = ops.w4a16_prepack(dev(p.q_gu, device), dev(p.s_gu.view(np.int16), device),
                           layout=ops.W4A16_LAYOUT_KTILE64_GLU16)
    dn = ops.w4a16_prepack(dev(p.q_dn, device), dev(p.s_dn.view(np.int16), device))
    return gu, dn


def _workspace(p, device):
    return torch.zeros(ops.w4a16_moe_few_tokens_workspace_size(p.tokens, p.topk, p.hidden, p.inter),
                       dtype=torch.uint8, device=device)


def _close(got, x, ids, weights, p):
    want, bound = ref.few_layer(x, ids, weights, p)
    got = got.cpu().numpy().astype(np.float64)
    ref.assert_within(got, want, bound, "out")
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= REL_L2 * norm, np.linalg.norm(got - want) / norm


def _run(p, device, ids=None, weights=None, packed=None, ws=None, **kw):
    gu, dn = packed or _packed(p, device)
    ids = p.topk_ids if ids is None else ids
    weights = p.topk_weights if weights is None else weights
    ws = _workspace(p, device) if ws is None else ws
    x = kw.pop("x", None)
    out = ops.w4a16_moe_few_tokens(
        gu, dn, p.num_experts, p.hidden, p.inter, bf16_tensor(p.x, device) if x is None else x,
        dev(ids, device), dev(weights, device), ws, **kw)
    st, word = ops.w4a16_read_device_status(ws)
    assert st == ops.W4A16_OK, hex(word)
    return out


SIZES = [  # tokens, hidden, inter, experts, topk
    (1, 32, 64, 1, 1), (1, 512, 512, 8, 2), (2, 96, 64, 3, 3), (3, 1056, 192, 12, 3),
    (5, 160, 128, 7, 2), (8, 512, 256, 8, 8), (9, 544, 320, 6, 2), (16, 1024, 512, 16, 4),
    (17, 2080, 64, 40, 5), (32, 512, 512, 8, 2), (32, 224, 128, 4, 4), (31, 7168, 256, 4, 2),
    (1, 7168, 2048, 3, 2), (4, 256, 4096, 2, 1), (32, 64, 64, 300, 32),
]


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", SIZES)
def test_layer(cuda_dev, tokens, hidden, inter, experts, topk):
    p = wl.uniform_problem(tokens, hidden, inter, experts, topk, seed=tokens + hidden)
    out = _run(p, cuda_dev)
    _close(out, oracle.bf16_bits_to_f64(p.x), p.topk_ids, p.topk_weights, p)


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", SIZES)
def test_layer_fp8_rows(cuda_dev, tokens, hidden, inter, experts, topk):
    p = wl.uniform_problem(tokens, hidden, inter, experts, topk, seed=tokens + hidden + 1)
    rng = np.random.default_rng(hidden)
    groups = -(-hidden // 128)
    values = rng.standard_normal((tokens, hidden)) * 100
    codes = torch.from_numpy(values.clip(-448, 448)).to(torch.float8_e4m3fn)
    scales = np.exp2(rng.uniform(-9, -5, (tokens, groups))).astype(np.float32)
    out = _run(p, cuda_dev, x=codes.to(cuda_dev), x_scales=dev(scales, cuda_dev))
    x = codes.to(torch.float64).numpy() * np.repeat(scales.astype(np.float64), 128, 1)[:, :hidden]
    _close(out, x, p.topk_ids, p.topk_weights, p)


@pytest.mark.parametrize("tokens", [1, 8, 13, 32])
@pytest.mark.parametrize("kind", ["one expert", "same slot twice", "none", "one local", "out of range"])
def test_routings(cuda_dev, tokens, kind):
    # every token on one expert (more rows than a tile holds); an expert twice
    # in one token's list; no local expert at all; one local pick in all
    p = wl.uniform_problem(tokens, 288, 128, 6, 2, seed=7)
    ids = p.topk_ids.copy()
    if kind == "one expert":
        ids[:, 0] = 4
        ids[:, 1] = -1
    elif kind == "same slot twice":
        ids[:, :] = 2
    elif kind == "none":
        ids[:, :] = -1
    elif kind == "one local":
        ids[:, :] = -1
        ids[tokens // 2, 1] = 5
    else:
        ids[::2, 0] = 6
        ids[1::2, 1] = 2 ** 31 - 1
        ids[0, 1] = -(2 ** 31)
    out = _run(p, cuda_dev, ids=ids)
    if kind == "none":
        assert out.abs().max() == 0
    else:
        _close(out, oracle.bf16_bits_to_f64(p.x), ids, p.topk_weights, p)
        idle = ~((ids >= 0) & (ids < 6)).any(1)
        assert np.all(out.cpu().numpy()[idle] == 0)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("tokens,experts,local,offset,topk,renorm", [
    (1, 384, 48, 48, 8, True), (32, 384, 48, 336, 8, True), (7, 20, 12, 8, 3, False),
    (32, 1024, 16, 500, 32, True), (3, 5, 5, 0, 5, False),
])
def test_from_logits(cuda_dev, tokens, experts, local, offset, topk, renorm, bf16):
    p = wl.uniform_problem(tokens, 192, 64, local, 1, seed=experts)
    p.topk = topk
    lg = np.random.default_rng(tokens).standard_normal((tokens, experts)).astype(np.float32)
    if bf16:
        lg = np.round(lg * 4) / 4            # ties: the lower expert first
    t = torch.from_numpy(lg).to(torch.bfloat16 if bf16 else torch.float32).to(cuda_dev)
    ids = torch.empty(tokens, topk, dtype=torch.int32, device=cuda_dev)
    w = torch.empty(tokens, topk, device=cuda_dev)
    gu, dn = _packed(p, cuda_dev)
    ws = _workspace(p, cuda_dev)
    out = ops.w4a16_moe_few_tokens(gu, dn, local, p.hidden, p.inter, bf16_tensor(p.x, cuda_dev),
                                   ids, w, ws, logits=t, renormalize=renorm, expert_offset=offset)
    rid, rw = oracle.topk_softmax(lg.astype(np.float64), topk, renorm, offset, local)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=1e-5, atol=1e-8)
    _close(out, oracle.bf16_bits_to_f64(p.x), rid, w.cpu().numpy(), p)


def test_masked_logits(cuda_dev):
    # -inf and the type's lowest value: rows with fewer experts than slots,
    # and a row with none
    p = wl.uniform_problem(12, 128, 64, 16, 1, seed=3)
    p.topk = 4
    rng = np.random.default_rng(8)
    lg = np.full((12, 16), -np.inf, dtype=np.float32)
    for t in range(12):
        keep = rng.choice(16, size=t % 6, replace=False)
        lg[t, keep] = rng.standard_normal(keep.size)
    ids = torch.empty(12, 4, dtype=torch.int32, device=cuda_dev)
    w = torch.empty(12, 4, device=cuda_dev)
    gu, dn = _packed(p, cuda_dev)
    out = ops.w4a16_moe_few_tokens(gu, dn, 16, p.hidden, p.inter, bf16_tensor(p.x, cuda_dev), ids,
                                   w, _workspace(p, cuda_dev), logits=dev(lg, cuda_dev))
    plain = ops.w4a16_topk_softmax(dev(lg, cuda_dev), 4)
    assert torch.equal(ids, plain[0]) and torch.equal(w, plain[1])
    assert out[0].abs().max() == 0 and out[6].abs().max() == 0
    _close(out, oracle.bf16_bits_to_f64(p.x), ids.cpu().numpy(), w.cpu().numpy(), p)


def test_accumulate_repeat_and_workspace_reuse(cuda_dev):
    # the bits of a call do not change when it is repeated, when the workspace
    # has served other sizes, or when it lies on another stream
    p = wl.uniform_problem(24, 1056, 192, 10, 3, seed=5)
    packed, ws = _packed(p, cuda_dev), _workspace(p, cuda_dev)
    first = _run(p, cuda_dev, packed=packed, ws=ws)
    q = wl.uniform_problem(3, 1056, 192, 10, 3, seed=6)
    q.q_gu, q.s_gu, q.q_dn, q.s_dn = p.q_gu, p.s_gu, p.q_dn, p.s_dn
    small = _run(q, cuda_dev, packed=packed, ws=ws)
    for _ in range(20):
        assert torch.equal(_run(p, cuda_dev, packed=packed, ws=ws), first)
        assert torch.equal(_run(q, cuda_dev, packed=packed, ws=ws), small)
    base = torch.randn(24, 1056, device=cuda_dev)
    got = _run(p, cuda_dev, packed=packed, ws=ws, out=base.clone(),
               flags=ops.W4A16_FLAG_ACCUMULATE)
    assert torch.equal(got, base + first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert torch.equal(_run(p, cuda_dev, packed=packed, ws=ws), first)


def test_back_to_back_calls_and_a_graph(cuda_dev):
    p = wl.uniform_problem(6, 512, 256, 8, 2, seed=15)
    gu, dn = _packed(p, cuda_dev)
    layer = moe_mod.W4A16MoE(
        moe_mod.PackedExperts(gu, 8, 512, 512, ops.W4A16_LAYOUT_KTILE64_GLU16),
        moe_mod.PackedExperts(dn, 8, 512, 256), 2, 32, device=cuda_dev)
    x = bf16_tensor(p.x, cuda_dev)
    ids, w = dev(p.topk_ids, cuda_dev), dev(p.topk_weights, cuda_dev)
    want = layer.few_tokens(x, ids, w).clone()
    outs = [torch.empty_like(want) for _ in range(50)]
    for o in outs:
        layer.few_tokens(x, ids, w, out=o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.few_tokens(x, ids, w, out=out)
        layer.few_tokens(x, ids, w, out=outs[0])
    for _ in range(3):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(outs[0], want)


@pytest.mark.parametrize("tokens", [2, 20])
def test_a_token_that_is_not_finite_stays_alone(cuda_dev, tokens):
    p = wl.uniform_problem(tokens, 544, 128, 6, 2, seed=11)
    packed, x = _packed(p, cuda_dev), bf16_tensor(p.x, cuda_dev)
    clean = _run(p, cuda_dev, packed=packed, x=x)
    x = x.clone()
    x[1, 543] = float("nan")
    got = _run(p, cuda_dev, packed=packed, x=x)
    keep = [t for t in range(tokens) if t != 1]
    assert torch.equal(got[keep], clean[keep]) and torch.isnan(got[1]).all()


def test_no_tokens(cuda_dev):
    p = wl.uniform_problem(4, 128, 64, 4, 2, seed=1)
    gu, dn = _packed(p, cuda_dev)
    out = ops.w4a16_moe_few_tokens(
        gu, dn, 4, 128, 64, torch.empty(0, 128, dtype=torch.bfloat16, device=cuda_dev),
        torch.empty(0, 2, dtype=torch.int32, device=cuda_dev),
        torch.empty(0, 2, device=cuda_dev), _workspace(p, cuda_dev))
    assert out.shape == (0, 128)


@pytest.mark.parametrize("tokens,hidden,inter,experts,topk", [(1, 96, 64, 3, 2), (19, 544, 192, 5, 3)])
def test_writes_only_its_buffers(cuda_dev, tokens, hidden, inter, experts, topk):
    p = wl.uniform_problem(tokens, hidden, inter, experts, topk, seed=2)
    lg = np.random.default_rng(4).standard_normal((tokens, experts)).astype(np.float32)
    gu, dn = _packed(p, cuda_dev)
    size = ops.w4a16_moe_few_tokens_workspace_size(tokens, topk, hidden, inter)
    g = {"workspace": Guarded(size, torch.uint8, cuda_dev, fill=0),
         "out": Guarded((tokens, hidden), torch.float32, cuda_dev),
         "topk_ids": Guarded((tokens, topk), torch.int32, cuda_dev),
         "topk_weights": Guarded((tokens, topk), torch.float32, cuda_dev)}
    out = ops.w4a16_moe_few_tokens(
        gu, dn, experts, hidden, inter, bf16_tensor(p.x, cuda_dev), g["topk_ids"].t,
        g["topk_weights"].t, g["workspace"].t, logits=dev(lg, cuda_dev), out=g["out"].t)
    for what, b in g.items():
        b.check(what)
    _close(out, oracle.bf16_bits_to_f64(p.x), g["topk_ids"].t.cpu().numpy(),
           g["topk_weights"].t.cpu().numpy(), p)


@pytest.mark.parametrize("tokens", [1, 32, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_block_runs_norm_router_and_experts(cuda_dev, tokens, fp8):
    # the three operators chained (few tokens), or in front of the GEMM path
    # (more), against the 64-bit chain on the routing the device chose
    p = wl.uniform_problem(tokens, 512, 256, 8, 2, seed=21)
    gu, dn = _packed(p, cuda_dev)
    layer = moe_mod.W4A16MoE(
        moe_mod.PackedExperts(gu, 8, 512, 512, ops.W4A16_LAYOUT_KTILE64_GLU16),
        moe_mod.PackedExperts(dn, 8, 512, 256), 2, tokens, device=cuda_dev)
    gen = torch.Generator().manual_seed(3)
    nw = (1 + 0.1 * torch.randn(512, generator=gen)).to(torch.bfloat16).to(cuda_dev)
    rw = (torch.randn(16, 512, generator=gen) / 512 ** 0.5).to(torch.bfloat16).to(cuda_dev)
    res = torch.randn(tokens, 512, generator=gen).to(torch.bfloat16).to(cuda_dev)
    x = bf16_tensor(p.x, cuda_dev)
    block = moe_mod.MoEBlock(nw, rw, layer, expert_offset=4, fp8_rows=fp8)
    out, new_res = block.forward(x, res)
    h, y = ref.norm(x.double().cpu().numpy(), res.double().cpu().numpy(),
                    nw.double().cpu().numpy(), 1e-6)
    assert np.abs(new_res.double().cpu().numpy() - h).max() <= np.abs(h).max() * ref.BF16_HALF
    ids = layer._route_ids[:tokens].cpu().numpy()
    weights = layer._route_w[:tokens].cpu().numpy()
    want, _ = ref.few_layer(y, ids, weights, p)
    # inputs of the experts are rounded once (BF16 half a step, e4m3 half a
    # step), the GEMM path rounds weights and activations to BF16 as well
    half = ref.E4M3_HALF if fp8 and tokens <= ops.W4A16_FEW_TOKENS_MAX else 4 * ref.BF16_HALF
    got = out.cpu().numpy().astype(np.float64)
    assert np.linalg.norm(got - want) <= half * np.linalg.norm(want)


def test_expired_waits_are_reported_and_the_next_call_is_right(cuda_dev, monkeypatch):
    # a bound far below the time of the first weight copy: the waits run out,
    # every warp still ends, the status says so, and the counters are clean
    p = wl.uniform_problem(9, 2048, 512, 8, 2, seed=41)
    packed, ws = _packed(p, cuda_dev), _workspace(p, cuda_dev)
    want = _run(p, cuda_dev, packed=packed, ws=ws)
    monkeypatch.setenv("W4A16_WAIT_TIMEOUT_CYCLES", "100")
    ops.w4a16_moe_few_tokens(packed[0], packed[1], 8, 2048, 512, bf16_tensor(p.x, cuda_dev),
                             dev(p.topk_ids, cuda_dev), dev(p.topk_weights, cuda_dev), ws)
    st, word = ops.w4a16_read_device_status(ws)
    assert st == ops.W4A16_ERR_TIMEOUT and 0x1021 <= word <= 0x1025, hex(word)
    monkeypatch.delenv("W4A16_WAIT_TIMEOUT_CYCLES")
    assert torch.equal(_run(p, cuda_dev, packed=packed, ws=ws), want)


def test_first_call_inside_a_capture_that_is_never_replayed(cuda_dev):
    # the layer's workspace is zero from its construction on
    p = wl.uniform_problem(6, 512, 256, 8, 2, seed=15)
    gu, dn = _packed(p, cuda_dev)
    layer = moe_mod.W4A16MoE(
        moe_mod.PackedExperts(gu, 8, 512, 512, ops.W4A16_LAYOUT_KTILE64_GLU16),
        moe_mod.PackedExperts(dn, 8, 512, 256), 2, 32, device=cuda_dev)
    x = bf16_tensor(p.x, cuda_dev)
    ids, w = dev(p.topk_ids, cuda_dev), dev(p.topk_weights, cuda_dev)
    out = torch.zeros(6, 512, device=cuda_dev)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.few_tokens(x, ids, w, out=out)
    assert not layer.few_workspace.any()
    _close(layer.few_tokens(x, ids, w), oracle.bf16_bits_to_f64(p.x), p.topk_ids, p.topk_weights, p)
    graph.replay()
    assert torch.equal(out, layer.few_tokens(x, ids, w))


def test_short_weights_and_foreign_workspaces_are_refused(cuda_dev):
    # on the host: nothing is launched
    p = wl.uniform_problem(4, 256, 128, 3, 2, seed=5)
    (gu, dn), ws = _packed(p, cuda_dev), _workspace(p, cuda_dev)
    for packed, space in (((gu[:-1], dn), ws), ((gu, dn[:-1]), ws), ((gu.cpu(), dn), ws),
                          ((gu, dn), ws.cpu()), ((gu, dn), ws[:-1]), ((gu, dn), ws[16:])):
        with pytest.raises(ops.W4A16Error):
            _run(p, cuda_dev, packed=packed, ws=space)

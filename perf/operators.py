"""The MoE half of a decoder layer around the expert pair: the residual's
addition with the RMS norm (BF16 and 8-bit outputs), the router's product and
the whole expert layer for a few tokens.

``own`` selects what ``run`` computes with: the plain torch forms, or the
library's entry points. Shapes are the library's own shard shapes (hidden
7168, 384 experts, top-8; EP8 holds 48 experts of intermediate 2048, TP8 all
384 of intermediate 256) and generic small or ragged ones.
"""

from __future__ import annotations

import math

import torch

own = False

F8 = torch.float8_e4m3fn
EPS = 1e-6
GROUP = 128          # columns that share a scale of the 8-bit form


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoding sequence: the norm in front of the experts, latency only
        _norm("norm_one", 1, 7168, residual=True, bf16=True, fp8=0, pitch=0),
        # a decode batch whose normed rows also leave in 8 bits for the exchange between GPUs
        _norm("norm_decode_fp8", 576, 7168, residual=True, bf16=True, fp8=128, pitch=0),
        # ragged: rows of a wider buffer, a hidden size that is no multiple of a group, one scale a row
        _norm("norm_ragged_fp8", 1021, 2088, residual=False, bf16=False, fp8=-1, pitch=2400),
        # a prefill chunk, everything written
        _norm("norm_prefill_fp8", 8192, 7168, residual=True, bf16=True, fp8=128, pitch=0),
        # one decoding sequence: the router reads its whole weight
        _router("router_one", 1, 7168, 384, pitch=0),
        # a small decode batch
        _router("router_decode", 48, 7168, 384, pitch=0),
        # ragged rows, experts and hidden size
        _router("router_ragged", 777, 2088, 60, pitch=2400),
        # a prefill chunk: a real dense product
        _router("router_prefill", 8192, 7168, 384, pitch=0),
        # one decoding sequence on the TP8 shard: eight slim experts
        _moe("moe_tp8_one", 1, 7168, 256, 384, 384, 8, fp8=False, bf16_logits=False),
        # a small batch on the TP8 shard: about a hundred experts with one or two rows each
        _moe("moe_tp8_16", 16, 7168, 256, 384, 384, 8, fp8=False, bf16_logits=False),
        # the EP8 shard at its few-token limit, rows that came in 8 bits
        _moe("moe_ep8_32_fp8", 32, 7168, 2048, 48, 384, 8, fp8=True, bf16_logits=False),
        # small ragged experts: odd hidden and intermediate sizes, logits in BF16
        _moe("moe_ragged", 5, 1056, 192, 12, 20, 3, fp8=False, bf16_logits=True),
    ]


def _norm(name, tokens, hidden, residual, bf16, fp8, pitch):
    c = {"op": "norm", "tokens": tokens, "hidden": hidden, "residual": residual, "bf16": bf16,
         "fp8": fp8, "pitch": pitch}
    return dict(c, name=name) if name else c


def _router(name, tokens, hidden, experts, pitch):
    c = {"op": "router", "tokens": tokens, "hidden": hidden, "experts": experts, "pitch": pitch}
    return dict(c, name=name) if name else c


def _moe(name, tokens, hidden, inter, local, experts, topk, fp8, bf16_logits):
    c = {"op": "moe", "tokens": tokens, "hidden": hidden, "inter": inter, "local": local,
         "experts": experts, "topk": topk, "fp8": fp8, "bf16_logits": bf16_logits}
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "router", "moe"])
    if op == "norm":
        tokens, hidden = _log(rng, 1, 8192), 8 * _log(rng, 8, 896)
        bf16 = rng.random() < 0.7
        return _norm("", tokens, hidden, rng.random() < 0.7, bf16,
                     rng.choice([0, 128, -1]) if bf16 else rng.choice([128, -1]),
                     hidden + 8 * rng.randint(1, 64) if rng.random() < 0.3 else 0)
    if op == "router":
        hidden = 8 * _log(rng, 16, 896)
        return _router("", _log(rng, 1, 8192), hidden, min(384, _log(rng, 2, 400)),
                       hidden + 8 * rng.randint(1, 64) if rng.random() < 0.3 else 0)
    kind, tokens = rng.choice(["tp8", "ep8", "small"]), _log(rng, 1, 32)
    fp8, bf16_logits = rng.random() < 0.4, rng.random() < 0.3
    if kind == "tp8":
        return _moe("", min(tokens, 24), 7168, 256, 384, 384, 8, fp8, bf16_logits)
    if kind == "ep8":
        return _moe("", tokens, 7168, 2048, 48, 384, 8, fp8, bf16_logits)
    local = _log(rng, 4, 64)
    experts = local * rng.choice([1, 2, 8])
    return _moe("", tokens, 32 * _log(rng, 4, 96), 64 * _log(rng, 1, 16), local, experts,
                rng.randint(1, min(8, local)), fp8, bf16_logits)


def work(case):
    t, h = case["tokens"], case["hidden"]
    if case["op"] == "norm":
        per = 2 + (4 if case["residual"] else 0) + (2 if case["bf16"] else 0)
        n = t * h * per + 2 * h
        if case["fp8"]:
            n += t * h + 4 * t * _groups(h, case["fp8"])
        return {"bytes": n, "flops": 6 * t * h}
    if case["op"] == "router":
        e = case["experts"]
        return {"bytes": 2 * t * h + 2 * e * h + 4 * t * e, "flops": 2 * t * h * e}
    i, local, e, k = case["inter"], case["local"], case["experts"], case["topk"]
    used = local * (1 - (1 - k / e) ** t)          # experts of this GPU that some token chose
    weights = used * 3 * i * h * (0.5 + 2 / 32)    # codes and group scales
    rows = t * h * (1 if case["fp8"] else 2) + t * e * (2 if case["bf16_logits"] else 4)
    return {"bytes": int(weights + rows + 4 * t * h + 8 * t * k),
            "flops": int(6 * i * h * t * k * local / e)}


def _groups(hidden, fp8):
    return 1 if fp8 < 0 else -(-hidden // fp8)


# ----------------------------------------------------------------- inputs --

def _rows(gen, case, spread):
    """BF16 rows of normal values; with a pitch, the first columns of a wider buffer."""
    t, h = case["tokens"], case["hidden"]
    wide = torch.randn(t, case["pitch"] or h, generator=gen, device="cuda") * spread
    return wide.to(torch.bfloat16)[:, :h]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t, h = case["tokens"], case["hidden"]
    if case["op"] == "norm":
        return _prepare_norm(case, gen)
    if case["op"] == "router":
        s = {"case": case, "x": _rows(gen, case, 1.0),
             "w": (torch.randn(case["experts"], h, generator=gen, device="cuda")
                   / math.sqrt(h)).to(torch.bfloat16)}
        if own:
            s["out"] = torch.empty(t, case["experts"], device="cuda")
        return s
    return _prepare_moe(case, gen)


def _prepare_norm(case, gen):
    t, h = case["tokens"], case["hidden"]
    s = {"case": case, "x": _rows(gen, case, 0.5),
         "w": (1 + 0.1 * torch.randn(h, generator=gen, device="cuda")).to(torch.bfloat16)}
    if case["residual"]:
        # a residual stream: a few channels are much larger than the rest
        chan = torch.where(torch.rand(h, generator=gen, device="cuda") < 0.005, 30.0, 2.0)
        s["r"] = (torch.randn(t, h, generator=gen, device="cuda") * chan).to(torch.bfloat16)
    if own:
        def buf(dtype, *shape):
            return torch.empty(*shape, dtype=dtype, device="cuda")
        s["out"] = (buf(torch.bfloat16, t, h) if case["bf16"] else None,
                    buf(torch.bfloat16, t, h) if case["residual"] else None,
                    buf(F8, t, h) if case["fp8"] else None,
                    buf(torch.float32, t, _groups(h, case["fp8"])) if case["fp8"] else None)
    return s


def _prepare_moe(case, gen):
    t, h, i, local = case["tokens"], case["hidden"], case["inter"], case["local"]

    def weights(n, k):
        q = torch.randint(0, 256, (local, n, k // 2), generator=gen, device="cuda",
                          dtype=torch.uint8)
        sc = torch.randn(local, n, k // 32, generator=gen, device="cuda").abs() * 0.02
        return q, sc.to(torch.bfloat16)

    s = {"case": case, "offset": min(local, case["experts"] - local)}
    s["q_gu"], s["s_gu"] = weights(2 * i, h)
    s["q_dn"], s["s_dn"] = weights(h, i)
    x = torch.randn(t, h, generator=gen, device="cuda")
    if case["fp8"]:
        pad = -h % GROUP
        amax = torch.nn.functional.pad(x.abs(), (0, pad)).view(t, -1, GROUP).amax(-1)
        s["x_scales"] = amax / 448.0
        s["x"] = (x / s["x_scales"].repeat_interleave(GROUP, 1)[:, :h]).to(F8)
    else:
        s["x"] = x.to(torch.bfloat16)
    logits = torch.randn(t, case["experts"], generator=gen, device="cuda")
    s["logits"] = logits.to(torch.bfloat16) if case["bf16_logits"] else logits
    if own:
        # the handle that a program keeps: packed weights, buffers and a workspace
        from w4a16_int4_moe_gb300 import moe, ops
        gu = moe.PackedExperts.from_checkpoint(s["q_gu"], s["s_gu"].view(torch.int16),
                                               layout=ops.W4A16_LAYOUT_KTILE64_GLU16)
        dn = moe.PackedExperts.from_checkpoint(s["q_dn"], s["s_dn"].view(torch.int16))
        s["layer"] = moe.W4A16MoE(gu, dn, case["topk"], t)
        s["out"] = torch.empty(t, h, device="cuda")
        s["routing"] = (torch.empty(t, case["topk"], dtype=torch.int32, device="cuda"),
                        torch.empty(t, case["topk"], device="cuda"))
    return s


# -------------------------------------------------------------------- run --

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "router": _own_router, "moe": _own_moe}[op](state)
    return {"norm": _plain_norm, "router": _plain_router, "moe": _plain_moe}[op](state)


def _own_norm(s):
    from w4a16_int4_moe_gb300 import ops
    y, r, y8, scales = ops.w4a16_add_rms_norm(s["x"], s["w"], EPS, residual=s.get("r"),
                                              fp8_group=s["case"]["fp8"], out=s["out"])
    return {"y": y, "residual": r, "y8": y8, "scales": scales}


def _own_router(s):
    from w4a16_int4_moe_gb300 import ops
    return ops.w4a16_router_logits(s["x"], s["w"], out=s["out"])


def _own_moe(s):
    ids, w = s["routing"]
    out = s["layer"].few_tokens_from_logits(s["x"], s["logits"], expert_offset=s["offset"],
                                            x_scales=s.get("x_scales"), out=s["out"],
                                            routing=s["routing"])
    return {"out": out, "topk_ids": ids, "topk_weights": w}


def _plain_norm(s):
    case = s["case"]
    h = s["x"].float()
    res = None
    if case["residual"]:
        h = h + s["r"].float()
        res = h.to(torch.bfloat16)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
    y8 = scales = None
    if case["fp8"]:
        t, n = y.shape
        g = n if case["fp8"] < 0 else case["fp8"]
        mag = torch.nn.functional.pad(y.abs(), (0, -n % g)).view(t, -1, g).amax(-1)
        scales = mag.clamp_min(1e-10) / 448.0
        y8 = (y / scales.repeat_interleave(g, 1)[:, :n]).to(F8)
    return {"y": y.to(torch.bfloat16) if case["bf16"] else None, "residual": res, "y8": y8,
            "scales": scales}


def _plain_router(s):
    return s["x"].float() @ s["w"].float().t()


def _plain_weights(q, scales, pick=None):
    """(q - 8) * scale in FP32, of all experts or of the picked ones."""
    if pick is not None:
        q, scales = q[pick], scales[pick]
    codes = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    return ((codes.float() - 8).unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _plain_moe(s):
    case = s["case"]
    t, h, i, k, local = (case[n] for n in ("tokens", "hidden", "inter", "topk", "local"))
    x = s["x"].float()
    if case["fp8"]:
        x = x * s["x_scales"].repeat_interleave(GROUP, 1)[:, :h]
    # routing: the largest logits, ties to the lower expert; softmax over all experts
    logits = s["logits"].float()
    best = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    e = torch.exp(logits - logits.amax(-1, keepdim=True))
    w = (e / e.sum(-1, keepdim=True)).gather(1, best)
    w = w / w.sum(-1, keepdim=True)
    ids = best - s["offset"]
    ids = torch.where((ids >= 0) & (ids < local), ids, -1)
    here = torch.where(ids >= 0, w, 0.0)
    at = ids.clamp_min(0)
    if t * k <= local:          # the picked experts' weights, one set a pick
        at = at.flatten()
        rows = x.repeat_interleave(k, 0)[:, :, None]
        gu = (_plain_weights(s["q_gu"], s["s_gu"], at) @ rows).squeeze(-1)
        act = gu[:, :i] / (1 + torch.exp(-gu[:, :i])) * gu[:, i:]
        dn = (_plain_weights(s["q_dn"], s["s_dn"], at) @ act[:, :, None]).view(t, k, h)
        out = (dn * here[..., None]).sum(1)
    else:                       # every expert on every token, weighted by the routing
        gu = x @ _plain_weights(s["q_gu"], s["s_gu"]).transpose(1, 2)
        act = gu[..., :i] / (1 + torch.exp(-gu[..., :i])) * gu[..., i:]
        dn = act @ _plain_weights(s["q_dn"], s["s_dn"]).transpose(1, 2)
        share = torch.zeros(t, local, device="cuda").scatter_add_(1, at, here)
        out = (dn * share.t()[..., None]).sum(0)
    return {"out": out, "topk_ids": ids.to(torch.int32), "topk_weights": w}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].double()
    if case["op"] == "router":
        return x @ s["w"].double().t()
    if case["op"] == "norm":
        return _exact_norm(case, s, x)
    return _exact_moe(case, s, x)


def _exact_norm(case, s, x):
    h = x + s["r"].double() if case["residual"] else x
    rms = torch.sqrt(h.square().sum(-1, keepdim=True) / case["hidden"] + EPS)
    y = h / rms * s["w"].double()
    y8 = scales = None
    if case["fp8"]:
        width = case["hidden"] if case["fp8"] < 0 else case["fp8"]
        parts = y.split(width, dim=1)
        scales = torch.stack([p.abs().amax(1).clamp(min=1e-10) for p in parts], 1) / 448
        y8 = torch.cat([p / scales[:, n:n + 1] for n, p in enumerate(parts)], 1)
    return {"y": y if case["bf16"] else None, "residual": h if case["residual"] else None,
            "y8": y8, "scales": scales}


def _exact_moe(case, s, x):
    t, i, k, local = case["tokens"], case["inter"], case["topk"], case["local"]
    if case["fp8"]:
        parts = x.split(GROUP, dim=1)
        x = torch.cat([p * s["x_scales"][:, n:n + 1].double() for n, p in enumerate(parts)], 1)
    logits = s["logits"].double()
    # the experts in order: larger logit first, then the lower number
    order = [sorted(range(case["experts"]), key=lambda e: (-row[e], e))[:k]
             for row in logits.tolist()]
    chosen = torch.tensor(order, device="cuda")
    share = torch.softmax(logits, -1).gather(1, chosen)
    share = share / share.sum(-1, keepdim=True)

    def weight(q, sc):
        low, high = (q % 16).double() - 8, (q // 16).double() - 8
        full = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device="cuda")
        full[:, 0::2], full[:, 1::2] = low, high
        return full * sc.double().repeat_interleave(32, dim=1)

    out = torch.zeros(t, case["hidden"], dtype=torch.float64, device="cuda")
    for e in range(local):
        tok = [n for n in range(t) if e + s["offset"] in order[n]]
        if not tok:
            continue
        slot = [order[n].index(e + s["offset"]) for n in tok]
        gu = x[tok] @ weight(s["q_gu"][e], s["s_gu"][e]).t()
        act = gu[:, :i] * torch.sigmoid(gu[:, :i]) * gu[:, i:]
        out[tok] += share[tok, slot][:, None] * (act @ weight(s["q_dn"][e], s["s_dn"][e]).t())
    return {"out": out, "topk_ids": None, "topk_weights": share}

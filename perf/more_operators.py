"""What stands next to the routed experts in a decoder layer: products with
INT4 weights for a few tokens, the shared expert's products in BF16 (plain, or
gated: both projections, the activation and the product), and the norms after
and before a block with its gate and residual scale.

``own`` selects what ``run`` computes with: the plain torch forms, or the
library's entry points. Shapes are the library's own (hidden 7168, intermediate
2048, 576 decoding tokens, 8192 of a prefill) and generic small, wide or ragged
ones.
"""

from __future__ import annotations

import math

import torch

own = False

BF16 = torch.bfloat16
F8 = torch.float8_e4m3fn
EPS = 1e-6
GROUP = 128          # columns that share a scale of the 8-bit form


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decoding sequence, a shared expert in the experts' own format: gate and up
        _int4("int4_one_gated", 1, 4096, 7168, gated=True, add=False, f32=False, pitch=0),
        # its way back, added to what the routed experts left: the smallest call
        _int4("int4_one_add", 1, 7168, 2048, gated=False, add=True, f32=True, pitch=0),
        # a few sequences, ragged: rows of a wider buffer, sizes that fill no tile
        _int4("int4_ragged", 5, 1000, 2080, gated=False, add=False, f32=False, pitch=2176),
        # a full few-token batch through a wide projection
        _int4("int4_32_wide", 32, 16384, 7168, gated=False, add=False, f32=False, pitch=0),
        # one decoding sequence, a shared expert in BF16: its weights are the time
        _dense("dense_one_gated", 1, 4096, 7168, gated=True, add=False, f32=False, pitch=0),
        # a ragged batch of a small gated block, rows of a wider buffer
        _dense("dense_ragged_gated", 77, 2 * 1000, 2088, gated=True, add=False, f32=False,
               pitch=2400),
        # a decode batch: between the weights' bytes and the tensor cores
        _dense("dense_decode_gated", 576, 4096, 7168, gated=True, add=False, f32=False, pitch=0),
        # a prefill chunk, gate and up: a real dense product
        _dense("dense_prefill_gated", 8192, 4096, 7168, gated=True, add=False, f32=False, pitch=0),
        # its way back, added to what the routed experts left
        _dense("dense_prefill_add", 8192, 7168, 2048, gated=False, add=True, f32=True, pitch=0),
        # one decoding sequence: the experts' FP32 sum, normed, into the residual, normed again
        _norm("norm_one", 1, 7168, x32=True, post=True, gate=0, residual=True, bf16=True, fp8=0,
              offset=False, pitch=0),
        # ragged: BF16 rows of a wider buffer, no norm after the block but a gate a channel,
        # the next block's rows in 8 bits only
        _norm("norm_ragged_fp8", 1021, 2088, x32=False, post=False, gate=1, residual=True,
              bf16=False, fp8=-1, offset=True, pitch=2400),
        # a prefill chunk with everything: gates of every token, 8-bit rows beside the BF16 ones
        _norm("norm_prefill_fp8", 8192, 7168, x32=True, post=True, gate=2, residual=True,
              bf16=True, fp8=128, offset=False, pitch=0),
    ]


def _product(op, name, tokens, n, k, gated, add, f32, pitch):
    c = {"op": op, "tokens": tokens, "n": n, "k": k, "gated": gated, "add": add, "f32": f32,
         "pitch": pitch}
    return dict(c, name=name) if name else c


def _int4(name, *args, **kw):
    return _product("int4", name, *args, **kw)


def _dense(name, *args, **kw):
    return _product("dense", name, *args, **kw)


def _norm(name, tokens, hidden, x32, post, gate, residual, bf16, fp8, offset, pitch):
    c = {"op": "norm", "tokens": tokens, "hidden": hidden, "x32": x32, "post": post, "gate": gate,
         "residual": residual, "bf16": bf16, "fp8": fp8, "offset": offset, "pitch": pitch}
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int4", "dense", "norm"])
    if op == "norm":
        hidden, bf16 = 8 * _log(rng, 8, 896), rng.random() < 0.7
        return _norm("", _log(rng, 1, 8192), hidden, rng.random() < 0.6, rng.random() < 0.6,
                     rng.choice([0, 0, 1, 2]), rng.random() < 0.8, bf16,
                     rng.choice([0, 128, -1]) if bf16 else rng.choice([128, -1]),
                     rng.random() < 0.3,
                     hidden + 8 * rng.randint(1, 64) if rng.random() < 0.3 else 0)
    gated = rng.random() < 0.5
    add = not gated and rng.random() < 0.5
    f32 = add or (not gated and rng.random() < 0.3)
    if op == "int4":
        k = 32 * _log(rng, 1, 256)
        n = 128 * _log(rng, 1, 128) if gated else _log(rng, 16, 16384)
        return _int4("", _log(rng, 1, 32), n, k, gated, add, f32,
                     k + 8 * rng.randint(1, 64) if rng.random() < 0.3 else 0)
    # long reductions leave in BF16, as a block's inner products do
    k = 8 * _log(rng, 8, 512 if f32 else 896)
    n = 2 * _log(rng, 16, 2048) if gated else _log(rng, 16, 7168)
    return _dense("", _log(rng, 1, 8192), n, k, gated, add, f32,
                  k + 8 * rng.randint(1, 64) if rng.random() < 0.3 else 0)


def work(case):
    t = case["tokens"]
    if case["op"] == "norm":
        h = case["hidden"]
        per = 4 if case["x32"] else 2
        per += (4 if case["residual"] else 2) + (2 if case["gate"] == 2 else 0)
        per += 2 if case["bf16"] else 0
        n = t * h * per + 2 * h * (1 + case["post"] + (case["gate"] == 1))
        if case["fp8"]:
            n += t * h + 4 * t * _groups(h, case["fp8"])
        return {"bytes": n, "flops": t * h * (8 + 4 * case["post"] + (case["gate"] > 0))}
    n, k = case["n"], case["k"]
    m = n // 2 if case["gated"] else n
    weight = n * k * (0.5 + 2 / 32) if case["op"] == "int4" else 2 * n * k
    out = t * m * ((4 if case["f32"] else 2) + (4 if case["add"] else 0))
    return {"bytes": int(weight + 2 * t * k + out), "flops": 2 * t * n * k}


def _groups(hidden, fp8):
    return 1 if fp8 < 0 else -(-hidden // fp8)


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_norm(case, gen) if case["op"] == "norm" else _prepare_product(case, gen)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _prepare_product(case, gen):
    t, n, k = case["tokens"], case["n"], case["k"]
    m = n // 2 if case["gated"] else n
    # BF16 rows of normal values; with a pitch, the first columns of a wider buffer
    s = {"case": case, "x": _randn(gen, t, case["pitch"] or k).to(BF16)[:, :k]}
    if case["op"] == "int4":
        s["q"] = torch.randint(0, 256, (n, k // 2), generator=gen, device="cuda",
                               dtype=torch.uint8)
        # weights of variance 1 / k
        s["s"] = (_randn(gen, n, k // 32).abs() * (0.2 / math.sqrt(k))).to(BF16)
    else:
        s["w"] = (_randn(gen, n, k) / math.sqrt(k)).to(BF16)
    s["add"] = _randn(gen, t, m) if case["add"] else None
    if own:
        s["out"] = torch.empty(t, m, dtype=torch.float32 if case["f32"] else BF16, device="cuda")
        if case["op"] == "int4":
            # packed once, at load
            from w4a16_int4_moe_gb300 import ops
            s["layout"] = (ops.W4A16_LAYOUT_KTILE64_GLU16 if case["gated"]
                           else ops.W4A16_LAYOUT_KTILE64)
            s["packed"] = ops.w4a16_prepack(s["q"][None], s["s"][None], layout=s["layout"])
    return s


def _prepare_norm(case, gen):
    t, h = case["tokens"], case["hidden"]
    one = 0.0 if case["offset"] else 1.0

    def weight():
        return (one + 0.1 * _randn(gen, h)).to(BF16)

    x = _randn(gen, t, case["pitch"] or h)[:, :h] * 0.5
    s = {"case": case, "pre": weight(), "post": weight() if case["post"] else None,
         "x": x if case["x32"] else x.to(BF16), "residual": None, "gate": None,
         "branch_scale": 0.5 if case["gate"] else 1.0,
         "residual_scale": 1.25 if case["offset"] else 1.0}
    if case["x32"] and not case["pitch"]:
        s["x"] = s["x"].contiguous()
    if case["residual"]:
        # a residual stream: a few channels are much larger than the rest
        chan = torch.where(torch.rand(h, generator=gen, device="cuda") < 0.005, 30.0, 2.0)
        s["residual"] = (_randn(gen, t, h) * chan).to(BF16)
    if case["gate"]:
        s["gate"] = torch.tanh(_randn(gen, t, h) if case["gate"] == 2 else _randn(gen, h)).to(BF16)
    if own:
        def buf(dtype, *shape):
            return torch.empty(*shape, dtype=dtype, device="cuda")
        s["out"] = (buf(BF16, t, h) if case["bf16"] else None, buf(BF16, t, h),
                    buf(F8, t, h) if case["fp8"] else None,
                    buf(torch.float32, t, _groups(h, case["fp8"])) if case["fp8"] else None)
    return s


# -------------------------------------------------------------------- run --

def run(state):
    op = state["case"]["op"]
    if own:
        return {"int4": _own_int4, "dense": _own_dense, "norm": _own_norm}[op](state)
    return {"int4": _plain_product, "dense": _plain_product, "norm": _plain_norm}[op](state)


def _own_int4(s):
    from w4a16_int4_moe_gb300 import ops
    return ops.w4a16_linear_few_tokens(s["x"], s["packed"], s["case"]["n"], layout=s["layout"],
                                       addend=s["add"], out=s["out"])


def _own_dense(s):
    from w4a16_int4_moe_gb300 import ops
    return ops.w4a16_dense(s["x"], s["w"], gated=s["case"]["gated"], addend=s["add"],
                           out=s["out"])


def _own_norm(s):
    from w4a16_int4_moe_gb300 import ops
    case = s["case"]
    y, h, y8, scales = ops.w4a16_block_norm(
        s["x"], s["pre"], EPS, post_weight=s["post"], gate=s["gate"], residual=s["residual"],
        branch_scale=s["branch_scale"], residual_scale=s["residual_scale"],
        weight_offset=1.0 if case["offset"] else 0.0, fp8_group=case["fp8"], out=s["out"])
    return {"y": y, "h": h, "y8": y8, "scales": scales}


def _plain_product(s):
    case = s["case"]
    if case["op"] == "int4":
        codes = torch.stack((s["q"] & 15, s["q"] >> 4), -1).flatten(-2)
        w = ((codes.float() - 8).unflatten(-1, (-1, 32)) * s["s"].float()[..., None]).flatten(-2)
    else:
        w = s["w"].float()
    out = s["x"].float() @ w.t()
    if case["gated"]:
        gate, up = out[:, :case["n"] // 2], out[:, case["n"] // 2:]
        out = gate / (1 + torch.exp(-gate)) * up
    if case["add"]:
        out = out + s["add"]
    return out if case["f32"] else out.to(BF16)


def _plain_norm(s):
    case = s["case"]
    offset = 1.0 if case["offset"] else 0.0
    b = s["x"].float()
    if case["post"]:
        b = b * torch.rsqrt((b * b).mean(-1, keepdim=True) + EPS) * (s["post"].float() + offset)
    b = b * s["branch_scale"]
    if case["gate"]:
        b = b * s["gate"].float()
    h = b + s["residual"].float() * s["residual_scale"] if case["residual"] else b
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * (s["pre"].float() + offset)
    y8 = scales = None
    if case["fp8"]:
        t, n = y.shape
        g = n if case["fp8"] < 0 else case["fp8"]
        mag = torch.nn.functional.pad(y.abs(), (0, -n % g)).view(t, -1, g).amax(-1)
        scales = mag.clamp_min(1e-10) / 448.0
        y8 = (y / scales.repeat_interleave(g, 1)[:, :n]).to(F8)
    return {"y": y.to(BF16) if case["bf16"] else None, "h": h.to(BF16), "y8": y8,
            "scales": scales}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_norm(case, s) if case["op"] == "norm" else _exact_product(case, s)


def _exact_product(case, s):
    n, k = case["n"], case["k"]
    if case["op"] == "int4":
        w = torch.empty(n, k, dtype=torch.float64, device="cuda")
        w[:, 0::2] = (s["q"] % 16).double() - 8
        w[:, 1::2] = (s["q"] // 16).double() - 8
        for c in range(0, k, 32):
            w[:, c:c + 32] *= s["s"][:, c // 32:c // 32 + 1].double()
    else:
        w = s["w"].double()
    x = s["x"].double()
    if case["gated"]:
        g = x @ w[:n // 2].t()
        return g * torch.sigmoid(g) * (x @ w[n // 2:].t())
    out = x @ w.t()
    return out + s["add"].double() if case["add"] else out


def _exact_norm(case, s):
    width = case["hidden"]

    def normed(v, w):
        rms = torch.sqrt(v.square().sum(-1, keepdim=True) / width + EPS)
        return v / rms * (w.double() + (1 if case["offset"] else 0))

    branch = s["x"].double()
    if s["post"] is not None:
        branch = normed(branch, s["post"])
    if s["gate"] is not None:
        branch = s["gate"].double() * branch
    h = s["branch_scale"] * branch
    if s["residual"] is not None:
        h = h + s["residual_scale"] * s["residual"].double()
    y = normed(h, s["pre"])
    y8 = scales = None
    if case["fp8"]:
        parts = y.split(width if case["fp8"] < 0 else case["fp8"], dim=1)
        scales = torch.stack([p.abs().amax(1).clamp(min=1e-10) for p in parts], 1) / 448
        y8 = torch.cat([p / scales[:, n:n + 1] for n, p in enumerate(parts)], 1)
    return {"y": y if case["bf16"] else None, "h": h, "y8": y8, "scales": scales}

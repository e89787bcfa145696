"""64-bit forms of the norm, the router's product and the few-token layer, and
bounds of their rounding errors (test infrastructure, no product code).

Bounds count roundings. A floating-point sum of n terms in any order, each
addition off by at most u relative to the partial sum it makes, is off by at
most n * u * sum|terms|; the kernels add at least 16 products between two such
roundings on a path, and a tensor core may cut instead of rounding, so u is a
whole step (2^-23) and the count is n / 16 plus the joining additions.
"""

import numpy as np
import torch

import oracle

U32 = 2.0 ** -24      # half a step of FP32
BF16_HALF = 2.0 ** -8
E4M3_HALF = 2.0 ** -4


def sum_bound(n):
    return (n / 16 + 64) * 2.0 ** -23


def norm(x, residual, weight, eps):
    """x, residual, weight float64 arrays -> (h, y)."""
    h = x if residual is None else x + residual
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * weight
    return h, y


def group_scales(y, group):
    """max(amax, 1e-10) / 448 of every group of columns."""
    cols = [y[:, c:c + group] for c in range(0, y.shape[1], group)]
    return np.stack([np.maximum(np.abs(c).max(axis=1), 1e-10) for c in cols], axis=1) / 448.0


def e4m3(bits):
    return torch.from_numpy(bits).view(torch.float8_e4m3fn).to(torch.float64).numpy()


def few_layer(x, ids, weights, p):
    """(out float64 [T, H], bound of |error|): the layer over the picks whose id is one of p's
    experts. x float64 [T, H], p holds q_gu, s_gu, q_dn, s_dn."""
    tokens, hidden = x.shape
    inter = p.inter
    out = np.zeros((tokens, hidden))
    err = np.zeros((tokens, hidden))
    for e in range(p.num_experts):
        rows, slots = np.nonzero(ids == e)
        if rows.size == 0:
            continue
        wg = oracle.dequant_weights(p.q_gu[e], p.s_gu[e])
        wd = oracle.dequant_weights(p.q_dn[e], p.s_dn[e])
        xe = x[rows]
        gu = xe @ wg.T
        gu_err = sum_bound(hidden) * (np.abs(xe) @ np.abs(wg).T)
        g, u = gu[:, :inter], gu[:, inter:]
        ge, ue = gu_err[:, :inter], gu_err[:, inter:]
        silu = g / (1.0 + np.exp(-g))
        act = silu * u
        # |silu'| <= 1.1; exp, the sum, the quotient and the product: at most
        # (|g| + 8) half steps (the exponent's argument carries |g| of them)
        act_err = 1.1 * ge * (np.abs(u) + ue) + np.abs(silu) * ue \
            + (np.abs(g) + 8) * U32 * np.abs(act)
        w = weights[rows, slots].astype(np.float64)[:, None]
        d_err = act_err @ np.abs(wd).T + sum_bound(inter) * (np.abs(act) @ np.abs(wd).T)
        np.add.at(out, rows, w * (act @ wd.T))
        np.add.at(err, rows, np.abs(w) * (d_err + 40 * U32 * (np.abs(act) @ np.abs(wd).T)))
    return out, err


def assert_within(got, ref, bound, what=""):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), f"{what}: not finite"
    over = np.abs(got - ref) - bound
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else ()
    assert over.size == 0 or over[at] <= 0, (
        f"{what}: {got[at]} for {ref[at]} at {at}, bound {np.broadcast_to(bound, ref.shape)[at]}")

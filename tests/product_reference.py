"""64-bit forms of the products with one weight and of the block's norms, and
bounds of their rounding errors (test infrastructure, no product code).

A floating-point sum of n terms in any order, each addition off by at most u
relative to the partial sum it makes, is off by at most n * u * sum|terms|. The
kernels add at least 16 products between two such roundings on a path, and a
tensor core may cut instead of rounding, so u is a whole step of FP32.
"""

import torch

STEP = 2.0 ** -23
BF16_HALF = 2.0 ** -8


def sum_bound(n):
    return (n / 16 + 64) * STEP


def int4_weight(q, scales):
    """(weights float64 [n, k], bound weights float64 [n, k]): sum over c of
    |x[c]| * bound[r, c] is what the group sums of row r may lose before their
    scale is applied: the codes enter as 16 + q (at most 31) and 24 comes off, and
    a group is four MMAs, each of which adds at most 17 terms."""
    n, kh = q.shape
    w = torch.empty(n, 2 * kh, dtype=torch.float64, device=q.device)
    w[:, 0::2] = (q & 15).double() - 8
    w[:, 1::2] = (q >> 4).double() - 8
    s = scales.double().repeat_interleave(32, dim=1)
    return w * s, s.abs() * (55 * 4 * 17 * STEP)


def product(x, w, loose, gated, addend):
    """(value, bound of |error|) float64 of x . w^T (+ addend), or gated."""
    x = x.double()
    v = x @ w.t()
    err = sum_bound(w.shape[1]) * (x.abs() @ w.abs().t())
    if loose is not None:
        err = err + x.abs() @ loose.t()
    if gated:
        i = w.shape[0] // 2
        g, u, ge, ue = v[:, :i], v[:, i:], err[:, :i], err[:, i:]
        silu = g * torch.sigmoid(g)
        v = silu * u
        # |silu'| <= 1.1; exp, the sum, the quotient and the product: at most
        # (|g| + 8) half steps (the exponent's argument carries |g| of them)
        err = 1.1 * ge * (u.abs() + ue) + silu.abs() * ue + (g.abs() + 8) * STEP * v.abs()
    if addend is not None:
        v = v + addend.double()
        err = err + STEP * v.abs()
    return v, err


def assert_within(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = (got - want).abs() - bound
    if over.numel() and over.max() > 0:
        at = tuple(int(i) for i in torch.nonzero(over == over.max())[0])
        raise AssertionError(f"{what}: {got[at]} for {want[at]} at {at}, "
                             f"bound {torch.broadcast_to(bound, want.shape)[at]}")


def check_product(out, x, w, loose=None, gated=False, addend=None, what=""):
    v, err = product(x, w, loose, gated, addend)
    if out.dtype is torch.bfloat16:
        err = err + (v.abs() + err) * BF16_HALF + 2.0 ** -133
    assert_within(out, v, err, what)


def block_norm(x, pre, eps, post=None, gate=None, residual=None, branch_scale=1.0,
               residual_scale=1.0, offset=0.0):
    """(y, h, bound weight of h) float64: h is off by at most a few steps of the
    sum of its two terms' magnitudes, the third result."""
    def normed(v, w):
        return v / torch.sqrt(v.square().mean(1, keepdim=True) + eps) * (w.double() + offset)
    b = x.double()
    if post is not None:
        b = normed(b, post)
    b = branch_scale * b
    if gate is not None:
        b = b * gate.double()
    h, size = b, b.abs()
    if residual is not None:
        r = residual_scale * residual.double()
        h, size = b + r, size + r.abs()
    return (None if pre is None else normed(h, pre)), h, size

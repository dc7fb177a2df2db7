"""The dense path's definitions in 64 bits, each with a bound on how far a result that rounds as the
library says may be off.

The bounds follow the roundings: a product of K bf16 pairs with fp32 sums errs by at most K·2^-23 of
the sum of the magnitudes (each of K additions by 2^-23 of a partial sum, also where it truncates), a
rounding to bf16 by 2^-8 of the value, an activation or an exponential in fp32 by 2^-19 of itself; what
an error of a factor does to a product is that error times the other factor. `SLACK` covers the
products of two errors.
"""
from __future__ import annotations

import math
from typing import NamedTuple

import torch

BF = 2.0 ** -8
ACT = 2.0 ** -19
SLACK = 1.05
TINY = 1e-37          # results near the end of fp32's and bf16's range are flushed


def unit(k):
    """Of a sum of k products, relative to the sum of their magnitudes."""
    return (k + 2) * 2.0 ** -23


class V(NamedTuple):
    """Values and a bound on their errors."""
    v: torch.Tensor
    e: torch.Tensor


def exactly(t):
    t = t.double()
    return V(t, torch.zeros_like(t))


def rounded(a, dtype=torch.bfloat16):
    step = BF if dtype == torch.bfloat16 else 2.0 ** -24
    return V(a.v, (a.e * (1 + step) + step * a.v.abs()) * SLACK + TINY)


def matmul(a, b):
    """a · b with fp32 sums."""
    size = a.v.abs() @ b.v.abs()
    e = a.e @ b.v.abs() + a.v.abs() @ b.e + a.e @ b.e + unit(a.v.shape[1]) * size
    return V(a.v @ b.v, e * SLACK + TINY)


def t(a):
    return V(a.v.t(), a.e.t())


def times(a, b):
    return V(a.v * b.v, a.e * b.v.abs() + a.v.abs() * b.e + a.e * b.e + ACT * (a.v * b.v).abs())


def plus(a, b):
    return V(a.v + b.v, a.e + b.e + 2.0 ** -23 * (a.v.abs() + b.v.abs()))


_S = 1 / math.sqrt(2 * math.pi)


def act_of(name, g):
    """(act(g), act'(g)) in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        p = 0.5 * torch.special.erfc(-g * math.sqrt(0.5))
        return g * p, p + g * _S * torch.exp(-g * g / 2)
    z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    th = torch.tanh(z)
    return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)


def act(name, g):
    """act and its derivative of values with errors: |act'| <= 1.13, |act''| <= 0.8 (silu 0.5; gelu 2/sqrt(2 pi); its
    tanh form within a hundredth of that). The derivative is a sum of two terms below 1 and 0.3."""
    a, slope = act_of(name, g.v)
    return V(a, 1.13 * g.e + ACT * (a.abs() + 1e-3 * torch.exp(-g.v.abs()))), V(slope, 0.82 * g.e + ACT * (1 + slope.abs()))


def gated_ffn(x, wg, wu, wd, name):
    """(out, gate, up, h) as values with errors."""
    x, wg, wu, wd = map(exactly, (x, wg, wu, wd))
    g, u = matmul(x, t(wg)), matmul(x, t(wu))
    h = rounded(times(act(name, g)[0], u))
    return rounded(matmul(h, t(wd))), rounded(g), rounded(u), h


def gated_ffn_grad(grad, x, wg, wu, wd, name, dtype=torch.bfloat16):
    """(dx, dwg, dwu, dwd)."""
    _, g, u, h = gated_ffn(x, wg, wu, wd, name)
    grad, x, wg, wu, wd = map(exactly, (grad, x, wg, wu, wd))
    dh = matmul(grad, wd)
    a, slope = act(name, g)
    dg, du = rounded(times(times(dh, u), slope)), rounded(times(dh, a))
    dx = rounded(plus(matmul(dg, wg), matmul(du, wu)))
    return dx, rounded(matmul(t(dg), x), dtype), rounded(matmul(t(du), x), dtype), rounded(matmul(t(grad), h), dtype)


def cross_entropy(x, w, targets, grad=None, dtype=torch.bfloat16):
    """(loss, lse), and with `grad` also (dx, dw). Rows of dropped targets are taken as zeros."""
    vocab = w.shape[0]
    kept = (targets >= 0) & (targets < vocab)
    x = torch.where(kept[:, None], x.double(), 0.0) if grad is not None else x.double()
    l = matmul(exactly(x), t(exactly(w)))
    lse = torch.logsumexp(l.v, 1)
    p = torch.exp(l.v - lse[:, None])
    # an error of a logit moves lse by its share; the exponentials' argument l·log2(e) rounds to 2^-23 of itself
    arg = l.e + 2.0 ** -22 * l.v.abs() + ACT
    e_lse = ((p * arg).sum(1) + unit(vocab) + 2.0 ** -22 * lse.abs()) * SLACK
    at = targets.clamp(0, vocab - 1).long()[:, None]
    loss = torch.where(kept, lse - l.v.gather(1, at)[:, 0], 0.0)
    e_loss = torch.where(kept, e_lse + l.e.gather(1, at)[:, 0] + 2.0 ** -23 * (lse.abs() + loss.abs()), 0.0)
    out = V(loss, e_loss + TINY), V(lse, e_lse + TINY)
    if grad is None:
        return out
    hot = torch.zeros_like(p).scatter_(1, at, 1.0)
    weight = torch.where(kept, grad.double(), 0.0)[:, None]
    relative = torch.expm1(arg + e_lse[:, None]) + 2 * ACT
    # exponentials are held relative to a power of two within 2^64 of a row's sum, and below 2^-126 of that as zeros:
    # a probability below 2^-126 · 2^64 may come out as none
    d = V((p - hot) * weight, weight.abs() * (p * relative + (p - hot).abs() * BF + 2.0 ** -62) * SLACK + TINY * (weight != 0))
    dx = rounded(matmul(d, exactly(w)))
    # the rows of x are rounded once more after their scaling
    xs = V(x, BF * x.abs() * SLACK)
    return *out, dx, rounded(matmul(t(d), xs), dtype)


def within(got, want, what):
    """got within want's bound, value by value."""
    got = got.double()
    assert got.shape == want.v.shape, (what, got.shape, want.v.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    far = (got - want.v).abs() / want.e.clamp_min(1e-300)
    far = torch.where((got == want.v), 0.0, far)
    worst = float(far.max()) if far.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst} of the bound at {int(far.argmax())}"
    return worst

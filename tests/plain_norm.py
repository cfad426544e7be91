"""Plain 64-bit form of the norms around a block and its gradients, written from
the formulas in include/tpmlp.h, for the tests; with each value the sum of the
magnitudes it is made of, from which the tests take their bounds."""
from __future__ import annotations

import torch

F32 = 2.0 ** -24
BF16 = 2.0 ** -8
#: roundings along the longest way from inputs to a value (loads are exact): the row
#: sums add 16 values in a thread, 5 + 5 shuffles and 4 warps' parts, twice where a
#: mean comes first; the rest is a handful of products
STEPS = 64


def stats_of(v, kind, eps):
    mean = v.mean(1) if kind == "layer" else torch.zeros_like(v[:, 0])
    var = (v - mean[:, None]).square().mean(1)
    return mean, (var + eps).rsqrt()


def normed(v, kind, gamma, beta, mean, rstd):
    """(value, magnitude) of N(v)."""
    if kind == "none":
        return v, v.abs()
    m, r = mean[:, None], rstd[:, None]
    b = beta if kind == "layer" else 0 * gamma
    return (v - m) * r * gamma + b, (v.abs() + m.abs()) * r * gamma.abs() + b.abs()


def forward(X, Z, kind, gamma, beta, gate, alpha, eps):
    """(Out, its magnitude, mean, rstd) in 64 bits; gate per row or None."""
    mean, rstd = stats_of(Z, kind, eps) if kind != "none" else (None, None)
    u, mag = normed(Z, kind, gamma, beta, mean, rstd)
    if gate is not None:
        u, mag = gate * u, gate.abs() * mag
    return alpha * X + u, abs(alpha) * X.abs() + mag, mean, rstd


def through(dy, v, kind, gamma, mean, rstd):
    """Gradient of v, its magnitude, and (dgamma, dbeta) terms per row with theirs."""
    m, r = mean[:, None], rstd[:, None]
    hat, big = (v - m) * r, (v.abs() + m.abs()) * r
    w = dy * gamma
    d = w - hat * (w * hat).mean(1, keepdim=True)
    mag = w.abs() + big * (w.abs() * big).mean(1, keepdim=True)
    if kind == "layer":
        d = d - w.mean(1, keepdim=True)
        mag = mag + w.abs().mean(1, keepdim=True)
    return r * d, r * mag, dy * hat, dy.abs() * big


def backward(dOut, dXn, Z, Out, post, pre, g1, b1, gate, g2, alpha, stats):
    """Every gradient as (value, magnitude); row sums left per row (dgate too)."""
    m1, r1, m2, r2 = stats
    got = {}
    g, mag = dOut, dOut.abs()
    if pre != "none":
        d, dm, terms, tm = through(dXn, Out, pre, g2, m2, r2)
        g, mag = g + d, mag + dm
        got["dpre_gamma"] = (terms, tm)
        if pre == "layer":
            got["dpre_beta"] = (dXn, dXn.abs())
    got["dX"] = (alpha * g, abs(alpha) * mag)
    if Z is None:
        return got
    u, um = normed(Z, post, g1, b1, m1, r1)
    if gate is not None:
        got["dgate"] = (g * u, mag * um)
        g, mag = g * gate, mag * gate.abs()
    if post != "none":
        if post == "layer":
            got["dpost_beta"] = (g, mag)
        d, _, terms, _ = through(g, Z, post, g1, m1, r1)
        _, dm, _, tm = through(mag, Z, post, g1.abs(), m1, r1)
        got["dpost_gamma"] = (terms, tm)
        g, mag = d, dm
    got["dZ"] = (g, mag)
    return got

"""Plain 64-bit forms of the 8-bit calls, for the tests: written from the
definitions in include/tpmlp.h, on whatever device their inputs are.

Rounding to 8 bits is done by arithmetic (steps of 2^(e - bits), ties to even),
not by a cast.
"""
from __future__ import annotations

import torch

FORMATS = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}  # largest, mantissa bits, min exponent
FLOOR = -119
# half a step relative to the value (bf16), one fp32 rounding
BF16 = 2.0 ** -8
F32 = 2.0 ** -24


def pow2(k: torch.Tensor) -> torch.Tensor:
    """2^k in float64 by its exponent bits (torch.pow is not exact on every device)."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def round8(x: torch.Tensor, fmt: str) -> torch.Tensor:
    """x (float64, within the format's range) to the nearest value of the format."""
    _, bits, low = FORMATS[fmt]
    _, e = torch.frexp(x)                      # x = m 2^e, m in [1/2, 1)
    e = (e - 1).clamp(min=low)
    step = pow2(e - bits)
    return torch.round(x / step) * step


def scale_of(amax: torch.Tensor, fmt: str) -> torch.Tensor:
    """The smallest power of two s >= 2^-119 with amax <= s * top; NaN if not finite."""
    top = FORMATS[fmt][0]
    fine = torch.isfinite(amax)
    a = torch.where(fine, amax, torch.ones_like(amax)).clamp(min=2.0 ** -200)
    _, e = torch.frexp(a / top)
    k = e - 1                                  # 2^k <= a / top < 2^(k + 1)
    k = torch.where(pow2(k) * top >= a, k, k + 1).clamp(min=FLOOR)
    return torch.where(fine, pow2(k), torch.nan)


def _group_max(x: torch.Tensor, dim: int) -> torch.Tensor:
    n = x.shape[dim]
    parts = [x.narrow(dim, i, min(128, n - i)).abs().amax(dim, keepdim=True)
             for i in range(0, n, 128)]
    return torch.cat(parts, dim)


def _spread(s: torch.Tensor, dim: int, n: int) -> torch.Tensor:
    return s.repeat_interleave(128, dim).narrow(dim, 0, n)


def _q(x, s, fmt):
    q = round8(torch.where(torch.isfinite(s), x / s, torch.zeros_like(x)), fmt)
    return torch.where(torch.isnan(s), torch.zeros_like(q), q)


def quantize(x: torch.Tensor, fmt: str, dim: int):
    """(q, s) in float64 of x [R, C] with groups of 128 along dim; s keeps x's axis order."""
    x = x.double()
    s = scale_of(_group_max(x, dim), fmt)
    return _q(x, _spread(s, dim, x.shape[dim]), fmt), s


def quantize_block(x: torch.Tensor, fmt: str):
    x = x.double()
    s = scale_of(_group_max(_group_max(x, 0), 1), fmt)
    return _q(x, _spread(_spread(s, 0, x.shape[0]), 1, x.shape[1]), fmt), s


def rows_value(q, s):
    """The matrix that row groups stand for; s [ceil(C/128), R] as the library lays it out."""
    return q.double() * _spread(s.double().T, 1, q.shape[1])


def cols_value(q, s):
    return q.double() * _spread(s.double(), 0, q.shape[0])


def block_value(q, s):
    return q.double() * _spread(_spread(s.double(), 0, q.shape[0]), 1, q.shape[1])


def product_bound(a: torch.Tensor, b: torch.Tensor, blocks: int) -> torch.Tensor:
    """How far fp32 sums of a @ b in K blocks of 128 may be off: at most 128
    roundings of 2^-23 (the tensor cores may truncate) inside a block, and for
    each block one for the two scales, one for the sum and one for their
    product, all relative to the sum of the magnitudes."""
    return (128 * 2.0 ** -23 + (blocks + 2) * 2 * F32) * (a.abs() @ b.abs())


def check(name, got, ref, bound):
    got, ref = got.double(), ref.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = torch.isnan(ref) != torch.isnan(got)
    assert not bad.any(), f"{name}: NaN in the wrong places ({int(bad.sum())})"
    d = (got - ref).abs() - bound
    d = torch.where(torch.isnan(ref), torch.full_like(d, -1.0), d)
    worst = float(d.max()) if d.numel() else -1.0
    assert worst <= 0, f"{name}: {int((d > 0).sum())} of {d.numel()} values beyond the bound by {worst:.3g}"

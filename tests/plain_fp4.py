"""Plain 64-bit forms of the 4-bit calls, for the tests: written from the
definitions in include/tpmlp.h, on whatever device their inputs are.
"""
from __future__ import annotations

import torch

from plain_fp8 import BF16, F32, check, pow2, round8  # noqa: F401

GROUP = {"mxfp4": 32, "nvfp4": 16}
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def round4(x: torch.Tensor) -> torch.Tensor:
    """x to the nearest 4-bit value, ties to the even code, by its distance from each."""
    a = x.abs().clamp(max=6.0)
    v = torch.tensor(VALUES, dtype=torch.float64, device=x.device)
    mids = (v[1:] + v[:-1]) / 2
    below = torch.searchsorted(mids, a.contiguous(), right=False)  # mids < a
    above = torch.searchsorted(mids, a.contiguous(), right=True)   # mids <= a
    code = torch.where(below % 2 == 0, below, above)               # on a tie: the even one
    return v[code] * torch.where(torch.signbit(x), -1.0, 1.0)


def least_power(amax: torch.Tensor, top: float, low: int) -> torch.Tensor:
    """The smallest power of two s >= 2^low with amax <= top * s."""
    a = amax.clamp(min=2.0 ** -300)
    _, e = torch.frexp(a / top)
    k = e - 1
    k = torch.where(pow2(k) * top >= a, k, k + 1).clamp(min=low)
    return pow2(k)


def tensor_scale(parts) -> torch.Tensor:
    x = torch.stack([p.double().abs() for p in parts])
    return least_power(torch.where(torch.isfinite(x), x, torch.zeros_like(x)).amax(), 6.0 * 448.0, -110)


def quantize(x: torch.Tensor, fmt: str, dim: int, g=None):
    """(q, s) in float64 of x [R, C], each of x's shape: 4-bit values with groups along dim, and
    the scale of each value's group, of nvfp4 in units of g."""
    x = x.double().movedim(dim, 1)
    n, size = x.shape[1], GROUP[fmt]
    p = torch.nn.functional.pad(x, (0, -n % size)).unflatten(1, (-1, size))
    amax = p.abs().amax(2, keepdim=True)
    fine = torch.isfinite(amax)
    amax = torch.where(fine, amax, torch.zeros_like(amax))
    if fmt == "mxfp4":
        s, unit = least_power(amax, 6.0, -126), 1.0
    else:
        unit = float(g)
        s = round8((amax / (6.0 * unit)).clamp(max=448.0), "e4m3").clamp(min=2.0 ** -9)
    q = round4(torch.where(fine, p, torch.zeros_like(p)) / (s * unit))
    s = torch.where(fine, s, torch.full_like(s, torch.nan)).expand_as(p)
    return tuple(v.flatten(1)[:, :n].movedim(1, dim) for v in (q, s))


def unpack(m):
    """(q, s) in float64 [R, K] of a library's matrix, decoded from its bytes as documented."""
    R, K = m.shape
    b = m.q.to(torch.int64)
    n = torch.stack([b & 15, b >> 4], 2).flatten(1)[:, :K]
    v = torch.tensor(VALUES, dtype=torch.float64, device=b.device)
    q = v[n & 7] * torch.where((n & 8) > 0, -1.0, 1.0)
    size = GROUP[m.fmt]
    blocks = 256 // size // 4                         # of 4 groups, for 256 of K
    kb = -(-K // 256)
    s = m.s.to(torch.int64).view(-1, kb, blocks, 32, 4, 4)    # row tile, 256 of K, block, r % 32, r / 32, j
    s = s.permute(0, 4, 3, 1, 2, 5).reshape(-1, kb * blocks * 4)[:R]  # row, group
    if m.fmt == "mxfp4":
        f = torch.where(s == 255, torch.nan, pow2(s - 127))
    else:
        e, frac = s >> 3, (s & 7).double()
        f = torch.where(e > 0, (1 + frac / 8) * pow2(e - 7), frac / 8 * 2.0 ** -6)
        f = torch.where(s == 127, torch.nan, f)
    return q, f.repeat_interleave(size, 1)[:, :K]


def value(m) -> torch.Tensor:
    """What a library's matrix stands for, float64 [R, K]."""
    q, s = unpack(m)
    return q * s * (1.0 if m.scale is None else m.scale.double())


def values(x, fmt, dim, g=None):
    """What x quantised along dim stands for, float64, of x's shape."""
    q, s = quantize(x, fmt, dim, g)
    return q * s * (1.0 if g is None else float(g))


def product_bound(a: torch.Tensor, b: torch.Tensor, blocks: int) -> torch.Tensor:
    """How far fp32 sums of a @ b in `blocks` steps of 64 of K may be off: at most 64 roundings
    of 2^-23 (the tensor cores may truncate) inside a step and one for each step's sum (or
    part), all relative to the sum of the magnitudes.  (The tensors' scales are powers of two.)"""
    return (64 + blocks + 8) * 2.0 ** -23 * (a.abs() @ b.abs())

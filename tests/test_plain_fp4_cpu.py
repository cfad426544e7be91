"""The plain 64-bit forms of the 4-bit calls against hand-worked values, and the backward
formulas against differences (CPU)."""
import pytest
import torch

import plain_fp4 as plain


def test_round4_by_hand():
    x = torch.tensor([0.0, 0.25, 0.2500001, 0.74, 0.75, 1.25, 1.26, 1.75, 2.5, 2.6, 3.5, 5.0, 5.1, 7.0, -0.3, -5.0],
                     dtype=torch.float64)
    want = [0.0, 0.0, 0.5, 0.5, 1.0, 1.0, 1.5, 2.0, 2.0, 3.0, 4.0, 4.0, 6.0, 6.0, -0.5, -4.0]
    assert plain.round4(x).tolist() == want


def test_scales_by_hand():
    a = torch.tensor([6.0, 6.01, 3.0, 2.99, 0.0, 1.0], dtype=torch.float64)
    assert plain.least_power(a, 6.0, -126).tolist() == [1.0, 2.0, 0.5, 0.5, 2.0 ** -126, 0.25]
    assert float(plain.tensor_scale([torch.tensor([2688.0, float("inf")])])) == 1.0
    assert float(plain.tensor_scale([torch.tensor([2689.0])])) == 2.0
    assert float(plain.tensor_scale([torch.zeros(3)])) == 2.0 ** -110


def test_groups_by_hand():
    x = torch.zeros(2, 64)
    x[0, 0], x[0, 40], x[1, 3] = 6.0, 12.0, 0.5
    q, s = plain.quantize(x, "mxfp4", 1)
    assert s[0, 0] == 1 and s[0, 40] == 2 and q[0, 40] == 6 and s[1, 3] == 0.125 and q[1, 3] == 4
    q, s = plain.quantize(x, "nvfp4", 1, 1.0)
    assert s[0, 0] == 1 and s[0, 40] == 2 and s[0, 20] == 2.0 ** -9
    # 0.5 / 6 = 0.08333 rounds to 0.0859375 in e4m3 (steps of 2^-7): 5.82 to 6
    assert s[1, 3] == 0.0859375 and q[1, 3] == 6


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_backward_formulas(fmt):
    """dX, dW and db of sum(dY * Y), Y = X W + b, against differences, on values that 4 bits hold
    exactly (then quantising is the identity, along either axis)."""
    g = torch.Generator()
    g.manual_seed(3)
    grid = torch.tensor([-6.0, -4.0, -3.0, -2.0, -1.5, -1.0, -0.5, 0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0],
                        dtype=torch.float64)

    def exact(r, c):
        m = grid[torch.randint(0, 15, (r, c), generator=g)]
        m[::16] = 6.0         # every group of either axis has a 6, and so the scale 1
        m[:, ::16] = 6.0
        return m
    X, W, dY = exact(32, 64), exact(64, 32), exact(32, 32)
    b = torch.randn(32, dtype=torch.float64, generator=g)
    unit = 1.0 if fmt == "nvfp4" else None
    for m in (X, W, dY):
        for dim in (0, 1):
            assert torch.equal(plain.values(m, fmt, dim, unit), m)
    loss = lambda x, w, v: float((dY * (x @ w + v)).sum())  # noqa: E731
    dX = plain.values(dY, fmt, 1, unit) @ plain.values(W, fmt, 1, unit).T
    dW = plain.values(X, fmt, 0, unit).T @ plain.values(dY, fmt, 0, unit)
    db = dY.sum(0)
    for i in range(6):
        for grad, at in ((dX, 0), (dW, 1), (db, 2)):
            args = [X, W, b]
            d = torch.randn(args[at].shape, dtype=torch.float64, generator=g)
            lo, hi = list(args), list(args)
            lo[at], hi[at] = args[at] - d / 2, args[at] + d / 2
            # the loss is linear in each: the difference is exact but for 64-bit rounding
            got, want = loss(*hi) - loss(*lo), float((grad * d).sum())
            assert abs(got - want) <= 1e-9 * (abs(want) + 1e3)

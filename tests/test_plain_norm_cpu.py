"""The plain 64-bit gradients of the norms and of the 8-bit linear layers against
central differences (CPU)."""
import itertools

import pytest
import torch

import plain_fp8
import plain_norm as plain

EPS, ALPHA = 1e-2, 0.7


@pytest.mark.parametrize("post,pre,gated", [
    (a, b, c) for a, b, c in itertools.product(["none", "rms", "layer"], ["none", "rms", "layer"],
                                               [False, True])])
def test_norm_gradients_are_the_differences(post, pre, gated):
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    T, h, L = 6, 10, 3
    v = {"X": r(T, h), "Z": r(T, h), "g1": 1 + 0.2 * r(h), "b1": r(h), "g2": 1 + 0.2 * r(h), "b2": r(h),
         "gate": r(T // L, h)}
    dOut, dXn = r(T, h), r(T, h)

    def rows(gate):
        return gate.repeat_interleave(L, 0) if gated else None

    def loss():
        out, _, _, _ = plain.forward(v["X"], v["Z"], post, v["g1"], v["b1"], rows(v["gate"]), ALPHA, EPS)
        t = (out * dOut).sum()
        if pre != "none":
            xn, _ = plain.normed(out, pre, v["g2"], v["b2"], *plain.stats_of(out, pre, EPS))
            t = t + (xn * dXn).sum()
        return t

    out, _, m1, r1 = plain.forward(v["X"], v["Z"], post, v["g1"], v["b1"], rows(v["gate"]), ALPHA, EPS)
    m2, r2 = plain.stats_of(out, pre, EPS)
    got = plain.backward(dOut, dXn, v["Z"], out, post, pre, v["g1"], v["b1"], rows(v["gate"]), v["g2"],
                         ALPHA, (m1, r1, m2, r2))
    names = {"X": "dX", "Z": "dZ"}
    if post != "none":
        names["g1"] = "dpost_gamma"
    if post == "layer":
        names["b1"] = "dpost_beta"
    if pre != "none":
        names["g2"] = "dpre_gamma"
    if pre == "layer":
        names["b2"] = "dpre_beta"
    if gated:
        names["gate"] = "dgate"
    for k, name in names.items():
        d = got[name][0]
        if name == "dgate":
            d = d.view(T // L, L, h).sum(1)
        elif name not in ("dX", "dZ"):
            d = d.sum(0)
        flat, e = v[k].view(-1), 1e-5
        for i in range(flat.numel()):
            keep = float(flat[i])
            flat[i] = keep + e
            up = float(loss())
            flat[i] = keep - e
            down = float(loss())
            flat[i] = keep
            # central differences of a smooth function: e^2 times its third derivative
            assert abs((up - down) / (2 * e) - float(d.reshape(-1)[i])) < 1e-6, (k, i)


def test_linear_gradients_are_the_differences():
    """dX = dY W^T and dW = X^T dY of the values that the 8-bit operands stand for:
    the product is linear in each, so differences of any size are exact."""
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    X = plain_fp8.rows_value(*(lambda q, s: (q, s.T))(*plain_fp8.quantize(r(5, 144), "e4m3", 1)))
    W = plain_fp8.block_value(*plain_fp8.quantize_block(r(144, 32), "e4m3"))
    dY = plain_fp8.cols_value(*plain_fp8.quantize(r(5, 32), "e5m2", 0))
    dX, dW = dY @ W.T, X.T @ dY
    for _ in range(20):
        eX, eW = r(5, 144).double(), r(144, 32).double()
        assert torch.allclose((dY * ((X + eX) @ W - X @ W)).sum(), (dX * eX).sum(), rtol=1e-10, atol=1e-9)
        assert torch.allclose((dY * (X @ (W + eW) - X @ W)).sum(), (dW * eW).sum(), rtol=1e-10, atol=1e-9)

"""Products of the 8-bit linear layers with every format in every place, and with scales
far from 1 that cancel."""
import itertools

import pytest
import torch

import plain_fp8 as plain
import test_gpu_fp8 as f8
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _layer(w, x_format, w_format, dy_format, seed, exponents=(0, 0, 0)):
    """A layer and its inputs, X, W and dY times 2^exponents."""
    from tensor_transformer_mlp_gemm_gb300 import fp8
    g = f8._gen(seed)
    ex, ew, ed = (2.0 ** e for e in exponents)
    col = w.split == "column"
    W = [f8._randn(g, *((w.in_features, w.shard) if col else (w.shard, w.out_features)), std=0.05 * ew)
         for _ in range(w.t)]
    q = [fp8.quantize_weight(x, w_format) for x in W]
    lay = fp8.DeviceFp8Linear(w, [x[0] for x in q], [x[1] for x in q], f8._randn(g, w.out_features, std=0.1),
                              x_format, w_format, dy_format)
    X = [f8._randn(g, *s, std=ex) for s in ([(w.tokens, w.in_features)] if col else [(w.tokens, w.shard)] * w.t)]
    dY = [f8._randn(g, *s, std=ed) for s in ([(w.tokens, w.shard)] * w.t if col else [(w.tokens, w.out_features)])]
    return lay, X, dY


# few tokens (16, 32, 64, 128, 256 of them a tile), and many
@pytest.mark.parametrize("T", [3, 30, 50, 100, 200, 700])
@pytest.mark.parametrize("split,din,dout,t", [("column", 400, 1296, 1), ("row", 1056, 784, 2)])
def test_formats(split, T, din, dout, t):
    for k, formats in enumerate(itertools.product(["e4m3", "e5m2"], repeat=3)):
        lay, X, dY = _layer(custom_linear(T, din, dout, t, split), *formats, seed=T + k)
        x = lay.quantize(X, cols=True)
        lay.forward(x)
        lay.backward(dY, x)
        f8._sync()
        f8._check_forward(lay, x)
        f8._check_backward(lay, x, dY, formats[2])


@pytest.mark.parametrize("T", [7, 150, 600])
@pytest.mark.parametrize("ex,ew", [(-108, 100), (100, -108)])
def test_scales_that_cancel(T, ex, ew):
    """Scales of 2^-120 and 2^90 in one product: its terms are ordinary numbers."""
    w = custom_linear(T, 528, 656, 1, "column")
    lay, X, dY = _layer(w, "e4m3", "e4m3", "e4m3", T, (ex, ew, ex))
    x = lay.quantize(X, cols=True)
    lay.forward(x)
    lay.backward(dY, x)
    f8._sync()
    f8._check_forward(lay, x)
    a, v = plain.rows_value(*_rows(dY[0])), plain.block_value(lay.Wq[0], lay.Ws[0]).T
    ref, bound = a @ v, plain.product_bound(a, v, -(-656 // 128))
    plain.check("dX", lay.dX[0], ref, bound + plain.BF16 * (ref.abs() + bound))
    lay, X, dY = _layer(w, "e4m3", "e4m3", "e4m3", T, (ex, 0, ew))
    x = lay.quantize(X, cols=True)
    lay.backward(dY, x)
    f8._sync()
    q, s = plain.quantize(dY[0], "e4m3", 0)
    a, v = plain.cols_value(x.cols, x.col_scale).T, plain.cols_value(q, s)
    plain.check("dW", lay.dW[0], a @ v, plain.product_bound(a, v, -(-T // 128)))


def _rows(dY):
    q, s = plain.quantize(dY, "e4m3", 1)
    return q, s.T

"""Waits of the 4-bit calls that run out: a loader that stops (on purpose, some copies into its
work) ends the kernel at the limit with a status, nothing of it is left under way, and the
next call is right."""
import pytest
import torch

import test_gpu_fp4 as f4
from test_gpu_fp8_norm_stalls import gives_up, stalled
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("copies", [0, 1, 3, 6])
@pytest.mark.parametrize("split,T,din,dout,t", [
    # (at least 8 stages of 256 for each CTA)
    ("column", 1, 32768, 1056, 1), ("row", 12, 16384, 512, 2), ("row", 20, 16384, 512, 2),
    ("column", 48, 16384, 4096, 2), ("column", 100, 16384, 4096, 1), ("column", 100, 16384, 12288, 1),
    ("column", 256, 16384, 512, 1)])
def test_few_tokens(split, T, din, dout, t, copies, fmt):
    w = custom_linear(T, din, dout, t, split)
    lay, X, _ = f4._layer(w, 5, fmt, backward=False)
    with stalled(copies):
        gives_up(lambda: lay.forward(X), 2)
    lay.forward(X)
    f4._sync()
    f4._check_forward(lay, X)


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("copies", [0, 1, 3, 5, 7])
@pytest.mark.parametrize("split,T,din,dout,t", [
    # (at least 8 stages a tile, of tokens too; more than one tile a CTA of the quantisation)
    ("column", 2100, 2304, 4128, 1), ("row", 2560, 4608, 2080, 2)])
def test_pairs(split, T, din, dout, t, copies, fmt):
    w = custom_linear(T, din, dout, t, split)
    lay, X, dY = f4._layer(w, 6, fmt)
    with stalled(copies):
        gives_up(lambda: lay.forward(X), 2)
    lay.forward(X, save=True)
    f4._sync()
    with stalled(copies):
        gives_up(lambda: lay.backward(dY), 3)
    lay.backward(dY)
    f4._sync()
    f4._check_forward(lay, X)
    f4._check_backward(lay, X, dY)


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("copies", [0, 1, 2])
def test_quantisation(copies, fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = f4._randn(f4._gen(1), 8192, 4096)
    g = torch.full((1,), 2.0 ** -9, device="cuda") if fmt == "nvfp4" else None
    with stalled(copies):
        gives_up(lambda: fp4.quantize_tokens(x, fmt, cols=True, scale=g))
    got = fp4.quantize_tokens(x, fmt, cols=True, scale=g)
    f4._sync()
    f4._check(got.rows, x, fmt, 1, None if g is None else float(g))
    f4._check(got.cols, x, fmt, 0, None if g is None else float(g))


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("copies", [0, 1, 3, 6])
@pytest.mark.parametrize("split,T,din,dout,t", [
    ("column", 333, 16384, 512, 1), ("row", 256, 16384, 4096, 2), ("column", 100, 2304, 12288, 1)])
def test_other_tiles(split, T, din, dout, t, copies, fmt):
    """Tiles of 256 tokens; pairs for 65 to 128 tokens."""
    w = custom_linear(T, din, dout, t, split)
    lay, X, _ = f4._layer(w, 5, fmt, backward=False)
    with stalled(copies):
        gives_up(lambda: lay.forward(X), 2)
    lay.forward(X)
    f4._sync()
    f4._check_forward(lay, X)

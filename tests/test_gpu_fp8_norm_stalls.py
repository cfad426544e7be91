"""Waits that run out: a loader that stops (on purpose, some copies into its work) ends the
kernel at the limit with a status, nothing of it is left under way, and the next call is
right.  A teardown that waited for what never comes would take its own limit of a second."""
import contextlib
import time

import pytest
import torch

import test_gpu_fp8 as f8
import test_gpu_norm as nm
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu

LIMIT_S = 0.03


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


@contextlib.contextmanager
def stalled(copies):
    from tensor_transformer_mlp_gemm_gb300 import binding
    binding.tpmlp_set_wait_timeout_ns(int(LIMIT_S * 1e9))
    binding.tpmlp_selftest_stall_loads(copies)
    try:
        yield
    finally:
        binding.tpmlp_selftest_stall_loads(-1)
        binding.tpmlp_set_wait_timeout_ns(2_000_000_000)


def gives_up(call, kernels=1):
    """call runs into the limit in `kernels` launches, each ending soon after."""
    from tensor_transformer_mlp_gemm_gb300 import binding
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    call()
    status = binding.tpmlp_sync_check()
    took = time.perf_counter() - t0
    assert status == binding.TPMLP_ERR_TIMEOUT
    # each wait of a kernel at most twice, one after the other
    assert LIMIT_S * 0.9 < took < kernels * LIMIT_S * 4 + 0.3, took


@pytest.mark.parametrize("copies", [0, 1, 3, 7])
@pytest.mark.parametrize("split,T,din,dout,t", [
    # (8 K blocks at least for each CTA)
    ("column", 1, 16384, 1040, 1), ("row", 20, 8192, 512, 2), ("column", 48, 8192, 4096, 2),
    ("column", 100, 8192, 4096, 1), ("column", 100, 8192, 12288, 1), ("column", 256, 8192, 512, 1)])
def test_few_tokens(split, T, din, dout, t, copies):
    w = custom_linear(T, din, dout, t, split)
    lay, X, dY = f8._layer(w, 5)
    x = lay.quantize(X)
    with stalled(copies):
        gives_up(lambda: lay.forward(x))
    lay.forward(x)
    f8._sync()
    f8._check_forward(lay, x)


@pytest.mark.parametrize("copies", [0, 1, 3, 6, 8])
@pytest.mark.parametrize("split,T,din,dout,t", [
    # (at least 9 K blocks a tile, of tokens too)
    ("column", 1100, 2048, 2064, 1), ("row", 1300, 2560, 1296, 2)])
def test_pairs(split, T, din, dout, t, copies):
    w = custom_linear(T, din, dout, t, split)
    lay, X, dY = f8._layer(w, 6)
    x = lay.quantize(X, cols=True)
    with stalled(copies):
        gives_up(lambda: lay.forward(x))
        gives_up(lambda: lay.backward(dY, x), 2)
    lay.forward(x)
    lay.backward(dY, x)
    f8._sync()
    f8._check_forward(lay, x)
    f8._check_backward(lay, x, dY, "e4m3")


@pytest.mark.parametrize("copies", [17, 31, 40])
def test_pairs_in_a_later_tile(copies):
    w = custom_linear(2560, 2048, 8192, 1, "column")      # 320 tiles of 16 K blocks
    lay, X, _ = f8._layer(w, 7)
    x = lay.quantize(X)
    with stalled(copies):
        gives_up(lambda: lay.forward(x))
    lay.forward(x)
    f8._sync()
    f8._check_forward(lay, x)


@pytest.mark.parametrize("copies", [0, 1, 2, 5])
@pytest.mark.parametrize("h,gate_rows,post,pre,quantize", [
    (4096, 512, "rms", "rms", "e4m3"), (4096, 0, None, "layer", None), (1040, 0, "layer", "none", None),
    (64, 0, "none", "none", None), (16384, 8192, "layer", "layer", None)])
def test_norm_forward(h, gate_rows, post, pre, quantize, copies):
    T = 8192                              # (at least 6 rows for each CTA)
    d = nm._inputs(T, h, gate_rows, 8)
    lay = nm._layer(d, T, h, post or "none", pre, gate_rows, 0.75, quantize=quantize)
    z = post is not None
    call = lambda: lay.forward(d["X"], d["Z"] if z else None, d["gate"])  # noqa: E731
    with stalled(copies):
        gives_up(call)
    call()
    nm._sync()
    nm._check_forward(d, lay, lay.Out if z else None, lay.Xn, lay.stats, z=z)


@pytest.mark.parametrize("copies", [0, 1, 2, 5])
@pytest.mark.parametrize("T,h,gate_rows,post,pre", [
    # (6 pairs of rows at least for each group of threads); post None: no block before
    (16384, 512, 2048, "rms", "rms"), (8192, 1024, 0, "none", "none"), (4096, 4096, 512, "layer", "layer"),
    (4096, 4096, 0, None, "rms"), (4096, 4096, 4096, "rms", "none"),
    # clusters: the CTAs that load go on until their sums do not come
    (2048, 6144, 512, "layer", "rms"), (2048, 8192, 512, "rms", "rms"), (2048, 9000, 0, None, "layer"),
    (2048, 12288, 512, "rms", "rms"), (2048, 12288, 0, "none", "none"), (1024, 12288, 0, "rms", "none"),
    (1024, 16384, 512, "layer", "layer")])
def test_norm_backward(T, h, gate_rows, post, pre, copies):
    d = nm._inputs(T, h, gate_rows, 9)
    lay = nm._layer(d, T, h, post or "none", pre, gate_rows, 0.75)
    z, dXn = post is not None, d["dXn"] if pre != "none" else None
    lay.forward(d["X"], d["Z"] if z else None, d["gate"])
    Out = lay.Out if z else d["X"]
    call = lambda: lay.backward(d["dOut"], dXn, d["Z"] if z else None, Out, gate=d["gate"])  # noqa: E731
    lay._gradients()
    with stalled(copies):
        gives_up(call)
    call()
    nm._sync()
    nm._check_backward(d, lay, Out, lay.stats, d["dOut"], dXn, z=z)

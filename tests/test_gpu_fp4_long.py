"""4-bit matrices whose summed axis is so long that offsets along it pass 2^31 and 2^32 bytes."""
import gc

import pytest
import torch

import plain_fp4 as plain
import test_gpu_fp4 as f4
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


@pytest.fixture(autouse=True)
def _room():
    """(up to 150 GB in a test)"""
    gc.collect()
    torch.cuda.empty_cache()
    yield
    gc.collect()
    torch.cuda.empty_cache()


# where the bytes of scales of 128 rows, times 128 of K 512 (mx) or 1024 (nv), pass 2^32
PAST = {"mxfp4": (1 << 30) + 512, "nvfp4": (1 << 29) + 512}
PERIOD = 1 << 16


def _periodic(m, x):
    """A matrix made of a piece of PERIOD along its summed axis, again and again, and of the start of
    one at the end: so are its values and scales."""
    for got, one, step in ((m.q, x.q, PERIOD // 2), (m.s.view(1, -1), x.s.view(1, -1), x.s.numel())):
        whole = got.shape[1] // step
        assert torch.equal(got[:, :step], one[:, :step])
        for k in range(1, whole):
            if not torch.equal(got[:, k * step:(k + 1) * step], one[:, :step]):
                pytest.fail(f"piece {k} of {whole}")
        rest = got.shape[1] - whole * step
        assert rest > 0 and torch.equal(got[:, whole * step:], one[:, :rest])


@pytest.mark.parametrize("fmt", f4.FORMATS)
def test_quantise_rows(fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    K = PAST[fmt]
    piece = f4._values(1, PERIOD, f4._gen(1))
    scale = None if fmt == "mxfp4" else torch.full((1,), 2.0 ** -3, device="cuda")
    one = fp4.quantize_tokens(piece, fmt, scale=scale).rows
    f4._check(one, piece, fmt, 1, None if scale is None else 2.0 ** -3)
    x = torch.cat([piece.repeat(1, K // PERIOD), piece[:, :K % PERIOD]], 1)
    got = fp4.quantize_tokens(x, fmt, scale=scale).rows
    f4._sync()
    _periodic(got, one)


@pytest.mark.parametrize("fmt", f4.FORMATS)
def test_quantise_columns(fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    T = PAST[fmt]
    piece = f4._values(PERIOD, 32, f4._gen(2))
    scale = None if fmt == "mxfp4" else torch.full((1,), 2.0 ** -3, device="cuda")
    one = fp4.quantize_tokens(piece, fmt, rows=False, cols=True, scale=scale).cols
    f4._check(one, piece, fmt, 0, None if scale is None else 2.0 ** -3)
    x = torch.empty(T, 32, dtype=torch.bfloat16, device="cuda")
    x[:T // PERIOD * PERIOD].view(-1, PERIOD, 32).copy_(piece.expand(T // PERIOD, -1, -1))
    x[T // PERIOD * PERIOD:] = piece[:T % PERIOD]
    got = fp4.quantize_tokens(x, fmt, rows=False, cols=True, scale=scale).cols
    f4._sync()
    _periodic(got, one)


# features in whose scales' bytes of 128 rows pass 2^31
LONG = {"mxfp4": (1 << 29) + 1024, "nvfp4": (1 << 28) + 1024}
END = 4096


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("split,T,t", [("column", 1, 1), ("row", 20, 1), ("row", 40, 2)])
def test_few_tokens(split, T, t, fmt):
    """A layer of so many features in that the scales of its last ones lie past 2^31 bytes: X is zero
    but for the first and the last of each shard, whose products are those of 8192 of K."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    din, dout = LONG[fmt], 32
    n = din // t
    g = f4._gen(T)
    ends = [[f4._randn(g, END, dout, std=0.05) for _ in range(2)] for _ in range(t)]
    W = []
    for a, b in ends:
        w = torch.zeros(n, dout, dtype=torch.bfloat16, device="cuda")
        w[:END], w[-END:] = a, b
        w[END:-END].fill_(0.01)           # (scales of their own in between)
        W.append(w)
    weights = fp4.quantize_weight(W, fmt)
    del W, w
    X, kept = [], []
    for _ in range(t):
        x = torch.zeros(T, n, dtype=torch.bfloat16, device="cuda")
        x[:, :END], x[:, -END:] = f4._randn(g, T, END), f4._randn(g, T, END)
        X.append(x)
        kept += [x[:, :END], x[:, -END:]]
    lay = fp4.DeviceFp4Linear(custom_linear(T, din, dout, t, split), weights, f4._randn(g, dout, std=0.1))
    lay.forward(X)
    f4._sync()
    gx = None if fmt == "mxfp4" else plain.tensor_scale([torch.cat(kept, 1)])
    gw = weights.scale
    a = torch.cat([plain.values(x, fmt, 1, gx) for x in kept], 1)
    v = torch.cat([plain.values(w, fmt, 0, gw) for pair in ends for w in pair], 0)
    ref = a @ v + lay.b.double()
    # (what X is zero for adds zeros, without a rounding)
    bound = plain.product_bound(a, v, a.shape[1] // 64) + 2 * plain.F32 * ref.abs()
    plain.check("Y", lay.Y[0], ref, bound + plain.BF16 * (ref.abs() + bound))

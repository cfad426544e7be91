"""The 8-bit calls on the GPU against plain 64-bit forms: quantisation value for
value, the linear layers within bounds that follow from their roundings (one
bf16 rounding of the output, fp32 sums inside)."""
import pytest
import torch

import plain_fp8 as plain
from guard import GuardBands
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _randn(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _same(got, ref):
    """Equal value for value, NaN in the same places (and nothing long to print)."""
    return bool(((got.double() == ref) | (torch.isnan(got.double()) & torch.isnan(ref))).all())


def _sync():
    from tensor_transformer_mlp_gemm_gb300 import binding
    assert binding.tpmlp_sync_check() == binding.TPMLP_OK


# ---- quantisation -----------------------------------------------------------------------

def _values(T, C, gen):
    """Activations over many magnitudes, with zeros, subnormals and single large features."""
    x = torch.randn(T, C, generator=gen, device="cuda")
    x = x * torch.pow(2.0, torch.randint(-20, 20, (T, 1), generator=gen, device="cuda").float())
    x[:, ::37] *= 64
    x[T // 2] = 0
    x[T // 3] *= 2.0 ** -110
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("T,C", [(1, 16), (1, 4096), (3, 272), (127, 128), (128, 144), (129, 1040),
                                 (1000, 2064)])
def test_quantize_tokens(T, C, fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp8
    x = _values(T, C, _gen(T * 31 + C))
    both = fp8.quantize_tokens(x, fmt, rows=True, cols=True)
    rows = fp8.quantize_tokens(x, fmt, rows=True, cols=False)
    cols = fp8.quantize_tokens(x, fmt, rows=False, cols=True)
    _sync()
    q, s = plain.quantize(x, fmt, 1)
    for got in (both, rows):
        assert _same(got.rows, q) and _same(got.row_scale, s.T)
    q, s = plain.quantize(x, fmt, 0)
    for got in (both, cols):
        assert _same(got.cols, q) and _same(got.col_scale, s)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("r,c", [(16, 16), (128, 128), (130, 272), (1040, 1000 + 8)])
def test_quantize_weight(r, c, fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp8
    w = _values(r, c, _gen(r + c))
    got_q, got_s = fp8.quantize_weight(w, fmt)
    _sync()
    q, s = plain.quantize_block(w, fmt)
    assert _same(got_q, q) and _same(got_s, s)


@pytest.mark.parametrize("top,bits", [(448.0, "e4m3"), (57344.0, "e5m2")])
def test_quantize_scale_borders(top, bits):
    """Group maxima at, just below and just above s * top, at the smallest scale,
    and the largest finite bf16."""
    from tensor_transformer_mlp_gemm_gb300 import fp8
    x = torch.zeros(8, 128, device="cuda")
    for r, v in enumerate([top, top * (1 + 2.0 ** -7), top * (1 - 2.0 ** -7), top / 2,
                           2.0 ** -119 * top, 2.0 ** -133, 3.3895313892515355e38, 1.0]):
        x[r, 5], x[r, 77] = v, -v / 3
    x = x.to(torch.bfloat16)
    got = fp8.quantize_tokens(x, bits)
    _sync()
    q, s = plain.quantize(x, bits, 1)
    assert _same(got.rows, q) and _same(got.row_scale, s.T)


def test_quantize_not_finite():
    """A group with an infinity or a NaN: scale NaN, zeros; its neighbours as ever."""
    from tensor_transformer_mlp_gemm_gb300 import fp8
    x = _randn(_gen(3), 300, 272)
    x[5, 200], x[140, 3], x[140, 4] = float("inf"), float("nan"), float("-inf")
    got = fp8.quantize_tokens(x, "e4m3", cols=True)
    w_q, w_s = fp8.quantize_weight(x, "e5m2")
    _sync()
    for dim, q, s in ((1, got.rows, got.row_scale.T), (0, got.cols, got.col_scale)):
        rq, rs = plain.quantize(x, "e4m3", dim)
        assert _same(q, rq) and _same(s, rs)
        assert int(torch.isnan(s).sum()) == (2 if dim == 1 else 3)
    rq, rs = plain.quantize_block(x, "e5m2")
    assert _same(w_q, rq) and _same(w_s, rs)


def test_quantize_chunks_and_shards():
    from tensor_transformer_mlp_gemm_gb300 import fp8
    x = _randn(_gen(4), 1024, 400)
    whole = fp8.quantize_tokens(x, cols=True)
    parts = fp8.quantize_tokens([c.clone() for c in x.chunk(4)], cols=True)
    _sync()
    for a in ("rows", "row_scale", "cols", "col_scale"):
        u, v = getattr(whole, a), getattr(parts, a)
        assert bool((u.view(torch.uint8) == v.view(torch.uint8)).all())
    shards = [_randn(_gen(5 + i), 77, 48) for i in range(8)]
    got = fp8.quantize_shards(shards, "e5m2", cols=True)
    _sync()
    for x, g in zip(shards, got):
        one = fp8.quantize_tokens(x, "e5m2", cols=True)
        _sync()
        for a in ("rows", "row_scale", "cols", "col_scale"):
            assert bool((getattr(one, a).view(torch.uint8) == getattr(g, a).view(torch.uint8)).all())


# ---- the linear layers --------------------------------------------------------------------

def _layer(w, seed, dy="e4m3", std_x=1.0):
    from tensor_transformer_mlp_gemm_gb300 import fp8
    g = _gen(seed)
    col = w.split == "column"
    wshape = (w.in_features, w.shard) if col else (w.shard, w.out_features)
    W = [_randn(g, *wshape, std=0.05) for _ in range(w.t)]
    b = _randn(g, w.out_features, std=0.1)
    q = [fp8.quantize_weight(x) for x in W]
    lay = fp8.DeviceFp8Linear(w, [x[0] for x in q], [x[1] for x in q], b, dy_format=dy)
    if col:
        X = [_randn(g, w.tokens // w.seq_chunks, w.in_features, std=std_x)
             for _ in range(w.seq_chunks)]
        dY = [_randn(g, w.tokens, w.shard) for _ in range(w.t)]
    else:
        X = [_randn(g, w.tokens, w.shard, std=std_x) for _ in range(w.t)]
        dY = [_randn(g, w.tokens // w.seq_chunks, w.out_features) for _ in range(w.seq_chunks)]
    return lay, X, dY


def _check_forward(lay, x):
    w, col = lay.w, lay.column
    V = [plain.block_value(q, s) for q, s in zip(lay.Wq, lay.Ws)]
    b = lay.b.double()
    xs = [x] if col else x
    A = [plain.rows_value(v.rows, v.row_scale) for v in xs]
    if col:
        got = torch.cat(lay.Y, 1)
        a, v = A[0], torch.cat(V, 1)
    else:
        got = torch.cat(lay.Y, 0)
        a, v = torch.cat(A, 1), torch.cat(V, 0)
    ref = a @ v + b
    blocks = sum(-(-m.shape[1] // 128) for m in A)
    bound = plain.product_bound(a, v, blocks) + 2 * plain.F32 * ref.abs()
    plain.check("Y", got, ref, bound + plain.BF16 * (ref.abs() + bound))


def _check_backward(lay, x, dY, fmt):
    w, col = lay.w, lay.column
    V = [plain.block_value(q, s) for q, s in zip(lay.Wq, lay.Ws)]
    xs = [x] if col else x
    A = [plain.cols_value(v.cols, v.col_scale) for v in xs]
    D = dY if col else [torch.cat(dY, 0)]
    rows = [plain.rows_value(q, s.T) for q, s in (plain.quantize(d, fmt, 1) for d in D)]
    cols = [plain.cols_value(q, s) for q, s in (plain.quantize(d, fmt, 0) for d in D)]
    tb = -(-w.tokens // 128)
    if col:
        pairs = [(torch.cat(rows, 1), torch.cat(V, 1).T, torch.cat(lay.dX, 0),
                  sum(-(-d.shape[1] // 128) for d in rows))]
        dw = [(A[0].T, c, g) for c, g in zip(cols, lay.dW)]
    else:
        pairs = [(rows[0], v.T, g, -(-w.out_features // 128)) for v, g in zip(V, lay.dX)]
        dw = [(a.T, cols[0], g) for a, g in zip(A, lay.dW)]
    for a, v, got, blocks in pairs:
        ref, bound = a @ v, plain.product_bound(a, v, blocks)
        plain.check("dX", got, ref, bound + plain.BF16 * (ref.abs() + bound))
    for a, v, got in dw:
        plain.check("dW", got, a @ v, plain.product_bound(a, v, tb))
    # a column sum: at most 17 additions in 128 rows, then tb / 16 + 17 more
    d = torch.cat([x.double() for x in D], 1)
    plain.check("db", lay.db, d.sum(0), (34 + tb / 16 + 1) * plain.F32 * d.abs().sum(0))


SHAPES = [
    # split, T, in, out, t, chunks
    ("column", 1, 256, 256, 1, 1),
    ("row", 1, 256, 256, 2, 1),
    ("column", 1, 4096, 1040, 1, 1),
    ("column", 16, 272, 2064, 1, 1),
    ("row", 17, 1040, 400, 1, 1),
    ("row", 48, 4096, 1024, 8, 1),
    ("column", 64, 16, 16, 1, 1),
    ("column", 65, 144, 272, 1, 1),
    ("column", 128, 2048, 4096, 2, 1),
    ("row", 200, 2080, 1296, 5, 1),
    ("column", 256, 1024, 2048, 8, 2),
    ("row", 333, 1032 * 2, 272, 3, 1),
    ("column", 333, 272, 48 * 43, 3, 1),
    ("row", 512, 1024, 256, 4, 4),
    ("column", 1024, 512, 2048, 8, 8),
    ("row", 1537, 2048, 2304, 1, 1),
    ("column", 2100, 1296, 4112, 1, 1),
]


@pytest.mark.parametrize("split,T,din,dout,t,chunks", SHAPES)
def test_linear(split, T, din, dout, t, chunks):
    w = custom_linear(T, din, dout, t, split, seq_chunks=chunks)
    lay, X, dY = _layer(w, T + din + dout)
    g = GuardBands()
    g.guard(lay, ["Y", "dX", "ws"])
    lay._grads = tuple(([g.like(x, f"dW[{i}]") for i, x in enumerate(lay.dW)],
                        g.like(lay.db, "db")))
    g.watch_inputs(lay, ["Wq", "Ws", "b"])
    x = lay.quantize(X, cols=True)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()
    g.check()
    _check_forward(lay, x)
    _check_backward(lay, x, dY, "e4m3")


@pytest.mark.parametrize("split,T,din,dout,t", [
    ("column", 3, 400, 784, 1), ("row", 40, 784, 400, 1), ("column", 130, 528, 1056, 2),
    ("row", 700, 1552, 656, 1), ("column", 515, 656, 1040, 1)])
def test_linear_scales_of_every_row(split, T, din, dout, t):
    """Every token, feature and weight block at a magnitude of its own, so that a
    scale taken from a wrong row, column or block shows."""
    from tensor_transformer_mlp_gemm_gb300 import fp8
    w = custom_linear(T, din, dout, t, split)
    lay, X, dY = _layer(w, 77)
    g = _gen(78)

    def spread(x, rows, cols):
        def f(n, step):
            e = torch.randint(-12, 13, (-(-n // step),), generator=g, device="cuda")
            return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e).repeat_interleave(step)[:n]
        return (x.float() * f(x.shape[0], rows)[:, None] * f(x.shape[1], cols)).to(torch.bfloat16)

    X = [spread(x, 1, 1) for x in X]
    dY = [spread(x, 1, 1) for x in dY]
    for i in range(t):
        W = spread(_randn(g, *lay.Wq[i].shape), 128, 128)
        q, s = fp8.quantize_weight(W)
        lay.Wq[i].copy_(q)
        lay.Ws[i].copy_(s)
    x = lay.quantize(X, cols=True)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()
    _check_forward(lay, x)
    _check_backward(lay, x, dY, "e4m3")


@pytest.mark.parametrize("T", [9, 300])
def test_linear_not_finite(T):
    """NaN where, and only where, a group that is not finite takes part."""
    w = custom_linear(T, 400, 528, 1, "column")
    lay, X, dY = _layer(w, 21)
    X[0][3, 200] = float("inf")
    dY[0][5, 7] = float("nan")
    x = lay.quantize(X, cols=True)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()
    nan = torch.isnan(lay.Y[0])
    assert nan[3].all() and int(nan.sum()) == w.out_features
    nan = torch.isnan(lay.dX[0])
    assert nan[5].all() and int(nan.sum()) == w.in_features
    nan = torch.isnan(lay.dW[0])
    assert nan[200].all() and nan[:, 7].all()
    assert int(nan.sum()) == w.in_features + w.out_features - 1
    assert torch.isnan(lay.db[7]) and int(torch.isnan(lay.db).sum()) == 1


@pytest.mark.parametrize("T", [4, 260])
def test_linear_other_scales_read_as_nan(T):
    """A scale that is not a positive power of two is never taken for another."""
    w = custom_linear(T, 256, 384, 1, "column")
    lay, X, _ = _layer(w, 31)
    x = lay.quantize(X)
    for j, bad in enumerate([0.75, -1.0, 0.0]):
        keep = float(lay.Ws[0][1, 1])
        lay.Ws[0][1, 1] = bad
        lay.forward(x)
        _sync()
        nan = torch.isnan(lay.Y[0])
        assert nan[:, 128:256].all() and int(nan.sum()) == T * 128, bad
        lay.Ws[0][1, 1] = keep


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("split", ["column", "row"])
def test_linear_mixed_formats(split, T):
    """e4m3 activations and weights, e5m2 gradients."""
    w = custom_linear(T, 528, 784, 1, split)
    lay, X, dY = _layer(w, 9, dy="e5m2")
    x = lay.quantize(X, cols=True)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()
    _check_forward(lay, x)
    _check_backward(lay, x, dY, "e5m2")

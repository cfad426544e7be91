"""The 4-bit calls on the GPU against plain 64-bit forms: quantisation value for value and
byte for byte, the linear layers within bounds that follow from their roundings (one bf16
rounding of the output, fp32 sums inside)."""
import pytest
import torch

import plain_fp4 as plain
from guard import GuardBands
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu
FORMATS = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _sync():
    from tensor_transformer_mlp_gemm_gb300 import binding
    assert binding.tpmlp_sync_check() == binding.TPMLP_OK


def _same(a, b):
    return a.shape == b.shape and bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


def _values(T, C, gen):
    """Magnitudes over many powers of two, zeros, and whole groups of zeros."""
    x = torch.randn(T, C, generator=gen, device="cuda")
    e = torch.randint(-14, 15, (T, -(-C // 8)), generator=gen, device="cuda").repeat_interleave(8, 1)[:, :C]
    x = torch.ldexp(x, e)
    x[torch.rand(T, C, generator=gen, device="cuda") < 0.1] = 0
    x[:, C // 2:C // 2 + 32] = 0
    return x.to(torch.bfloat16)


def _check(m, x, fmt, dim, g):
    q, s = plain.quantize(x, fmt, dim, g)
    if dim == 0:
        q, s = q.T, s.T
    got_q, got_s = plain.unpack(m)
    assert _same(got_q, q) and _same(got_s, s)
    want = torch.where(torch.isnan(s), torch.nan, q * s * (1.0 if g is None else float(g)))
    assert _same(m.values().double(), want.to(torch.bfloat16).double())


# ---- quantisation ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,C", [(1, 32), (1, 4096), (3, 288), (31, 64), (33, 96), (127, 128), (128, 160),
                                 (129, 1056), (257, 256), (1000, 2080)])
def test_quantize_tokens(T, C, fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = _values(T, C, _gen(T * 31 + C))
    both = fp4.quantize_tokens(x, fmt, rows=True, cols=True)
    rows = fp4.quantize_tokens(x, fmt, rows=True, cols=False)
    cols = fp4.quantize_tokens(x, fmt, rows=False, cols=True)
    _sync()
    g = None
    if fmt == "nvfp4":
        g = plain.tensor_scale([x])
        for m in (both.rows, both.cols, rows.rows, cols.cols):
            assert float(m.scale) == float(g)
    for m in (both.rows, rows.rows):
        _check(m, x, fmt, 1, g)
    for m in (both.cols, cols.cols):
        _check(m, x, fmt, 0, g)
    assert rows.cols is None and cols.rows is None


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,C", [(5, 96), (129, 288)])
def test_what_fills_up(T, C, fmt):
    """Behind the last token values are zero and scales the smallest, in every byte."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = fp4.quantize_tokens(_randn(_gen(1), T, C), fmt, cols=True)
    _sync()
    size = plain.GROUP[fmt]
    for m in (x.rows, x.cols):
        R, K = m.shape
        assert m.q.shape[1] == -(-K // 32) * 16
        b = m.q.to(torch.int64)
        n = torch.stack([b & 15, b >> 4], 2).flatten(1)
        assert bool((n[:, K:] & 7 == 0).all())
        kb, blocks = -(-K // 256), 64 // size
        s = m.s.to(torch.int64).view(-1, kb, blocks, 32, 4, 4).permute(0, 4, 3, 1, 2, 5)
        s = s.reshape(-1, kb * blocks * 4)
        assert bool((s[R:] == 1).all()) and bool((s[:, -(-K // size):] == 1).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_borders(fmt):
    """Every bf16 significand over the borders between 4-bit values, for every scale
    significand: ties go to even, their neighbours to the nearer."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    size = plain.GROUP[fmt]
    tops = (torch.arange(128, 256, device="cuda").float() / 32)       # 4 .. 8: the groups' largest
    rest = torch.arange(128, 256, device="cuda").float()
    rows = []
    for k in range(-6, 0):                                            # 2^k .. of the top
        for c in range(0, 128, size - 1):
            part = rest[c:c + size - 1] / 128 * 2.0 ** (k + 2)
            x = torch.zeros(len(tops), size, device="cuda")
            x[:, 0] = tops
            x[:, 1:1 + len(part)] = torch.minimum(part, tops[:, None])
            x[:, 1::2] *= -1
            rows.append(x)
    x = torch.cat(rows)
    x = torch.nn.functional.pad(x, (0, 32 - size)).to(torch.bfloat16)
    for scale in ([None] if fmt == "mxfp4" else [2.0 ** -8, 2.0 ** -2, 1.0]):
        g = None if scale is None else torch.full((1,), scale, device="cuda")
        got = fp4.quantize_tokens(x, fmt, cols=True, scale=g)
        _sync()
        _check(got.rows, x, fmt, 1, scale)
        _check(got.cols, x, fmt, 0, scale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_extremes(fmt):
    """The largest and smallest bf16 values, groups at the scale's limits."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = torch.zeros(8, 64, device="cuda")
    big = 3.3895313892515355e38
    for r, v in enumerate([6.0, 6.0 * (1 + 2.0 ** -7), 2.0 ** -126, 2.0 ** -133, 448.0 * 6, 2.0 ** 126, 1.0, 2.0 ** -9]):
        x[r, 5], x[r, 40] = v, -v / 3
    for x in (x, torch.where(x == 6.0, big, x)):
        x = x.to(torch.bfloat16)
        got = fp4.quantize_tokens(x, fmt, cols=True)
        _sync()
        g = None if fmt == "mxfp4" else plain.tensor_scale([x])
        for m, dim in ((got.rows, 1), (got.cols, 0)):
            q, s = plain.quantize(x, fmt, dim, g)
            gq, gs = plain.unpack(m)
            assert _same(gq, q.T if dim == 0 else q) and _same(gs, s.T if dim == 0 else s)


@pytest.mark.parametrize("scale", [2.0 ** -110, 2.0 ** -20, 2.0 ** 20, 2.0 ** 117])
def test_given_scales_out_of_range(scale):
    """A given scale that leaves groups out of range: they get the largest or smallest."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = _values(40, 96, _gen(9))
    got = fp4.quantize_tokens(x, "nvfp4", cols=True, scale=torch.full((1,), scale, device="cuda"))
    _sync()
    for m, dim in ((got.rows, 1), (got.cols, 0)):
        q, s = plain.quantize(x, "nvfp4", dim, scale)
        gq, gs = plain.unpack(m)
        assert _same(gq, q.T if dim == 0 else q) and _same(gs, s.T if dim == 0 else s)


@pytest.mark.parametrize("bad", [0.0, 0.75, -1.0, float("nan"), float("inf"), 2.0 ** -111, 2.0 ** 118])
def test_other_scales_read_as_nan(bad):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = fp4.quantize_tokens(_randn(_gen(2), 5, 64), "nvfp4", scale=torch.full((1,), bad, device="cuda"))
    _sync()
    assert bool(torch.isnan(x.rows.values()).all())
    assert bool((plain.unpack(x.rows)[0] == 0).all())


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_not_finite(fmt):
    """A group with an infinity or a NaN: scale NaN, zeros; its neighbours as ever."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = _randn(_gen(3), 300, 288)
    x[5, 200], x[140, 3], x[140, 4] = float("inf"), float("nan"), float("-inf")
    got = fp4.quantize_tokens(x, fmt, cols=True)
    _sync()
    g = None if fmt == "mxfp4" else plain.tensor_scale([x])
    _check(got.rows, x, fmt, 1, g)
    _check(got.cols, x, fmt, 0, g)
    size = plain.GROUP[fmt]
    assert int(torch.isnan(got.rows.values()).sum()) == 2 * size
    assert int(torch.isnan(got.cols.values()).sum()) == 3 * size


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_chunks_and_shards(fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = _randn(_gen(4), 640, 416)
    whole = fp4.quantize_tokens(x, fmt, cols=True)
    parts = fp4.quantize_tokens([c.clone() for c in x.chunk(5)], fmt, cols=True)
    _sync()
    for a, b in ((whole.rows, parts.rows), (whole.cols, parts.cols)):
        assert bool((a.q == b.q).all()) and bool((a.s == b.s).all())
    W = [_randn(_gen(5 + i), 96, 160, std=0.1 * (i + 1)) for i in range(8)]
    got = fp4.quantize_weight(W, fmt, backward=True)
    one = fp4.quantize_weight(W, fmt)
    _sync()
    g = None if fmt == "mxfp4" else plain.tensor_scale(W)
    assert one.backward is None and (g is None or float(got.scale) == float(g))
    for i, w in enumerate(W):
        _check(got.forward[i], w, fmt, 0, g)
        _check(one.forward[i], w, fmt, 0, g)
        _check(got.backward[i], w, fmt, 1, g)


# ---- the linear layers --------------------------------------------------------------------

def _layer(w, seed, fmt, backward=True, x_scale=None, W=None):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    g = _gen(seed)
    col = w.split == "column"
    wshape = (w.in_features, w.shard) if col else (w.shard, w.out_features)
    W = W or [_randn(g, *wshape, std=0.05) for _ in range(w.t)]
    b = _randn(g, w.out_features, std=0.1)
    lay = fp4.DeviceFp4Linear(w, fp4.quantize_weight(W, fmt, backward=backward), b, x_scale=x_scale)
    if col:
        X = [_randn(g, w.tokens // w.seq_chunks, w.in_features) for _ in range(w.seq_chunks)]
        dY = [_randn(g, w.tokens, w.shard, std=1e-3) for _ in range(w.t)]
    else:
        X = [_randn(g, w.tokens, w.shard) for _ in range(w.t)]
        dY = [_randn(g, w.tokens // w.seq_chunks, w.out_features, std=1e-3) for _ in range(w.seq_chunks)]
    return lay, X, dY


def _whole(lay, parts, token_chunks):
    return [torch.cat(parts, 0)] if token_chunks else parts


def _scale(lay, parts):
    return None if lay.fmt == "mxfp4" else plain.tensor_scale(parts)


def _check_forward(lay, X, Y=None):
    col, Y = lay.column, lay.Y if Y is None else Y
    g = _scale(lay, X) if lay.x_scale is None else float(lay.x_scale)
    A = [plain.values(x, lay.fmt, 1, g) for x in _whole(lay, X, col)]
    V = [plain.value(m).T for m in lay.weights.forward]
    if col:
        got, a, v = torch.cat(Y, 1), A[0], torch.cat(V, 1)
    else:
        got, a, v = torch.cat(Y, 0), torch.cat(A, 1), torch.cat(V, 0)
    ref = a @ v + lay.b.double()
    blocks = sum(-(-m.shape[1] // 256) * 4 for m in A)
    bound = plain.product_bound(a, v, blocks) + 2 * plain.F32 * ref.abs()
    plain.check("Y", got, ref, bound + plain.BF16 * (ref.abs() + bound))


def _check_backward(lay, X, dY):
    w, col, fmt = lay.w, lay.column, lay.fmt
    gx = _scale(lay, X) if lay.x_scale is None else float(lay.x_scale)
    gd = _scale(lay, dY)
    A = [plain.values(x, fmt, 0, gx) for x in _whole(lay, X, col)]
    D = _whole(lay, dY, not col)
    rows = [plain.values(d, fmt, 1, gd) for d in D]
    cols = [plain.values(d, fmt, 0, gd) for d in D]
    V = [plain.value(m) for m in lay.weights.backward]
    tb = -(-w.tokens // 256) * 4
    if col:
        pairs = [(torch.cat(rows, 1), torch.cat(V, 1).T, torch.cat(lay.dX, 0),
                  sum(-(-d.shape[1] // 256) * 4 for d in rows))]
        dw = [(A[0].T, c, g) for c, g in zip(cols, lay.dW)]
    else:
        pairs = [(rows[0], v.T, g, -(-w.out_features // 256) * 4) for v, g in zip(V, lay.dX)]
        dw = [(a.T, cols[0], g) for a, g in zip(A, lay.dW)]
    for a, v, got, blocks in pairs:
        ref, bound = a @ v, plain.product_bound(a, v, blocks)
        plain.check("dX", got, ref, bound + plain.BF16 * (ref.abs() + bound))
    for a, v, got in dw:
        plain.check("dW", got, a @ v, plain.product_bound(a, v, tb))
    # a column sum: 33 additions in 128 rows, then at most t128 / 16 + 17 more
    d = torch.cat([x.double() for x in D], 1)
    t128 = -(-w.tokens // 128)
    plain.check("db", lay.db, d.sum(0), (33 + 17 + t128 / 16 + 1) * plain.F32 * d.abs().sum(0))


SHAPES = [
    # split, T, in, out, t, chunks
    ("column", 1, 256, 256, 1, 1),
    ("row", 1, 256, 256, 2, 1),
    ("column", 1, 4096, 1056, 1, 1),
    ("column", 16, 288, 2080, 1, 1),
    ("row", 17, 1056, 416, 1, 1),
    ("row", 48, 4096, 1024, 8, 1),
    ("column", 64, 32, 32, 1, 1),
    ("column", 65, 160, 288, 1, 1),
    ("column", 128, 2048, 4096, 2, 1),
    ("row", 200, 2080, 1312, 5, 1),
    ("column", 256, 1024, 2048, 8, 2),
    ("row", 333, 2112, 288, 3, 1),
    ("column", 333, 288, 96 * 43, 3, 1),
    ("row", 512, 1024, 256, 4, 4),
    ("column", 1024, 512, 2048, 8, 8),
    ("row", 1537, 2048, 2304, 1, 1),
    ("column", 2100, 1312, 4128, 1, 1),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("split,T,din,dout,t,chunks", SHAPES)
def test_linear(split, T, din, dout, t, chunks, fmt):
    w = custom_linear(T, din, dout, t, split, seq_chunks=chunks)
    lay, X, dY = _layer(w, T + din + dout, fmt)
    g = GuardBands()
    g.guard(lay, ["Y", "dX", "ws"])
    dW = [g.like(x, f"dW[{i}]") for i, x in enumerate(lay.dW)]
    from tensor_transformer_mlp_gemm_gb300.fp8 import _pointers
    lay._grads = (dW, g.like(lay.db, "db"), _pointers(dW))
    g.watch_inputs(lay, ["b"])
    lay.forward(X, save=True)
    lay.backward(dY)
    _sync()
    g.check()
    _check_forward(lay, X)
    _check_backward(lay, X, dY)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("split,T,din,dout,t", [
    ("column", 3, 416, 800, 1), ("row", 40, 800, 416, 1), ("column", 130, 544, 1088, 2),
    ("row", 700, 1568, 672, 1), ("column", 515, 672, 1056, 1)])
def test_linear_scales_of_every_group(split, T, din, dout, t, fmt):
    """Every token, feature and run of 8 of them at a magnitude of its own, so that a scale
    taken from a wrong row, group or block shows."""
    w = custom_linear(T, din, dout, t, split)
    g = _gen(78)

    def spread(x):
        def f(n):
            e = torch.randint(-5, 6, (n,), generator=g, device="cuda")
            return torch.ldexp(torch.ones(n, device="cuda"), e)
        r, c = x.shape
        both = torch.randint(-4, 5, (-(-r // 8), -(-c // 8)), generator=g, device="cuda")
        both = both.repeat_interleave(8, 0)[:r].repeat_interleave(8, 1)[:, :c]
        return (torch.ldexp(x.float(), both) * f(r)[:, None] * f(c)).to(torch.bfloat16)

    shape = (din, w.shard) if split == "column" else (w.shard, dout)
    W = [spread(_randn(g, *shape)) for _ in range(t)]
    lay, X, dY = _layer(w, 77, fmt, W=W)
    X, dY = [spread(x) for x in X], [spread(x) for x in dY]
    lay.forward(X, save=True)
    lay.backward(dY)
    _sync()
    _check_forward(lay, X)
    _check_backward(lay, X, dY)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T", [9, 300])
def test_linear_not_finite(T, fmt):
    """NaN where, and only where, a group that is not finite takes part."""
    w = custom_linear(T, 416, 544, 1, "column")
    lay, X, dY = _layer(w, 21, fmt)
    X[0][3, 200] = float("inf")
    dY[0][5, 7] = float("nan")
    lay.forward(X, save=True)
    lay.backward(dY)
    _sync()
    nan = torch.isnan(lay.Y[0])
    assert nan[3].all() and int(nan.sum()) == w.out_features
    nan = torch.isnan(lay.dX[0])
    assert nan[5].all() and int(nan.sum()) == w.in_features
    nan = torch.isnan(lay.dW[0])
    assert nan[200].all() and nan[:, 7].all()
    assert int(nan.sum()) == w.in_features + w.out_features - 1
    assert torch.isnan(lay.db[7]) and int(torch.isnan(lay.db).sum()) == 1


@pytest.mark.parametrize("split,T", [("column", 5), ("row", 130), ("row", 600)])
def test_linear_calibrated_scale(split, T):
    """A calibrated scale is the one that is used, also where it cuts values off."""
    w = custom_linear(T, 512, 768, 2, split)
    for k in (-12, -9, 3):
        lay, X, dY = _layer(w, 5, "nvfp4", x_scale=torch.full((1,), 2.0 ** k, device="cuda"))
        lay.forward(X, save=True)
        lay.backward(dY)
        _sync()
        assert float(lay.x_scale) == 2.0 ** k
        _check_forward(lay, X)
        _check_backward(lay, X, dY)


def test_forward_between_keeps_what_was_saved():
    """A forward call that saves nothing, between one that does and its backward call."""
    w = custom_linear(70, 256, 512, 1, "column")
    lay, X, dY = _layer(w, 6, "nvfp4")
    other = [x * 64 for x in X]
    lay.forward(X, save=True)
    lay.forward(other)
    _sync()
    _check_forward(lay, other)
    lay.backward(dY)
    _sync()
    _check_backward(lay, X, dY)


@pytest.mark.parametrize("fmt,calibrated", [("mxfp4", False), ("nvfp4", False), ("nvfp4", True)])
@pytest.mark.parametrize("split,T,din,dout,t", [
    ("column", 1, 4096, 1056, 1), ("column", 7, 288, 416, 1), ("row", 1, 256, 256, 2), ("row", 16, 1088, 416, 2),
    ("row", 9, 4096, 1024, 8), ("column", 16, 32, 32, 1), ("column", 13, 9248, 2048, 2),
    ("row", 17, 1024, 416, 2), ("row", 40, 1088, 416, 2), ("column", 64, 288, 800, 1),
    ("column", 33, 4096, 1056, 1), ("row", 48, 4096, 1024, 8), ("row", 65, 4096, 1024, 8)])
def test_forward_alone(split, T, din, dout, t, fmt, calibrated):
    """Without keeping X, where few tokens are quantised on the way; the same result as with."""
    w = custom_linear(T, din, dout, t, split)
    lay, X, dY = _layer(w, T + din, fmt, x_scale=torch.full((1,), 2.0 ** -9, device="cuda") if calibrated else None)
    X[0][0, 3] = 40.0
    g = GuardBands()
    g.guard(lay, ["Y", "ws"])
    lay.forward(X)
    _sync()
    g.check()
    _check_forward(lay, X)
    alone = [y.clone() for y in lay.Y]
    lay.forward(X, save=True)
    _sync()
    assert all(torch.equal(a, b) for a, b in zip(alone, lay.Y))


@pytest.mark.parametrize("fmt", FORMATS)
def test_forward_alone_not_finite(fmt):
    w = custom_linear(5, 1024, 288, 2, "row")
    lay, X, _ = _layer(w, 3, fmt)
    X[1][3, 77] = float("nan")
    lay.forward(X)
    _sync()
    nan = torch.isnan(lay.Y[0])
    assert nan[3].all() and int(nan.sum()) == 288


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("split,T,din,dout,t", [("row", 300, 2048, 416, 4), ("column", 300, 416, 2048, 8),
                                                ("row", 1100, 1024, 2048, 2), ("column", 60, 288, 1024, 4)])
def test_segments_of_whole_stages(split, T, din, dout, t, fmt):
    """Shards that are multiples of 256, whose 4-bit segments lie in one matrix."""
    w = custom_linear(T, din, dout, t, split)
    lay, X, dY = _layer(w, T + din, fmt)
    lay.forward(X, save=True)
    lay.backward(dY)
    _sync()
    _check_forward(lay, X)
    _check_backward(lay, X, dY)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,C", [(1024, 1024), (1025, 1024), (511, 2080), (130, 8224), (1, 32), (300, 288)])
def test_quantize_rows_alone(T, C, fmt):
    """By rows alone, on both sides of the number of values that takes another kernel; what
    fills up is written."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    x = _values(T, C, _gen(T + C))
    got = fp4.quantize_tokens(x, fmt).rows
    both = fp4.quantize_tokens(x, fmt, cols=True).rows
    _sync()
    _check(got, x, fmt, 1, None if fmt == "mxfp4" else plain.tensor_scale([x]))
    assert torch.equal(got.q, both.q) and torch.equal(got.s, both.s)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("split,T,din,dout,t", [
    # tiles of 256 tokens: K long, features few, up to 256 tokens and more
    ("column", 333, 4128, 1056, 1), ("row", 300, 8192, 512, 2), ("column", 250, 8224, 4096, 1),
    # pairs of CTAs for 65 to 128 tokens: one tile each
    ("column", 66, 544, 12288, 1), ("column", 127, 288, 10400, 1), ("row", 100, 768, 12064, 3)])
def test_linear_by_other_tiles(split, T, din, dout, t, fmt):
    w = custom_linear(T, din, dout, t, split)
    lay, X, dY = _layer(w, T + din + dout, fmt)
    g = GuardBands()
    g.guard(lay, ["Y", "dX", "ws"])
    lay.forward(X, save=True)
    lay.backward(dY)
    _sync()
    g.check()
    _check_forward(lay, X)
    _check_backward(lay, X, dY)


@pytest.mark.parametrize("T", [40, 300, 1100])
def test_bias_gradient_not_finite(T):
    """Sums of infinities are what adding them gives."""
    w = custom_linear(T, 288, 416, 1, "column")
    lay, X, dY = _layer(w, 22, "mxfp4")
    inf = float("inf")
    dY[0][1, 3], dY[0][T - 1, 4], dY[0][2, 5], dY[0][T - 2, 5], dY[0][0, 6] = inf, -inf, inf, -inf, float("nan")
    lay.forward(X, save=True)
    lay.backward(dY)
    _sync()
    assert lay.db[3] == inf and lay.db[4] == -inf
    assert torch.isnan(lay.db[5]) and torch.isnan(lay.db[6])
    assert int(torch.isfinite(lay.db).sum()) == 416 - 4


@pytest.mark.parametrize("T,C,n", [(1, 32, 1), (1, 4096, 8), (3, 288, 5), (16, 16384, 1), (16, 2048, 8),
                                   (16, 2080, 8), (17, 16384, 1), (129, 2080, 3), (0, 96, 2)])
def test_tensor_scale_of_parts(T, C, n):
    """The largest anywhere, also the last of the last part, counts; what is not finite does not."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    g = _gen(T + C + n)
    parts = [_randn(g, T, C) for _ in range(n)]
    if T:
        parts[0][0, 3], parts[n // 2][T - 1, 5] = float("inf"), float("nan")
    for i in (0, n // 2, n - 1):
        for r, c in ((0, 0), (T - 1, C - 1), (T // 2, C // 3)) if T else ():
            kept = parts[i][r, c].clone()
            parts[i][r, c] = -1000.0
            got = fp4.tensor_scale(parts)
            _sync()
            assert float(got) == 2.0 ** -1   # the smallest power of two >= 1000 / 2688
            parts[i][r, c] = kept
    got = fp4.tensor_scale(parts)
    _sync()
    assert float(got) == (float(plain.tensor_scale(parts)) if T else 2.0 ** -110)

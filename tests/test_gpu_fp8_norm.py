"""The norms, the quantisation and the 8-bit linear layers together, as a step uses
them: in a row, captured and replayed, on other streams and threads, with buffers and
workspaces that are shared or exchanged, and at offsets beyond 32 bits."""
import threading

import pytest
import torch

import test_gpu_fp8 as f8
import test_gpu_norm as nm
from tensor_transformer_mlp_gemm_gb300.inputs import WORKLOADS, custom_linear, make_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


_sync = f8._sync


def _bits(x):
    return x.contiguous().view(torch.uint8)


def _equal(xs, ys):
    return all(torch.equal(_bits(x), _bits(y)) for x, y in zip(xs, ys, strict=True))


class Step:
    """A part of a residual stream: the norm before, a column- and a row-parallel layer
    in 8 bits, the norm after with its gate, and the next norm before."""

    def __init__(self, T, h, f, t, chunks=1, gate_rows=0, post="rms", pre="rms", alpha=1.0, seed=0,
                 device="cuda:0"):
        self.d = nm._inputs(T, h, gate_rows, seed)
        c = lambda x: [v.clone() for v in x.chunk(chunks)] if chunks > 1 else [x.clone()]  # noqa: E731
        self.X, self.dOut, self.dXn = c(self.d["X"]), c(self.d["dOut"]), c(self.d["dXn"])
        self.before = nm._layer(self.d, T, h, "none", pre, 0, 1.0, seq_chunks=chunks)
        self.after = nm._layer(self.d, T, h, post, pre, gate_rows, alpha, seq_chunks=chunks)
        self.up = f8._layer(custom_linear(T, h, f, t, "column", seq_chunks=chunks), seed + 1, dy="e5m2")[0]
        self.down = f8._layer(custom_linear(T, f, h, t, "row", seq_chunks=chunks), seed + 2, dy="e5m2")[0]

    @staticmethod
    def _of(x):
        return x if isinstance(x, list) else [x]

    def forward(self, stream=None):
        self.before.forward(self.X, stream=stream)
        self.x = self.up.quantize(self._of(self.before.Xn), cols=True, stream=stream)
        self.up.forward(self.x, stream=stream)
        self.y = self.down.quantize(self.up.Y, cols=True, stream=stream)
        self.down.forward(self.y, stream=stream)
        self.after.forward(self.X, self.down.Y, self.d["gate"], stream=stream)

    def backward(self, stream=None):
        out = self._of(self.after.Out)
        self.after.backward(self.dOut, self.dXn, self.down.Y, out, gate=self.d["gate"], stream=stream)
        self.down.backward(self._of(self.after.dZ), self.y, stream=stream)
        self.up.backward(self.down.dX, self.x, stream=stream)
        self.before.backward(self._of(self.after.dX), self.up.dX, None, self.X, stream=stream)

    def step(self, stream=None):
        self.forward(stream)
        self.backward(stream)

    def outputs(self):
        a, b = self.after, self.before
        one = [a.dpost_gamma, a.dpost_beta, a.dpre_gamma, a.dpre_beta, a.dgate, b.dpre_gamma, b.dpre_beta,
               self.up.db, self.down.db]
        return [x for x in one if x is not None] + [
            x for xs in (a.Out, a.Xn, a.dX, a.dZ, b.dX, self.up.Y, self.down.Y, self.up.dX, self.down.dX,
                         self.up.dW, self.down.dW) for x in self._of(xs)]


SMALL = dict(T=96, h=512, f=1024, t=2, gate_rows=32)
LARGE = dict(T=640, h=1040, f=2048, t=4, gate_rows=128, post="layer", pre="layer", alpha=0.7)


@pytest.mark.parametrize("kw", [
    dict(T=1, h=4096, f=4096, t=1, gate_rows=1),
    dict(T=7, h=400, f=1296, t=3, post="none", pre="layer"),
    SMALL, LARGE,
    dict(T=1024, h=512, f=1024, t=8, chunks=8, gate_rows=1024, alpha=0.83)])
def test_step(kw):
    """Each part against its plain form, on what the part before it left."""
    s = Step(**kw)
    s.step()
    _sync()
    cat = lambda xs: torch.cat(Step._of(xs))  # noqa: E731
    d, a, b = s.d, s.after, s.before
    nm._check_forward(d, b, None, cat(b.Xn), b.stats, z=False)
    f8._check_forward(s.up, s.x)
    f8._check_forward(s.down, s.y)
    d = dict(d, Z=cat(s.down.Y))
    nm._check_forward(d, a, cat(a.Out), cat(a.Xn), a.stats)
    nm._check_backward(d, a, cat(a.Out), a.stats, d["dOut"], d["dXn"])
    f8._check_backward(s.down, s.y, Step._of(a.dZ), "e5m2")
    f8._check_backward(s.up, s.x, s.down.dX, "e5m2")
    nm._check_backward(dict(d, X=cat(s.X)), b, cat(s.X), b.stats, cat(a.dX), cat(s.up.dX), z=False)


@pytest.mark.parametrize("T", [1, 48, 300])
def test_norm_rows_feed_the_linear(T):
    """8-bit rows written by the norm give what its bf16 rows give, quantised."""
    d = nm._inputs(T, 528, 0, T)
    kw = dict(post="rms", pre="rms", gate_rows=0, alpha=1.0)
    plain, eight = nm._layer(d, T, 528, **kw), nm._layer(d, T, 528, **kw, quantize="e4m3")
    lay = f8._layer(custom_linear(T, 528, 1040, 1, "column"), 3)[0]
    plain.forward(d["X"], d["Z"])
    lay.forward(lay.quantize(plain.Xn))
    _sync()
    want = [x.clone() for x in lay.Y]
    eight.forward(d["X"], d["Z"])
    lay.forward(eight.tokens_by_rows)
    _sync()
    assert _equal(lay.Y, want)


def test_around_a_block():
    """The norms around the bf16 block: what it computes is what it computes alone."""
    from tensor_transformer_mlp_gemm_gb300.block import DeviceBlock
    w = WORKLOADS["small_gpt"]
    blk = DeviceBlock(w, make_inputs(w, 1))
    T, h, n = w.tokens, w.hidden, w.seq_chunks
    d = nm._inputs(T, h, T, 4)
    before = nm._layer(d, T, h, "none", "layer", 0, 1.0, seq_chunks=n)
    after = nm._layer(d, T, h, "layer", "rms", T, 0.9, seq_chunks=n)
    X = [x.clone() for x in d["X"].chunk(n)]
    before.forward(X)
    blk.X = Step._of(before.Xn)
    blk.forward()
    after.forward(X, blk.Z, d["gate"])
    dOut, dXn = ([x.clone() for x in d[k].chunk(n)] for k in ("dOut", "dXn"))
    after.backward(dOut, dXn, blk.Z, after.Out, gate=d["gate"])
    blk.dZ = Step._of(after.dZ)
    blk.backward()
    before.backward(after.dX, blk.dX, None, X)
    _sync()
    d = dict(d, Z=torch.cat(blk.Z))
    cat = lambda xs: torch.cat(Step._of(xs))  # noqa: E731
    nm._check_forward(d, after, cat(after.Out), cat(after.Xn), after.stats)
    nm._check_backward(d, after, cat(after.Out), after.stats, d["dOut"], d["dXn"])
    nm._check_backward(d, before, d["X"], before.stats, cat(after.dX), cat(blk.dX), z=False)
    alone = DeviceBlock(w, make_inputs(w, 1))
    alone.X, alone.dZ = [x.clone() for x in blk.X], [x.clone() for x in blk.dZ]
    alone.step()
    _sync()
    assert _equal(alone.Z + alone.dX, blk.Z + blk.dX)


@pytest.mark.parametrize("kw", [SMALL, LARGE])
def test_same_bits_every_run(kw):
    s = Step(**kw)
    s.step()
    _sync()
    want = [x.clone() for x in s.outputs()]
    for _ in range(3):
        for x in s.outputs():
            x.fill_(7.0)
        s.step()
        _sync()
        assert _equal(s.outputs(), want)


@pytest.mark.parametrize("kw", [SMALL, LARGE])
def test_capture_and_replay(kw):
    s = Step(**kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    # the inputs of another seed, in place
    for seed in (5, 6):
        d = nm._inputs(kw["T"], kw["h"], kw["gate_rows"], seed)
        for dst, src in ((s.X, "X"), (s.dOut, "dOut"), (s.dXn, "dXn")):
            dst[0].copy_(d[src])
        graph.replay()
        _sync()
        got = [x.clone() for x in s.outputs()]
        s.step()
        _sync()
        assert _equal(s.outputs(), got)
        s.x = s.y = None


def test_two_graphs_with_one_workspace_in_turn():
    """Two layers with one workspace, each step captured by itself, replayed one after
    the other."""
    from tensor_transformer_mlp_gemm_gb300 import fp8
    layers, graphs, wants = [], [], []
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    for seed, (T, din, dout) in enumerate(((300, 528, 1040), (64, 1040, 272))):
        lay, X, dY = f8._layer(custom_linear(T, din, dout, 1, "column"), seed)
        lay = fp8.DeviceFp8Linear(lay.w, lay.Wq, lay.Ws, lay.b, workspace=ws)
        x = lay.quantize(X, cols=True)
        lay.forward(x)
        lay.backward(dY, x)
        _sync()
        wants.append([t.clone() for t in lay.Y + lay.dX + lay.dW + [lay.db]])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lay.forward(x)
            lay.backward(dY, x)
        layers.append((lay, x, dY))
        graphs.append(graph)
    for lay, _, _ in layers:
        for t in lay.Y + lay.dX + lay.dW + [lay.db]:
            t.zero_()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    _sync()
    for (lay, _, _), want in zip(layers, wants):
        assert _equal(lay.Y + lay.dX + lay.dW + [lay.db], want)


@pytest.mark.parametrize("raw", [False, True])
def test_another_stream(raw):
    """Everything on a stream that is not the current one, behind work that it waits for."""
    s = Step(**SMALL)
    s.step()
    _sync()
    want = [x.clone() for x in s.outputs()]
    for x in s.outputs():
        x.zero_()
    kept = s.X[0].clone()
    s.X[0].zero_()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        torch.cuda._sleep(2_000_000)
        s.X[0].copy_(kept)
    s.step(other.cuda_stream if raw else other)
    other.synchronize()
    _sync()
    assert _equal(s.outputs(), want)


def test_first_gradients_on_another_stream():
    """Buffers that a call makes itself belong to the stream that it was given."""
    other = torch.cuda.Stream()
    s, ref = Step(**SMALL), Step(**SMALL)
    ref.step()
    torch.cuda.synchronize()
    # blocks of the sizes the step will ask for, freed on the current stream while it is busy
    torch.cuda._sleep(20_000_000)
    sizes = [x.numel() * x.element_size() for x in ref.outputs()]
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes for _ in range(3)]
    del junk
    s.step(other)
    torch.cuda.synchronize()
    _sync()
    assert _equal(s.outputs(), ref.outputs())


def test_threads():
    """Two threads, each with a step and a stream of its own."""
    steps = [Step(**SMALL), Step(**dict(LARGE, seed=9))]
    wants = []
    for s in steps:
        s.step()
        _sync()
        wants.append([x.clone() for x in s.outputs()])
        for x in s.outputs():
            x.zero_()
    torch.cuda.synchronize()
    errors = []

    def run(s):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for _ in range(20):
                    s.step()
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(s,)) for s in steps]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    _sync()
    assert not errors
    for s, want in zip(steps, wants):
        assert _equal(s.outputs(), want)


@pytest.mark.parametrize("split,T,din,dout,t,chunks", [
    ("row", 2048, 512, 2064, 2, 4),       # pairs of CTAs writing token chunks
    ("column", 2048, 1296, 512, 2, 8),
    ("row", 1280, 2064, 2576, 3, 1),
    ("column", 257, 272, 1552, 1, 1),     # one row into a second tile
    ("column", 130, 400, 528, 1, 1),      # tiles of 256 tokens
    ("row", 256, 6160, 144, 5, 2),
    ("column", 100, 272, 9984, 1, 1)])    # two CTAs on an SM with 128 tokens each
def test_linear_more_shapes(split, T, din, dout, t, chunks):
    lay, X, dY = f8._layer(custom_linear(T, din, dout, t, split, seq_chunks=chunks), T + din)
    x = lay.quantize(X, cols=True)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()
    f8._check_forward(lay, x)
    f8._check_backward(lay, x, dY, "e4m3")


@pytest.mark.parametrize("T,h,gate_rows,post,pre", [
    (90, 6152, 30, "layer", "layer"),     # clusters of two: 512 threads a CTA, then 384
    (61, 6144, 61, "rms", "layer"),
    (40, 9224, 8, "layer", "rms"),        # clusters of four
    (31, 3208, 31, "layer", "layer"),
    (50, 4096, 0, "none", "layer"),
    (9, 1032, 3, "rms", "layer")])
def test_norm_more_widths(T, h, gate_rows, post, pre):
    nm.test_norm(T, h, gate_rows, post, pre)


@pytest.mark.parametrize("split", ["column", "row"])
def test_linear_empty(split):
    lay, X, dY = f8._layer(custom_linear(0, 256, 512, 2, split), 1)
    x = lay.quantize(X, cols=True)
    for t in lay.dW + [lay.db]:
        t.fill_(3.0)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()
    assert all(torch.count_nonzero(t) == 0 for t in lay.dW + [lay.db])


def test_buffers_are_exchanged():
    lay, X, dY = f8._layer(custom_linear(64, 256, 512, 2, "column"), 2)
    x = lay.quantize(X, cols=True)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()
    want = [t.clone() for t in lay.Y + lay.dX]
    lay.Y = [torch.zeros_like(t) for t in lay.Y]
    lay.dX = [torch.zeros_like(t) for t in lay.dX]
    lay.Y[0] = None                       # (a list of its own: the layer keeps its buffers)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()
    assert _equal(lay.Y + lay.dX, want)
    with pytest.raises(ValueError, match="2 tensors"):
        lay.Y = lay.Y[:1]
    with pytest.raises(ValueError):
        lay.dX = [t.float() for t in lay.dX]
    # outputs of one call
    Y = [torch.zeros_like(t) for t in lay.Y]
    lay.forward(x, Y=Y)
    # and quantised tensors that a caller brings itself
    from tensor_transformer_mlp_gemm_gb300.fp8 import Fp8Tokens
    own = Fp8Tokens(x.rows.clone(), x.row_scale.clone(), x.cols.clone(), x.col_scale.clone())
    lay.Y = [torch.zeros_like(t) for t in lay.Y]
    lay.forward(own)
    _sync()
    assert _equal(Y + lay.Y, want[:2] * 2)


@pytest.mark.parametrize("split,T,din,dout,t", [("column", 219, 592, 2432, 8), ("row", 32, 2208, 1040, 2),
                                                ("column", 4, 832, 4608, 8), ("row", 1300, 2432, 2320, 8)])
def test_scales_inside_larger_arrays(split, T, din, dout, t):
    """Scales of all shards in one array: a shard's start on 4 bytes."""
    from tensor_transformer_mlp_gemm_gb300 import fp8
    lay, X, dY = f8._layer(custom_linear(T, din, dout, t, split), T)
    x = lay.quantize(X, cols=True)
    lay.forward(x)
    lay.backward(dY, x)
    _sync()

    def together(xs):
        flat = torch.cat([torch.zeros(1, device="cuda")] + [v.reshape(-1) for v in xs])[1:]
        return [v.view(xs[0].shape) for v in flat.split(xs[0].numel())]
    own = fp8.DeviceFp8Linear(lay.w, lay.Wq, together(lay.Ws), lay.b)
    xs = [x] if split == "column" else list(x)
    parts = [fp8.Fp8Tokens(v.rows, r, v.cols, c) for v, r, c in
             zip(xs, together([v.row_scale for v in xs]), together([v.col_scale for v in xs]))]
    assert any(s.data_ptr() % 16 for s in own.Ws) and all(p.row_scale.data_ptr() % 16 for p in parts[:1])
    own.forward(parts)
    own.backward(dY, parts)
    _sync()
    assert _equal(own.Y + own.dX + own.dW + [own.db], lay.Y + lay.dX + lay.dW + [lay.db])
    # and as outputs
    out = fp8.Fp8Tokens(torch.empty_like(xs[0].rows), together([torch.empty_like(xs[0].row_scale)])[0],
                        torch.empty_like(xs[0].cols), together([torch.empty_like(xs[0].col_scale)])[0])
    src = X if split == "column" else X[0]
    fp8.quantize_tokens(src, cols=True, out=out)
    _sync()
    assert _equal([out.rows, out.row_scale, out.cols, out.col_scale],
                  [xs[0].rows, xs[0].row_scale, xs[0].cols, xs[0].col_scale])


def test_quantize_into_buffers():
    from tensor_transformer_mlp_gemm_gb300 import fp8
    g = f8._gen(1)
    a, b = f8._randn(g, 130, 272), f8._randn(g, 130, 272)
    x = fp8.quantize_tokens(a, cols=True)
    y = fp8.quantize_tokens(b, cols=True)
    z = fp8.quantize_tokens(b, cols=True, out=x)
    _sync()
    assert z is x and _equal([x.rows, x.row_scale, x.cols, x.col_scale],
                             [y.rows, y.row_scale, y.cols, y.col_scale])
    rows = fp8.quantize_tokens(a)
    for bad in (lambda: fp8.quantize_tokens(b, cols=True, out=rows),
                lambda: fp8.quantize_tokens(b, "e5m2", out=x),
                lambda: fp8.quantize_tokens(b[:128].contiguous(), out=x)):
        with pytest.raises(ValueError):
            bad()


def test_python_refusals():
    from tensor_transformer_mlp_gemm_gb300 import binding, fp8
    from tensor_transformer_mlp_gemm_gb300.norm import DeviceNormResidual
    g = f8._gen(2)
    lay, X, dY = f8._layer(custom_linear(64, 256, 512, 2, "column"), 2)
    x = lay.quantize(X)
    e5 = fp8.quantize_tokens(X[0], "e5m2", cols=True)
    shards = fp8.quantize_shards([X[0], X[0]])
    strided = f8._randn(g, 64, 512)[:, ::2]
    n = nm._layer(nm._inputs(64, 256, 8, 1), 64, 256, "rms", "rms", 8, 1.0)
    d = nm._inputs(64, 256, 8, 1)
    none = nm._layer(d, 64, 256, "rms", "none", 0, 1.0)
    bad = [
        lambda: lay.backward(dY, x),                                # no groups along the tokens
        lambda: lay.forward(e5),                                    # another format
        lambda: lay.forward(shards),                                # two inputs
        lambda: lay.forward(lay.quantize([X[0][:32].contiguous()])),
        lambda: lay.forward(x, Y=lay.Y[:1]),
        lambda: lay.backward(dY[:1], lay.quantize(X, cols=True)),
        lambda: lay.backward([t.float() for t in dY], lay.quantize(X, cols=True)),
        lambda: lay.quantize([strided]),
        lambda: fp8.quantize_tokens(X[0], rows=False),
        lambda: fp8.quantize_tokens([X[0][:63].contiguous()] * 2),  # chunks of 63 tokens
        lambda: fp8.quantize_tokens([X[0], X[0].cpu()]),
        lambda: fp8.quantize_tokens([X[0], X[0].float()]),
        lambda: fp8.quantize_weight(X[0].T),
        lambda: fp8.DeviceFp8Linear(lay.w, lay.Wq[:1], lay.Ws[:1], lay.b),
        lambda: fp8.DeviceFp8Linear(lay.w, lay.Wq, [s[:1].contiguous() for s in lay.Ws], lay.b),
        lambda: fp8.DeviceFp8Linear(lay.w, lay.Wq, lay.Ws, lay.b, w_format="e5m2"),
        lambda: fp8.DeviceFp8Linear(lay.w, lay.Wq, lay.Ws, lay.b, workspace=lay.ws[:16]),
        lambda: fp8.DeviceFp8Linear(lay.w, lay.Wq, lay.Ws, lay.b, workspace=lay.ws.cpu()),
        lambda: n.forward(d["X"], d["Z"]),                          # its gate is missing
        lambda: n.forward(d["X"], gate=d["gate"]),                  # a gate without Z
        lambda: n.forward(d["X"], d["Z"], d["gate"][:4].contiguous()),
        lambda: n.forward(d["X"][:32].contiguous(), d["Z"], d["gate"]),
        lambda: n.forward([d["X"]] * 2, d["Z"], d["gate"]),
        lambda: n.forward(d["X"].float(), d["Z"], d["gate"]),
        lambda: n.backward(d["dOut"], None, d["Z"], n.Out, gate=d["gate"]),
        lambda: n.backward(d["dOut"], d["dXn"], d["Z"], n.Out, n.stats[:2], gate=d["gate"]),
        lambda: none.backward(d["dOut"], d["dXn"], d["Z"], none.Out),
        lambda: DeviceNormResidual(64, 256, pre_gamma=d["pre_gamma"]),
        lambda: DeviceNormResidual(64, 256, post_gamma=d["post_gamma"][:128], pre_gamma=d["pre_gamma"]),
        lambda: DeviceNormResidual(64, 256, post_gamma=d["post_gamma"], pre_gamma=d["pre_gamma"].cpu()),
    ]
    for k, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was taken")
    # what only the library can see: a pointer that is not on 16 bytes
    odd = torch.empty(64 * 256 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 64 * 256].view(64, 256)
    with pytest.raises(Exception, match="(?i)unsupported|align"):
        fp8.quantize_tokens(odd)
    assert binding.tpmlp_sync_check() == binding.TPMLP_OK


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows are what they are alone."""
    from tensor_transformer_mlp_gemm_gb300 import fp8
    T, h, last = 135168, 16384, 384       # 2.2e9 elements
    g = f8._gen(3)
    row = f8._randn(g, 4096, h)
    X = row.repeat(T // 4096, 1)
    X[-last:] = f8._randn(g, last, h)
    tail = X[-last:].clone()
    x, y = fp8.quantize_tokens(X, cols=True), fp8.quantize_tokens(tail, cols=True)
    _sync()
    assert _equal([x.rows[-last:], x.row_scale[:, -last:], x.cols[-last:], x.col_scale[-3:]],
                  [y.rows, y.row_scale, y.cols, y.col_scale])
    del x, y
    d = nm._inputs(last, h, 0, 1)
    big, small = (nm._layer(d, n, h, "rms", "rms", 0, 1.0) for n in (T, last))
    big.forward(X, X)
    small.forward(tail, tail)
    big.backward(X, X, X, big.Out)
    small.backward(tail, tail, tail, small.Out)
    _sync()
    assert _equal([t[-last:] for t in (big.Out, big.Xn, big.dX, big.dZ)],
                  [small.Out, small.Xn, small.dX, small.dZ])
    del big, small, X, tail
    # outputs and gradients of a linear layer
    T = 528384
    w = custom_linear(T, 256, 4112, 1, "column")
    lay, X, _ = f8._layer(w, 4)
    one = fp8.DeviceFp8Linear(custom_linear(last, 256, 4112, 1, "column"), lay.Wq, lay.Ws, lay.b)
    lay.forward(lay.quantize(X))
    one.forward(one.quantize([X[0][-last:].clone()]))
    _sync()
    assert _equal([lay.Y[0][-last:]], one.Y)
    x = lay.quantize(X, cols=True)
    lay.backward(lay.Y, x)
    _sync()
    # (384 rows alone take the few-rows kernel, which adds in another order)
    plain = f8.plain
    q, sc = plain.quantize(lay.Y[0][-last:], "e4m3", 1)
    a, v = plain.rows_value(q, sc.T), plain.block_value(lay.Wq[0], lay.Ws[0]).T
    ref, bound = a @ v, plain.product_bound(a, v, -(-4112 // 128))
    plain.check("dX", lay.dX[0][-last:], ref, bound + plain.BF16 * (ref.abs() + bound))

"""A 4-bit layer's training step and the clipping of its gradients as one run: captured, on
other streams, in threads, with shared workspaces, with no tokens, past 32-bit offsets; and
what the Python layer refuses."""
import math
import threading

import pytest
import torch

import plain_fp4 as plain
import test_gpu_fp4 as f4
import test_gpu_grad as tg
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu
SMALL = dict(split="column", T=40, din=288, dout=416, t=1, fmt="nvfp4")
LARGE = dict(split="row", T=1100, din=2048, dout=1056, t=4, fmt="mxfp4")
NVROW = dict(split="row", T=300, din=1024, dout=2080, t=2, fmt="nvfp4")


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


class Step:
    """Forward, backward, clipping in place."""

    def __init__(self, split, T, din, dout, t, fmt, seed=1, workspace=None):
        from tensor_transformer_mlp_gemm_gb300 import fp4
        from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
        self.lay, self.X, self.dY = f4._layer(custom_linear(T, din, dout, t, split), seed, fmt)
        if workspace is not None:
            self.lay = fp4.DeviceFp4Linear(self.lay.w, self.lay.weights, self.lay.b, workspace=workspace)
        self.clip = DeviceGradients(self.lay.dW + [self.lay.db])
        self.max_norm = 0.05

    def step(self, stream=None):
        self.lay.forward(self.X, save=True, stream=stream)
        self.lay.backward(self.dY, stream=stream)
        self.clip.clip(self.max_norm, stream=stream)

    def outputs(self):
        return self.lay.Y + self.lay.dX + self.lay.dW + [self.lay.db, self.clip.norm]


@pytest.mark.parametrize("kw", [SMALL, LARGE, NVROW])
def test_step(kw):
    s = Step(**kw)
    s.lay.forward(s.X, save=True)
    s.lay.backward(s.dY)
    f4._sync()
    f4._check_forward(s.lay, s.X)
    f4._check_backward(s.lay, s.X, s.dY)
    before = [x.clone() for x in s.clip.grads]
    s.step()
    f4._sync()
    want = tg._check_norm(s.clip.norm, before)
    assert want > s.max_norm
    tg._check_out(s.clip.grads, before, want, s.max_norm)


@pytest.mark.parametrize("kw", [SMALL, LARGE, NVROW])
def test_same_bits_every_run(kw):
    s = Step(**kw)
    s.step()
    f4._sync()
    want = [x.clone() for x in s.outputs()]
    for _ in range(3):
        for x in s.outputs():
            x.fill_(7.0)
        s.step()
        f4._sync()
        assert _equal(s.outputs(), want)


@pytest.mark.parametrize("kw", [SMALL, LARGE, NVROW])
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
    for seed in (5, 6):
        for x in s.X + s.dY:
            x.copy_(f4._randn(f4._gen(seed), *x.shape, std=0.3 * seed))
        for x in s.outputs():
            x.zero_()
        graph.replay()
        f4._sync()
        got = [x.clone() for x in s.outputs()]
        s.step()
        f4._sync()
        assert _equal(s.outputs(), got)


def test_weights_updated_in_place():
    """Weights quantised again into the same buffers right before the next call, again and again,
    with few tokens and with many: each call reads the new ones."""
    from tensor_transformer_mlp_gemm_gb300 import binding
    from tensor_transformer_mlp_gemm_gb300.fp8 import _pointers
    for T in (1, 40, 100, 600):
        w = custom_linear(T, 1024, 2048, 1, "column")
        lay, X, _ = f4._layer(w, T, "mxfp4", backward=False)
        Ws = [f4._randn(f4._gen(i), 1024, 2048, std=0.1 * (i + 1)) for i in range(4)]
        m = lay.weights.forward[0]
        outs = [torch.empty_like(lay.Y[0]) for _ in range(12)]
        quant = binding.make_fp4_quant(1024, 2048, 1, False, 0)
        for i, out in enumerate(outs):
            binding.tpmlp_fp4_quantize(quant, _pointers([Ws[i % 4]]), None, None, None, _pointers([m.q]),
                                       _pointers([m.s]))
            lay.forward(X, Y=[out])
        f4._sync()
        for i, out in enumerate(outs):
            binding.tpmlp_fp4_quantize(quant, _pointers([Ws[i % 4]]), None, None, None, _pointers([m.q]),
                                       _pointers([m.s]))
            f4._sync()
            if i < 4:
                f4._check_forward(lay, X, [out])
            else:
                assert torch.equal(out, outs[i % 4])


def test_two_graphs_with_one_workspace_in_turn():
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    steps = [Step(**dict(SMALL, seed=3), workspace=ws), Step(**dict(LARGE, seed=4), workspace=ws)]
    graphs, wants = [], []
    for s in steps:
        s.step()
        f4._sync()
        wants.append([x.clone() for x in s.outputs()])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
        graphs.append(graph)
    for s in steps:
        for x in s.outputs():
            x.zero_()
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    f4._sync()
    for s, want in zip(steps, wants):
        assert _equal(s.outputs(), want)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("kw", [SMALL, NVROW])
def test_another_stream(kw, raw):
    """Everything on a stream that is not the current one, behind work that it waits for."""
    s = Step(**kw)
    s.step()
    f4._sync()
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
    f4._sync()
    assert _equal(s.outputs(), want)


def test_first_buffers_on_another_stream():
    """Buffers that a call makes itself belong to the stream that it was given."""
    other = torch.cuda.Stream()
    s, ref = Step(**NVROW), Step(**NVROW)
    ref.step()
    torch.cuda.synchronize()
    want = ref.lay.Y + ref.lay.dX
    s.lay._dX = s.lay._saved = None
    torch.cuda._sleep(20_000_000)
    sizes = [x.numel() * x.element_size() for x in want] + [ref.lay._saved.buf.numel()]
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255) for n in sizes + [1 << 20] for _ in range(3)]
    del junk
    s.step(other)
    torch.cuda.synchronize()
    f4._sync()
    assert _equal(s.outputs(), ref.outputs())


def test_threads():
    steps = [Step(**SMALL), Step(**dict(LARGE, seed=9)), Step(**dict(NVROW, seed=2))]
    wants = []
    for s in steps:
        s.step()
        f4._sync()
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
    f4._sync()
    assert not errors
    for s, want in zip(steps, wants):
        assert _equal(s.outputs(), want)


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("split", ["column", "row"])
def test_empty(split, fmt):
    """No tokens: nothing to do forward, zero gradients backward."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    s = Step(split, 0, 256, 512, 2, fmt)
    for x in s.lay.dW + [s.lay.db]:
        x.fill_(3.0)
    s.step()
    f4._sync()
    assert all(bool((x == 0).all()) for x in s.lay.dW + [s.lay.db]) and float(s.clip.norm) == 0
    x = fp4.quantize_tokens(torch.empty(0, 64, device="cuda", dtype=torch.bfloat16), fmt, cols=True)
    assert x.rows.values().shape == (0, 64) and x.cols.values().shape == (64, 0)
    f4._sync()


def test_buffers_are_exchanged():
    s = Step(**NVROW)
    s.step()
    f4._sync()
    want = [x.clone() for x in s.lay.Y + s.lay.dX]
    s.lay.Y = [torch.zeros_like(x) for x in s.lay.Y]
    s.lay.dX = [torch.zeros_like(x) for x in s.lay.dX]
    s.step()
    f4._sync()
    assert _equal(s.lay.Y + s.lay.dX, want)
    Y, dX = [torch.zeros_like(x) for x in s.lay.Y], [torch.zeros_like(x) for x in s.lay.dX]
    s.lay.forward(s.X, save=True, Y=Y)
    s.lay.backward(s.dY, dX=dX)
    f4._sync()
    assert _equal(Y + dX, want)


def test_matrices_inside_larger_arrays():
    """Values, scales and the tensor's scale as views of a caller's own storage; shards at
    unequal steps."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    w = custom_linear(200, 512, 768, 4, "row")
    lay, X, _ = f4._layer(w, 3, "nvfp4", backward=False)
    lay.forward(X)
    scale = torch.zeros(7, device="cuda")[3:4].copy_(lay.weights.scale)
    ms = []
    for i, m in enumerate(lay.weights.forward):
        q = torch.empty(m.q.numel() + 16 * (i * i + 1), dtype=torch.uint8, device="cuda")[16 * (i * i + 1):].view_as(m.q)
        s = torch.empty(m.s.numel() + 16 * (i + 1), dtype=torch.uint8, device="cuda")[16 * (i + 1):]
        ms.append(fp4.Fp4Matrix(q.copy_(m.q), s.copy_(m.s), scale, m.shape, m.fmt))
    other = fp4.DeviceFp4Linear(w, fp4.Fp4Weights(ms, None), lay.b)
    other.forward(X)
    f4._sync()
    assert _equal(other.Y, lay.Y)
    assert torch.equal(ms[1].values(out=torch.empty(ms[1].shape, dtype=torch.bfloat16, device="cuda")),
                       lay.weights.forward[1].values())


def test_python_refusals():
    from tensor_transformer_mlp_gemm_gb300 import binding, fp4
    x = torch.zeros(64, 256, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(1, device="cuda")
    mx, nv = fp4.quantize_weight(x, "mxfp4"), fp4.quantize_weight(x, "nvfp4", backward=True)
    w, b = custom_linear(8, 64, 256, 1, "column"), torch.zeros(256, dtype=torch.bfloat16, device="cuda")
    lay = fp4.DeviceFp4Linear(w, nv, b)
    only = fp4.DeviceFp4Linear(w, mx, b)
    X, dY = x[:8, :64].contiguous(), torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    F, L, M = fp4.Fp4Matrix, fp4.DeviceFp4Linear, nv.forward[0]
    ws = torch.empty(1, dtype=torch.uint8, device="cuda")
    for k, call in enumerate([
            lambda: fp4.quantize_tokens(x, "fp4"), lambda: fp4.quantize_tokens(x.float()),
            lambda: fp4.quantize_tokens(x.t()), lambda: fp4.quantize_tokens(x.cpu()),
            lambda: fp4.quantize_tokens(x, rows=False), lambda: fp4.quantize_tokens([x] * 2),
            lambda: fp4.quantize_tokens([x] * 9), lambda: fp4.quantize_tokens([]),
            lambda: fp4.quantize_tokens(x, "mxfp4", scale=one), lambda: fp4.quantize_tokens(x, "nvfp4", scale=one.cpu()),
            lambda: fp4.quantize_tokens(x, "nvfp4", scale=one.double()),
            lambda: fp4.quantize_weight([x, x[:32]]), lambda: fp4.tensor_scale(x.float()),
            lambda: F(M.q[:-1], M.s, M.scale, M.shape, "nvfp4"), lambda: F(M.q, M.s[:-16], M.scale, M.shape, "nvfp4"),
            lambda: F(M.q, M.s, None, M.shape, "nvfp4"), lambda: F(M.q, M.s, M.scale, M.shape, "mxfp4"),
            lambda: M.values(out=x), lambda: fp4.Fp4Weights([], None), lambda: fp4.Fp4Weights([M], [M, M]),
            lambda: fp4.Fp4Weights([M, mx.forward[0]], None),
            lambda: fp4.Fp4Weights([M, fp4.quantize_weight(x, "nvfp4").forward[0]], None),  # another scale
            lambda: L(w, nv, b.float()), lambda: L(w, nv, b[:128]), lambda: L(w, nv, b.cpu()),
            lambda: L(custom_linear(8, 64, 256, 2, "column"), nv, b),
            lambda: L(custom_linear(8, 256, 64, 1, "column"), nv, b[:64].contiguous()),
            lambda: L(custom_linear(8, 48, 256, 1, "column"), nv, b), lambda: L(w, nv, b, workspace=ws),
            lambda: L(w, mx, b, x_scale=one), lambda: L(w, nv, b, x_scale=torch.ones(2, device="cuda")),
            lambda: setattr(lay, "x_scale", 1.0 * torch.ones(1)), lambda: setattr(only, "x_scale", one),
            lambda: lay.forward(X.float()), lambda: lay.forward([X, X]), lambda: lay.forward(X[:4]),
            lambda: lay.forward(X, Y=X), lambda: lay.backward(dY),                # nothing saved
            lambda: only.forward(X, save=True), lambda: only.backward(dY)]):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {k} was taken")
    lay.forward(X, save=True)
    for call in (lambda: lay.backward(X), lambda: lay.backward(dY, dX=dY)):
        with pytest.raises(ValueError):
            call()
    # what only the library can see: a pointer that is not on 16 bytes
    odd = torch.empty(64 * 256 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 64 * 256].view(64, 256)
    with pytest.raises(binding.TpmlpError):
        fp4.quantize_tokens(odd)
    with pytest.raises(binding.TpmlpError):
        fp4.quantize_tokens(torch.empty(64, 48, dtype=torch.bfloat16, device="cuda"))
    assert binding.tpmlp_sync_check() == binding.TPMLP_OK


@pytest.mark.parametrize("fmt", f4.FORMATS)
def test_offsets_beyond_32_bits(fmt):
    """More than 2^32 elements and 2^31 bytes: the last rows are what they are alone."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    T, C, last = 266240, 16384, 384       # 4.4e9 elements, 2.2e9 bytes of values
    g = f4._gen(3)
    row = f4._randn(g, 4096, C)
    X = row.repeat(T // 4096, 1)
    X[-last:] = f4._randn(g, last, C)
    tail = X[-last:].clone()
    scale = torch.full((1,), 2.0 ** -9, device="cuda") if fmt == "nvfp4" else None
    x = fp4.quantize_tokens(X, fmt, cols=True, scale=scale)
    y = fp4.quantize_tokens(tail, fmt, cols=True, scale=scale)
    f4._sync()
    assert torch.equal(x.rows.q[-last:], y.rows.q) and torch.equal(x.cols.q[:, -last // 2:], y.cols.q)
    assert torch.equal(x.rows.s[-3 * (y.rows.s.numel() // 3):], y.rows.s)
    v = x.rows.values()
    assert torch.equal(v[-last:], y.rows.values())
    if fmt == "nvfp4":
        X[-1, -1] = 6.0 * 448 * 8
        assert float(fp4.tensor_scale(X)) == 8.0
    del v, x, X
    # outputs of a layer past 2^31 elements, and gradients over that many tokens
    T = 528384
    w = custom_linear(T, 256, 4128, 1, "column")
    lay, X, _ = f4._layer(w, 4, fmt, x_scale=scale)
    one = fp4.DeviceFp4Linear(custom_linear(last, 256, 4128, 1, "column"), lay.weights, lay.b, x_scale=scale)
    lay.forward(X, save=True)
    one.forward([X[0][-last:].clone()])
    f4._sync()
    assert torch.equal(lay.Y[0][-last:], one.Y[0])
    dY = f4._randn(f4._gen(5), 2048, 4128, std=1e-3).repeat(T // 2048, 1)
    lay.backward([dY])
    one.forward([X[0][-last:].clone()], save=True)
    one.backward([dY[-last:].clone()])
    f4._sync()
    # the last rows alone: another scale for dY only where its largest value is elsewhere
    gd = None if fmt == "mxfp4" else plain.tensor_scale([dY[:2048]])
    a, b = plain.values(dY[-last:], fmt, 1, gd), plain.value(lay.weights.backward[0]).T
    ref, bound = a @ b, plain.product_bound(a, b, -(-4128 // 256) * 4)
    plain.check("dX", lay.dX[0][-last:], ref, bound + plain.BF16 * (ref.abs() + bound))


def test_gradients_beyond_32_bits():
    """One tensor of more than 2^32 bytes, and its last values."""
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    n = (1 << 31) + 5
    x = torch.zeros(n, dtype=torch.float16, device="cuda")
    x[-3:] = 3.0
    x[0] = 4.0
    out = torch.full_like(x, 9.0)
    d = DeviceGradients([x], [out])
    d.clip(1.0)
    f4._sync()
    norm = math.sqrt(9 * 3 + 16)
    assert abs(float(d.norm) - norm) <= tg.NORM * norm
    tg._check_out([out[-4:].clone(), out[:2].clone()], [x[-4:], x[:2]], norm, 1.0)
    assert int((out == 9.0).sum()) == 0


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("T,din,mid,dout", [
    (24, 288, 416, 96), (100, 512, 2080, 416), (300, 1056, 2080, 288), (2300, 1024, 2080, 1056)])
def test_two_layers_without_a_pause(T, din, mid, dout, fmt):
    """Two layers forward, back and clipped, with new tokens each time and nothing that waits in
    between: every step's results are those of the same calls one at a time."""
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    one, X, _ = f4._layer(custom_linear(T, din, mid, 1, "column"), 3, fmt)
    two, _, dY = f4._layer(custom_linear(T, mid, dout, 1, "row"), 4, fmt)
    clip = DeviceGradients(one.dW + [one.db] + two.dW + [two.db])
    gen = f4._gen(5)
    data = [(f4._randn(gen, T, din), f4._randn(gen, *dY[0].shape)) for _ in range(6)]
    layers = (one, two)

    def run(between):
        seen = []
        for x, dy in data:
            one.forward([x], save=True), between()
            two.forward(one.Y, save=True), between()
            two.backward([dy]), between()
            one.backward(two.dX), between()
            clip.clip(0.05), between()
            seen.append([v.clone() for lay in layers for v in lay.Y + lay.dX + lay.dW + [lay.db]])
        f4._sync()
        return seen

    apart = run(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(apart, run(lambda: None)):
            assert _equal(a, b)


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("split,T,n,t", [
    ("column", 1, 4096, 1), ("row", 8, 512, 1), ("column", 24, 512, 1), ("row", 100, 512, 1), ("column", 600, 1056, 1)])
def test_results_over_inputs(split, T, n, t, fmt):
    """Y where X lies, or a little behind it, and dX where dY lies."""
    lay, X, dY = f4._layer(custom_linear(T, n, n, t, split), 8, fmt)
    lay.forward(X, save=True)
    lay.backward(dY)
    want = [x[0].clone() for x in (lay.Y, lay.dX)]
    for shift in (0, 8, -8, 64, n * (T // 2)):
        # (buffers with room on both sides)
        room = torch.zeros((T + 2) * n + 2 * abs(shift), dtype=torch.bfloat16, device="cuda")
        at = n + abs(shift)
        x, y = (room[k:k + T * n].view(T, n) for k in (at, at + shift))
        for save in (False, True):
            for _ in range(3):
                x.copy_(X[0])
                lay.forward([x], save=save, Y=[y])
                f4._sync()
                assert torch.equal(y, want[0])
        x.copy_(dY[0])
        lay.backward([x], dX=[y])
        f4._sync()
        assert torch.equal(y, want[1])

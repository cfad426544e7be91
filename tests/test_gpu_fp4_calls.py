"""The library's 4-bit and gradient calls under their own names (``binding``), with a caller's tensors:
the same bits as the layers that hold buffers."""
import pytest
import torch

import test_gpu_fp4 as f4
import test_gpu_grad as tg
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _bytes(*sizes):
    return [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("split,T,din,dout,t,chunks", [
    ("column", 9, 256, 320, 2, 1), ("row", 256, 512, 288, 2, 2), ("column", 512, 288, 1088, 1, 4)])
def test_linear(split, T, din, dout, t, chunks, fmt):
    from tensor_transformer_mlp_gemm_gb300 import binding as b
    w = custom_linear(T, din, dout, t, split, seq_chunks=chunks)
    lay, X, dY = f4._layer(w, T, fmt)
    lay.forward(X, save=True)
    lay.backward(dY)
    code, col, n = b.FP4_FORMATS[fmt], split == "column", 1 if split == "column" else t
    K = din // n
    dims = b.make_linear_dims(T, din, dout, t, chunks)
    ws, = _bytes(b.tpmlp_fp4_linear_workspace_bytes(dims, code, True))
    q = _bytes(*[b.tpmlp_fp4_packed_bytes(K, T)] * n)
    s = _bytes(*[b.tpmlp_fp4_scale_bytes(K, T, code)] * n)
    g = torch.empty(1, device="cuda") if code else None
    outs = [torch.empty_like(x) for x in lay.Y + lay.dX + lay.dW + [lay.db]]
    ny, nx = len(lay.Y), len(lay.dX)
    Y, dX, dW, db = outs[:ny], outs[ny:ny + nx], outs[ny + nx:-1], outs[-1]
    kept = (q[0], s[0]) if col else (q, s)

    def shards(ms):
        return [m.q for m in ms], [m.s for m in ms]
    forward = b.tpmlp_fp4_column_linear_forward if col else b.tpmlp_fp4_row_linear_forward
    backward = b.tpmlp_fp4_column_linear_backward if col else b.tpmlp_fp4_row_linear_backward
    forward(dims, code, X, g, False, *kept, *shards(lay.weights.forward), lay.weights.scale, lay.b, Y, ws)
    backward(dims, code, dY, *kept, g, *shards(lay.weights.backward), lay.weights.scale, dX, dW, db, ws)
    f4._sync()
    for a, want in zip(outs, lay.Y + lay.dX + lay.dW + [lay.db]):
        assert torch.equal(a, want)
    # without keeping X, and with the scale that was found
    Y[0].zero_()
    forward(dims, code, X, g, bool(code), None, None, *shards(lay.weights.forward), lay.weights.scale, lay.b, Y, ws)
    f4._sync()
    assert all(torch.equal(a, want) for a, want in zip(Y, lay.Y))


@pytest.mark.parametrize("fmt", f4.FORMATS)
def test_there_and_back(fmt):
    from tensor_transformer_mlp_gemm_gb300 import binding as b, fp4
    xs = [f4._values(130, 96, f4._gen(i)) for i in range(3)]
    code = b.FP4_FORMATS[fmt]
    quant = b.make_fp4_quant(130, 96, 3, False, code)
    g = None
    if code:
        g = torch.empty(1, device="cuda")
        b.tpmlp_fp4_tensor_scale(quant, xs, g)
        assert float(g) == float(fp4.tensor_scale(xs))
    q = _bytes(*[b.tpmlp_fp4_packed_bytes(96, 130)] * 3)
    s = _bytes(*[b.tpmlp_fp4_scale_bytes(96, 130, code)] * 3)
    b.tpmlp_fp4_quantize(quant, xs, g, None, None, q, s)
    for x, qi, si in zip(xs, q, s):
        out = torch.empty(96, 130, dtype=torch.bfloat16, device="cuda")
        b.tpmlp_fp4_dequantize(96, 130, code, qi, si, g, out)
        one = fp4.quantize_tokens(x, fmt, rows=False, cols=True, scale=g).cols
        f4._sync()
        f4._check(one, x, fmt, 0, g)
        assert torch.equal(out, one.values())


def test_gradients():
    from tensor_transformer_mlp_gemm_gb300 import binding as b
    xs = tg._grads([3001, 70, 0, 20000], [torch.float32, torch.bfloat16, torch.float16])
    out = [torch.empty_like(x) for x in xs]
    ts = b.make_grad_tensors([(x, o, x.numel(), b.GRAD_TYPES[x.dtype]) for x, o in zip(xs, out)])
    norm, (ws,) = torch.empty(1, device="cuda"), _bytes(b.tpmlp_grad_workspace_bytes(len(xs)))
    b.tpmlp_grad_norm(ts, len(xs), norm, ws)
    tg._sync()
    want = tg._check_norm(norm, xs)
    norm.zero_()
    b.tpmlp_grad_clip(ts, len(xs), want / 2, norm, ws)
    tg._sync()
    tg._check_norm(norm, xs)
    tg._check_out(out, xs, want, want / 2)

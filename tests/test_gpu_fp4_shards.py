"""4-bit weight shards anywhere in a caller's storage: two of them are always at one step from each
other, which need not be one that a tensor map takes (whole rows of the matrix)."""
import pytest
import torch

import test_gpu_fp4 as f4
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _apart(ms, q_gap, s_gap):
    """The matrices again, with q_gap and s_gap bytes between one's end and the next's start."""
    from tensor_transformer_mlp_gemm_gb300 import fp4

    def lay_out(xs, gap):
        room = torch.full((len(xs) * (xs[0].numel() + gap) + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        at, views = 0, []
        for x in xs:
            views.append(room[at:at + x.numel()].view_as(x).copy_(x))
            at += x.numel() + gap
        return views
    return [fp4.Fp4Matrix(q, s, m.scale, m.shape, m.fmt)
            for m, q, s in zip(ms, lay_out([m.q for m in ms], q_gap), lay_out([m.s for m in ms], s_gap))]


def _misses():
    from tensor_transformer_mlp_gemm_gb300 import binding
    return binding.tpmlp_map_cache_stats()["misses"]


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("split,T,din,dout,t", [
    ("column", 1, 512, 832, 2), ("row", 40, 1088, 416, 2), ("column", 300, 544, 1088, 2), ("row", 700, 1024, 288, 2),
    ("column", 700, 288, 1152, 4)])
def test_any_step(split, T, din, dout, t, fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    lay, X, dY = f4._layer(custom_linear(T, din, dout, t, split), T, fmt)
    lay.forward(X, save=True)
    lay.backward(dY)
    f4._sync()
    f4._check_forward(lay, X)
    f4._check_backward(lay, X, dY)
    want = [x.clone() for x in lay.Y + lay.dX + lay.dW + [lay.db]]
    row = {"forward": lay.weights.forward[0].q.shape[1], "backward": lay.weights.backward[0].q.shape[1]}
    for k, (q_gap, s_gap) in enumerate([(16, 0), (0, 16), (48, 528), (0, 0), ("row", 16), (16, 32), (112, 0)]):
        def gap(way):
            return row[way] if q_gap == "row" else q_gap
        other = fp4.Fp4Weights(_apart(lay.weights.forward, gap("forward"), s_gap),
                               _apart(lay.weights.backward, gap("backward"), s_gap))
        one = fp4.DeviceFp4Linear(lay.w, other, lay.b)
        before = _misses()
        one.forward(X, save=True)
        one.backward(dY)
        f4._sync()
        got = one.Y + one.dX + one.dW + [one.db]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (q_gap, s_gap)
        # a step of no whole rows is in no map: one for each shape, made once
        if k and q_gap not in (0, "row"):
            assert _misses() == before, (q_gap, s_gap)

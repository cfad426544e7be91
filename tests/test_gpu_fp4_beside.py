"""The weight gradient's product runs beside the end of the input gradient's: its results are those
of the same launches one behind the other (event records between them keep them apart)."""
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


@pytest.mark.parametrize("fmt", f4.FORMATS)
@pytest.mark.parametrize("split,T,din,dout,t", [
    # dX: one tile more than pairs, of a long K; dW: many tiles for each pair, one stage each
    ("column", 256, 19712, 8192, 1),
    # dX of few tokens, dW on pairs; several shards; dX and dW of several waves
    ("row", 40, 8192, 4096, 8), ("column", 333, 1056, 2080, 1), ("row", 4096, 4096, 2048, 4)])
def test_beside_and_apart(split, T, din, dout, t, fmt):
    from tensor_transformer_mlp_gemm_gb300 import binding
    lay, X, dY = f4._layer(custom_linear(T, din, dout, t, split), T, fmt)
    lay.forward(X, save=True)
    outs = lay.dX + lay.dW + [lay.db]

    def run(apart):
        for x in outs:
            x.fill_(float("nan"))
        torch.cuda.synchronize()
        if apart:
            binding.tpmlp_profile_begin(64)
        for _ in range(3):
            lay.backward(dY)
        f4._sync()
        if apart:
            binding.tpmlp_profile_end()
        return [x.clone() for x in outs]

    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))

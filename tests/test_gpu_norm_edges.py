"""The norms around a block at the edges of what they take: no tokens with a gate or 8-bit rows."""
import pytest
import torch

import test_gpu_norm as nm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


WEIGHTS = ("dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta")


@pytest.mark.parametrize("gate_rows", [0, 8])
@pytest.mark.parametrize("quantize", [None, "e4m3"])
@pytest.mark.parametrize("chunks", [1, 2])
def test_empty(gate_rows, quantize, chunks):
    d = nm._inputs(0, 64, gate_rows, 11)
    lay = nm._layer(d, 0, 64, "layer", "layer", gate_rows, 1.0, quantize=quantize, seq_chunks=chunks)
    c = lambda x: [x] * chunks  # noqa: E731
    for k in WEIGHTS:
        getattr(lay, k).fill_(3.0)
    lay.forward(c(d["X"]), c(d["Z"]), d["gate"])
    lay.backward(c(d["dOut"]), c(d["dXn"]), c(d["Z"]), lay.Out, gate=d["gate"])
    nm._sync()
    for k in WEIGHTS:
        assert torch.count_nonzero(getattr(lay, k)) == 0
    if gate_rows:
        assert lay.dgate.shape == (0, 64)

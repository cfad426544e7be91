"""The norms around a block at the edges of what they take: no tokens with a gate or 8-bit
rows, wide rows with no norm before, and how many kernels a backward pass launches."""
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


@pytest.mark.parametrize("T,h,gate_rows", [(701, 4096, 0), (701, 3080, 701), (305, 8192, 61), (151, 9000, 0),
                                           (305, 12288, 0), (151, 16384, 151)])
@pytest.mark.parametrize("post", ["rms", "layer", "none"])
def test_no_norm_before(T, h, gate_rows, post):
    """Wide rows, an odd number of them, several pairs for each group: a stage of the ring is
    freed by a barrier of its own where there are no sums of a norm before."""
    nm.test_norm(T, h, gate_rows, post, "none")


@pytest.mark.parametrize("post,pre,gate_rows,launches", [
    ("none", "none", 0, 1), ("none", "none", 1, 1), ("none", "none", 512, 2), ("rms", "none", 0, 2),
    ("none", "rms", 0, 2)])
def test_launches_of_the_backward_pass(post, pre, gate_rows, launches):
    """The profile counts the kernels that were launched: the second one only where there
    are sums over rows for it."""
    from tensor_transformer_mlp_gemm_gb300 import binding
    d = nm._inputs(2048, 256, gate_rows, 3)
    lay = nm._layer(d, 2048, 256, post, pre, gate_rows, 1.0)
    lay.forward(d["X"], d["Z"], d["gate"])
    lay._gradients()
    binding.tpmlp_profile_begin(8)
    lay.backward(d["dOut"], d["dXn"] if pre != "none" else None, d["Z"], lay.Out, gate=d["gate"])
    torch.cuda.synchronize()
    counts = binding.tpmlp_profile_end()[1]
    assert counts["layernorm_bwd"] == launches


@pytest.mark.parametrize("T,chunks,gate_rows", [(96, 4, 32), (240, 8, 80), (240, 8, 20), (60, 2, 12)])
def test_gates_across_chunks(T, chunks, gate_rows):
    """Gates that begin and end inside token chunks, with 8-bit rows and bf16 ones: what whole
    tensors give."""
    from tensor_transformer_mlp_gemm_gb300 import binding
    h = 528
    d = nm._inputs(T, h, gate_rows, T)
    whole = nm._layer(d, T, h, "rms", "layer", gate_rows, 0.9)
    parts = nm._layer(d, T, h, "rms", "layer", gate_rows, 0.9, seq_chunks=chunks)
    eight = nm._layer(d, T, h, "rms", "layer", gate_rows, 0.9, seq_chunks=chunks, quantize="e4m3")
    one = nm._layer(d, T, h, "rms", "layer", gate_rows, 0.9, quantize="e4m3")
    c = lambda x: [t.clone() for t in x.chunk(chunks)]  # noqa: E731
    whole.forward(d["X"], d["Z"], d["gate"])
    one.forward(d["X"], d["Z"], d["gate"])
    X, Z = c(d["X"]), c(d["Z"])
    parts.forward(X, Z, d["gate"])
    eight.forward(X, Z, d["gate"])
    # both forms of Xn, in chunks
    Xn, q, s = c(torch.zeros_like(d["X"])), torch.zeros_like(eight.q), torch.zeros_like(eight.q_scale)
    binding.tpmlp_norm_forward(eight.params, X, Z, eight.post_gamma, None, d["gate"], eight.pre_gamma,
                               eight.pre_beta, [torch.empty_like(x) for x in X], Xn, q, s, None)
    whole.backward(d["dOut"], d["dXn"], d["Z"], whole.Out, gate=d["gate"])
    parts.backward(c(d["dOut"]), c(d["dXn"]), Z, parts.Out, gate=d["gate"])
    nm._sync()
    for k in ("Out", "Xn", "dX", "dZ"):
        assert torch.equal(getattr(whole, k), torch.cat(getattr(parts, k)))
    for k in ("dgate", "dpost_gamma", "dpre_gamma", "dpre_beta"):
        assert torch.equal(getattr(whole, k), getattr(parts, k))
    assert torch.equal(torch.cat(Xn), whole.Xn)
    for got, scale in ((eight.q, eight.q_scale), (q, s)):
        assert torch.equal(got.view(torch.uint8), one.q.view(torch.uint8)) and torch.equal(scale, one.q_scale)
    nm._check_forward(d, whole, whole.Out, whole.Xn, whole.stats)
    nm._check_backward(d, whole, whole.Out, whole.stats, d["dOut"], d["dXn"])

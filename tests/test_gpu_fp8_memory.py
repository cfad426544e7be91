"""What an 8-bit linear layer holds: gradients only once it goes backward."""
import pytest
import torch

import test_gpu_fp8 as f8
from tensor_transformer_mlp_gemm_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


@pytest.mark.parametrize("split", ["column", "row"])
def test_forward_alone_holds_no_gradients(split):
    from tensor_transformer_mlp_gemm_gb300 import fp8
    T, n = 4096, 2048
    w = inputs.custom_linear(T, n, n, 2, split)
    lay, X, dY = f8._layer(w, 3)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    own = fp8.DeviceFp8Linear(w, lay.Wq, lay.Ws, lay.b, workspace=lay.ws)
    x = own.quantize(X, cols=True)
    own.forward(x)
    held = torch.cuda.memory_allocated() - before
    # Y (or Z) in bf16, and X by rows and by columns with their scales
    assert held < 2 * T * n + 2 * (T * n + T * n // 32) + (1 << 20)
    lay.forward(x)
    lay.backward(dY, x)
    own.backward(dY, x)
    f8._sync()
    for a, b in zip(own.Y + own.dX + own.dW + [own.db], lay.Y + lay.dX + lay.dW + [lay.db], strict=True):
        assert torch.equal(a, b)
    # a call's own dX makes none
    third = fp8.DeviceFp8Linear(w, lay.Wq, lay.Ws, lay.b, workspace=lay.ws)
    third.backward(dY, x, dX=[torch.empty_like(t) for t in lay.dX])
    assert third._dX is None
    f8._sync()

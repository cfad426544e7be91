"""Tensors whose addresses a layer holds from the start: nothing takes them out from under it."""
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


def test_weight_shards_stay():
    """A shard, or all of them, are not exchanged beneath a layer (which would go on with the freed
    ones), and a caller's own lists may change."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    w = custom_linear(24, 256, 320, 2, "column")
    lay, X, dY = f4._layer(w, 1, "nvfp4")
    lists = [list(lay.weights.forward), list(lay.weights.backward)]
    own = fp4.Fp4Weights(*lists)
    other = fp4.DeviceFp4Linear(w, own, lay.b)
    for x in lists:
        x.clear()
    for weights in (own, lay.weights):
        for name in ("forward", "backward"):
            shards = getattr(weights, name)
            with pytest.raises(TypeError):
                shards[0] = shards[1]
            with pytest.raises(AttributeError):
                setattr(weights, name, shards[::-1])
    for layer in (lay, other):
        layer.forward(X, save=True)
        layer.backward(dY)
        f4._sync()
        f4._check_forward(layer, X)
        f4._check_backward(layer, X, dY)
    assert torch.equal(other.Y[1], lay.Y[1])


def test_gradients_stay():
    """Neither gradients nor outputs are exchanged beneath a list (which would go on with the freed
    ones), and a caller's own lists may change."""
    import test_gpu_grad as tg
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    xs = tg._grads([3000, 70], [torch.float32, torch.bfloat16])
    out = [torch.empty_like(x) for x in xs]
    keep = [[x.clone() for x in xs], list(out)]
    d = DeviceGradients(xs, out)
    xs.clear()
    out.clear()
    for name in ("grads", "out"):
        with pytest.raises(AttributeError):
            setattr(d, name, ())
        with pytest.raises(TypeError):
            getattr(d, name)[0] = keep[0][0]
    d.clip(1e-3)
    tg._sync()
    want = tg._check_norm(d.norm, keep[0])
    tg._check_out(keep[1], keep[0], want, 1e-3)

"""Clipping by factors that fp32 does not hold, whose products with large gradients it does."""
import pytest
import torch

import test_gpu_grad as tg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _clip(value, max_norm):
    """fp32 and bf16 gradients of this magnitude, and many that are 2^20 times smaller."""
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    xs = tg._grads([1000, 70_001, 40], [torch.float32, torch.bfloat16], 5, value)
    xs[1][40:] *= 2.0 ** -20
    keep = [x.clone() for x in xs]
    out = [torch.empty_like(x) for x in xs]
    into, here = DeviceGradients(xs, out), DeviceGradients(xs)
    into.clip(max_norm)
    here.clip(max_norm)
    tg._sync()
    limit = float(torch.tensor(max_norm))      # (a call takes it in fp32)
    for d, got in ((into, out), (here, xs)):
        want = tg._check_norm(d.norm, keep)
        tg._check_out(got, keep, want, limit)
    assert all(bool((o != 0).any()) for o in out)


@pytest.mark.parametrize("max_norm", [1e-25, 1e-30, 1e-34, 1e-36])
@pytest.mark.parametrize("value", [1e-5, 1.0, 1e5, 1e10])
def test_small_limits(value, max_norm):
    """The quotient of a limit and a norm that fp32 holds may be a number that it does not."""
    _clip(value, max_norm)


@pytest.mark.parametrize("max_norm", [1e-10, 1e-20, 1e-30, 1e-36])
@pytest.mark.parametrize("value", [1e20, 1e28, 1e37])
def test_large_gradients(value, max_norm):
    """Factors down to 1e-75: no one number of fp32, and no product of two with 2^-64 for one."""
    _clip(value, max_norm)

"""The scale of a small nvfp4 tensor, which one cluster of eight CTAs finds: each CTA's largest
value counts, whenever that CTA starts beside what still runs."""
import pytest
import torch

import plain_fp4 as plain
import test_gpu_fp4 as f4
from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

pytestmark = pytest.mark.gpu
CTA = 1024 * 8  # values that a CTA takes of each 8 * CTA


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


@pytest.mark.parametrize("parts", [1, 2, 8])
def test_largest_in_each_cta(parts):
    """The largest in each CTA's share in turn, call behind call without a pause, each with another
    scale: a maximum that were lost, or were another call's, would show."""
    from tensor_transformer_mlp_gemm_gb300 import fp4
    values = 1 << 18
    rows = values // parts // 512
    xs, scales, wants = [], [], []
    for i in range(64):
        x = torch.full((values,), 2.0 ** -3, device="cuda", dtype=torch.bfloat16)
        x[(i % 32) * CTA + 7 * i] = 6.0 * 448.0 * 2.0 ** (i % 13)
        xs.append(list(x.view(parts, rows, 512).unbind(0)))
        wants.append(2.0 ** (i % 13))
    torch.cuda.synchronize()
    for _ in range(4):
        scales += [fp4.tensor_scale(x) for x in xs]
    f4._sync()
    assert [float(s) for s in scales] == wants * 4


def test_behind_kernels_that_still_run():
    """Uncalibrated forward calls of few tokens behind a larger layer's product, whose CTAs leave
    their SMs one by one while the cluster starts."""
    big, X, _ = f4._layer(custom_linear(2048, 2048, 4096, 1, "column"), 1, "nvfp4", backward=False)
    few, _, _ = f4._layer(custom_linear(8, 512, 1024, 1, "column"), 2, "nvfp4", backward=False)
    inputs = [f4._randn(f4._gen(i), 8, 512, std=4.0 ** (i % 9)) for i in range(24)]
    outs = [torch.empty_like(few.Y[0]) for _ in inputs]
    scales = []
    for x, y in zip(inputs, outs):
        big.forward(X)
        few.forward([x], Y=[y])
        scales.append(few._scales[0].clone())
    f4._sync()
    for x, y, s in zip(inputs, outs, scales):
        assert float(s) == float(plain.tensor_scale([x]))
        f4._check_forward(few, [x], [y])

"""4-bit matrices whose summed axis is so long that offsets along it pass 2^31 and 2^32 bytes."""
import gc

import pytest
import torch

import test_gpu_fp4 as f4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


@pytest.fixture(autouse=True)
def _room():
    """(up to 150 GB in a test)"""
    gc.collect()
    torch.cuda.empty_cache()
    yield
    gc.collect()
    torch.cuda.empty_cache()


# where the bytes of scales of 128 rows, times 128 of K 512 (mx) or 1024 (nv), pass 2^32
PAST = {"mxfp4": (1 << 30) + 512, "nvfp4": (1 << 29) + 512}
PERIOD = 1 << 16


def _periodic(m, x):
    """A matrix made of a piece of PERIOD along its summed axis, again and again, and of the start of
    one at the end: so are its values and scales."""
    for got, one, step in ((m.q, x.q, PERIOD // 2), (m.s.view(1, -1), x.s.view(1, -1), x.s.numel())):
        whole = got.shape[1] // step
        assert torch.equal(got[:, :step], one[:, :step])
        for k in range(1, whole):
            if not torch.equal(got[:, k * step:(k + 1) * step], one[:, :step]):
                pytest.fail(f"piece {k} of {whole}")
        rest = got.shape[1] - whole * step
        assert rest > 0 and torch.equal(got[:, whole * step:], one[:, :rest])


@pytest.mark.parametrize("fmt", f4.FORMATS)
def test_quantise_rows(fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    K = PAST[fmt]
    piece = f4._values(1, PERIOD, f4._gen(1))
    scale = None if fmt == "mxfp4" else torch.full((1,), 2.0 ** -3, device="cuda")
    one = fp4.quantize_tokens(piece, fmt, scale=scale).rows
    f4._check(one, piece, fmt, 1, None if scale is None else 2.0 ** -3)
    x = torch.cat([piece.repeat(1, K // PERIOD), piece[:, :K % PERIOD]], 1)
    got = fp4.quantize_tokens(x, fmt, scale=scale).rows
    f4._sync()
    _periodic(got, one)


@pytest.mark.parametrize("fmt", f4.FORMATS)
def test_quantise_columns(fmt):
    from tensor_transformer_mlp_gemm_gb300 import fp4
    T = PAST[fmt]
    piece = f4._values(PERIOD, 32, f4._gen(2))
    scale = None if fmt == "mxfp4" else torch.full((1,), 2.0 ** -3, device="cuda")
    one = fp4.quantize_tokens(piece, fmt, rows=False, cols=True, scale=scale).cols
    f4._check(one, piece, fmt, 0, None if scale is None else 2.0 ** -3)
    x = torch.empty(T, 32, dtype=torch.bfloat16, device="cuda")
    x[:T // PERIOD * PERIOD].view(-1, PERIOD, 32).copy_(piece.expand(T // PERIOD, -1, -1))
    x[T // PERIOD * PERIOD:] = piece[:T % PERIOD]
    got = fp4.quantize_tokens(x, fmt, rows=False, cols=True, scale=scale).cols
    f4._sync()
    _periodic(got, one)

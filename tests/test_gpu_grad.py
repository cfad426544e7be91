"""The norm of many gradients and clipping by it, on the GPU, against 64 bits."""
import math

import pytest
import torch

from guard import GuardBands

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
# at most 64 squares are added in fp32, each addition off by 2^-24 of the sum, which the root
# halves; one rounding of the norm
NORM = 33 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _grads(sizes, dtypes, seed=0, std=1e-3):
    g = _gen(seed)
    return [(torch.randn(n, generator=g, device="cuda") * std).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def _sync():
    from tensor_transformer_mlp_gemm_gb300 import binding
    assert binding.tpmlp_sync_check() == binding.TPMLP_OK


def _norm64(xs):
    return math.sqrt(math.fsum(float(x.double().square().sum()) for x in xs))


def _check_norm(got, xs):
    want = _norm64(xs)
    # above fp32's range, as 3e37 sqrt(70501) = 8.0e39 is (the largest: 3.4e38): an infinity;
    # gradients are clipped by the norm that it stands for
    if want > torch.finfo(F32).max * (1 + NORM):
        assert float(got) == math.inf
        return want
    assert abs(float(got) - want) <= NORM * want, (float(got), want)
    return want


def _check_out(out, grads, norm, max_norm):
    """The factor is off by the norm's error and a rounding, the product by one of its type (of
    fp16's smallest values, by half their step)."""
    c = min(1.0, max_norm / (norm + 1e-6))
    for o, g in zip(out, grads):
        assert o.dtype == g.dtype and o.shape == g.shape
        ref = g.double() * c
        eps = torch.finfo(g.dtype).eps / 2
        bound = ref.abs() * (eps * (1 + 2.0 ** -10) + NORM + 2.0 ** -24)
        bound = bound + (2.0 ** -25 if g.dtype is F16 else 2.0 ** -133 if g.dtype is BF16 else 2.0 ** -149)
        d = (o.double() - ref).abs() - bound
        assert d.numel() == 0 or float(d.max()) <= 0, float(d.max())


SIZES = [
    [1], [5], [1024], [4096 * 3 + 1], [1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 31, 33],
    [0, 7, 0, 100000, 0], [256 * 512] * 4 + [1024, 256], [1 << 20, 3, (1 << 20) + 1, 12345],
    [7_000_001, 9, 500_003], [513] * 40, [129] * 1100, [40_000_000 + 3],
]


@pytest.mark.parametrize("dtypes", [[F32], [BF16], [F16], [F32, BF16, F16]])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(sizes, dtypes):
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    xs = _grads(sizes, dtypes, len(sizes) + max(sizes))
    guard = GuardBands()
    few = len(xs) <= 50
    out = [guard.like(x, str(i)) if few and x.numel() else torch.empty_like(x) for i, x in enumerate(xs)]
    keep = [x.clone() for x in xs]
    d = DeviceGradients(xs, out)
    want = _check_norm(d.measure(), keep)
    for max_norm in (want / 3, want * 2):
        assert d.clip(max_norm) is d.norm
        _sync()
        _check_norm(d.norm, keep)
        _check_out(out, keep, want, max_norm)
        guard.check()
    for x, k in zip(xs, keep):
        assert torch.equal(x, k)
    # in place
    d = DeviceGradients(xs)
    d.clip(want * 2)
    _sync()
    for x, k in zip(xs, keep):
        assert torch.equal(x, k)
    d.clip(want / 3)
    _sync()
    _check_norm(d.norm, keep)
    _check_out(xs, keep, want, want / 3)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_views_of_any_alignment(dtype):
    """Gradients and outputs that start anywhere in a larger buffer, at different places of 16 bytes."""
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    for a in range(0, 9):
        for b in (0, 1, a):
            flat = (torch.randn(3000, generator=_gen(a), device="cuda")).to(dtype)
            to = torch.full((3000,), 7.0, device="cuda").to(dtype)
            sizes = [1, 2, 1001 + a, 8, 900]
            xs, out, at = [], [], 0
            for n in sizes:
                xs.append(flat[at + a:at + a + n])
                out.append(to[at + b:at + b + n])
                at += n + 3
            d = DeviceGradients(xs, out)
            d.clip(0.25)
            _sync()
            _check_out(out, xs, _check_norm(d.norm, xs), 0.25)
            # what lies between is left as it was
            mark = torch.zeros(3000, dtype=torch.bool, device="cuda")
            at = 0
            for n in sizes:
                mark[at + b:at + b + n] = True
                at += n + 3
            assert bool((to[~mark] == 7.0).all())


@pytest.mark.parametrize("value", [1e-30, 1e-22, 1e-19, 1e-3, 1e15, 1e19, 3e37])
def test_magnitudes(value):
    """Squares that fp32 cannot hold."""
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    xs = [torch.full((n,), value, device="cuda") for n in (1, 1000, 70000)]
    xs[1][::2] = 0
    xs.append(torch.zeros(30000, device="cuda"))
    d = DeviceGradients(xs, [torch.empty_like(x) for x in xs])
    d.clip(1.0)
    _sync()
    want = _check_norm(d.norm, xs)
    _check_out(d.out, xs, want, 1.0)


def test_mixed_magnitudes():
    """A few large values among many whose squares vanish beside them, and the other way."""
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    x = _grads([100_000], [F32], 3)[0]
    x[::1000] *= 1e20
    x[1::7] *= 1e-25
    d = DeviceGradients([x], [torch.empty_like(x)])
    d.clip(1.0)
    _sync()
    _check_out(d.out, [x], _check_norm(d.norm, [x]), 1.0)


def test_zeros_and_empty():
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    for xs in ([torch.zeros(5000, device="cuda")], [torch.zeros(0, device="cuda")],
               [torch.zeros(0, device="cuda"), torch.zeros(3, device="cuda", dtype=BF16)]):
        out = [torch.full_like(x, 3.0) for x in xs]
        d = DeviceGradients(xs, out)
        d.norm.fill_(5)
        d.clip(1.0)
        _sync()
        assert float(d.norm) == 0.0 and all(bool((o == 0).all()) for o in out)
        d.norm.fill_(5)
        d.measure()
        _sync()
        assert float(d.norm) == 0.0


def test_max_norm_zero():
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    x = _grads([1000], [F32])[0]
    d = DeviceGradients([x])
    d.clip(0.0)
    _sync()
    assert bool((x == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
def test_not_finite(dtype):
    """An infinity: the norm is infinite, everything 0, infinities NaN.  A NaN: all NaN."""
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    xs = _grads([5000, 77], [dtype])
    xs[1][3] = -math.inf
    out = [torch.empty_like(x) for x in xs]
    d = DeviceGradients(xs, out)
    d.clip(1.0)
    _sync()
    assert float(d.norm) == math.inf
    assert bool((out[0] == 0).all()) and int(torch.isnan(out[1]).sum()) == 1 and bool(torch.isnan(out[1][3]))
    assert int((out[1] == 0).sum()) == 76
    xs[0][4999] = math.nan
    d.clip(1.0)
    _sync()
    assert math.isnan(float(d.norm)) and all(bool(torch.isnan(o).all()) for o in out)


def test_same_bits_every_run():
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    xs = _grads([3_000_001, 70, 1_234_567], [F32, BF16])
    out = [torch.empty_like(x) for x in xs]
    d = DeviceGradients(xs, out)
    first = None
    for _ in range(10):
        d.clip(0.1)
        _sync()
        now = [d.norm.clone()] + [o.clone() for o in out]
        if first is None:
            first = now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_capture_and_replay():
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    xs = _grads([300_001, 50, 40_000], [F32, F16])
    out = [torch.empty_like(x) for x in xs]
    d = DeviceGradients(xs, out)
    d.clip(0.1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.clip(0.1)
    for k in range(3):
        for x in xs:
            x.mul_(1.5)
        graph.replay()
        _sync()
        _check_out(out, xs, _check_norm(d.norm, xs), 0.1)


@pytest.mark.parametrize("raw", [False, True])
def test_another_stream(raw):
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    s = torch.cuda.Stream()
    xs = _grads([5_000_000], [F32])
    out = [torch.empty_like(x) for x in xs]
    d = DeviceGradients(xs, out)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            xs[0].mul_(1.01)
    d.clip(0.1, stream=s.cuda_stream if raw else s)
    s.synchronize()
    _check_out(out, xs, _check_norm(d.norm, xs), 0.1)


def test_refusals():
    from tensor_transformer_mlp_gemm_gb300 import binding
    from tensor_transformer_mlp_gemm_gb300.grad import DeviceGradients
    x, y = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    for grads, out in (([], None), ([x], []), ([x], [y, y]), ([x], [y[:32]]), ([x], [y.bfloat16()]),
                       ([x.double()], None), ([x[::2]], None), ([x.cpu()], None), ([x], [y.cpu()]),
                       ([x.view(8, 8).t()], None), ([x.int()], None),
                       ([x, x], None), ([x[:32], x[16:48]], None), ([x[:32], x[32:]], [x[32:], y[:32]]),
                       ([x[:32], y[:32]], [y[32:], y[32:]]), ([x[:32]], [x[8:40]])):
        with pytest.raises(ValueError):
            DeviceGradients(grads, out)
    d = DeviceGradients([x])
    for bad in (-1.0, math.nan, math.inf):
        with pytest.raises(binding.TpmlpError):
            d.clip(bad)
    # one behind the other, and swapped with room between, is fine
    DeviceGradients([x[:32], x[32:]], [y[32:], y[:32]])

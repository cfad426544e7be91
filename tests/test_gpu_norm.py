"""The norms around a block on the GPU against the plain 64-bit form, within bounds
that follow from their roundings (one bf16 rounding of an output, fp32 inside)."""
import pytest
import torch

import plain_fp8
import plain_norm as plain
from guard import GuardBands

pytestmark = pytest.mark.gpu

EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _setup(gpu):
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    yield


def _sync():
    from tensor_transformer_mlp_gemm_gb300 import binding
    assert binding.tpmlp_sync_check() == binding.TPMLP_OK


def _inputs(T, h, gate_rows, seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    r = lambda *s, std=1.0, mean=0.0: (mean + std * torch.randn(*s, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
    d = {"X": r(T, h, std=2.0, mean=0.5), "Z": r(T, h, std=0.7, mean=-0.3), "dOut": r(T, h), "dXn": r(T, h),
         "post_gamma": r(h, std=0.2, mean=1.0), "post_beta": r(h, std=0.1),
         "pre_gamma": r(h, std=0.2, mean=1.0), "pre_beta": r(h, std=0.1)}
    d["gate"] = r(T // gate_rows, h, std=0.5) if gate_rows else None
    return d


def _layer(d, T, h, post, pre, gate_rows, alpha, **kw):
    from tensor_transformer_mlp_gemm_gb300.norm import DeviceNormResidual
    return DeviceNormResidual(T, h, post, pre, gate_rows, alpha, EPS, d["post_gamma"], d["post_beta"],
                              d["pre_gamma"], d["pre_beta"], device="cuda:0", **kw)


def _within(name, got, ref, mag, rounding, steps=plain.STEPS):
    bound = steps * plain.F32 * mag
    plain_fp8.check(name, got, ref, bound + rounding * (ref.abs() + bound))


def _rows(gate, gate_rows):
    return gate.double().repeat_interleave(gate_rows, 0) if gate is not None else None


def _check_forward(d, lay, Out, Xn, stats, z=True):
    """Out from X and Z; Xn and the statistics from the Out that was stored."""
    post, pre = lay.post, lay.pre
    if z:
        Z = d["Z"].double()
        ref, mag, mean, rstd = plain.forward(d["X"].double(), Z, post, d["post_gamma"].double(),
                                             d["post_beta"].double(), _rows(d["gate"], lay.gate_rows),
                                             lay.params.residual_scale, EPS)
        _within("Out", Out, ref, mag, plain.BF16)
        if post != "none":
            _within("mean of Z", stats[0], mean, Z.abs().mean(1), plain.F32)
            _within("rstd of Z", stats[1], rstd, rstd, plain.F32)
    else:
        Out = d["X"]
    if pre == "none":
        return None
    o = Out.double()
    mean, rstd = plain.stats_of(o, pre, EPS)
    _within("mean of Out", stats[2], mean, o.abs().mean(1), plain.F32)
    _within("rstd of Out", stats[3], rstd, rstd, plain.F32)
    ref, mag = plain.normed(o, pre, d["pre_gamma"].double(), d["pre_beta"].double(), mean, rstd)
    if Xn is not None:
        _within("Xn", Xn, ref, mag, plain.BF16)
    return ref, mag


def _check_backward(d, lay, Out, stats, dOut, dXn, z=True):
    T, L = lay.tokens, lay.gate_rows
    zero = torch.zeros_like(d["X"]).double()
    w = {k: d[k].double() for k in ("post_gamma", "post_beta", "pre_gamma")}
    ref = plain.backward(zero if dOut is None else dOut.double(),
                         zero if dXn is None else dXn.double(), d["Z"].double() if z else None,
                         Out.double(), lay.post, lay.pre, w["post_gamma"], w["post_beta"],
                         _rows(d["gate"], L) if z else None, w["pre_gamma"],
                         lay.params.residual_scale if z else 1.0, tuple(stats.double()))
    # a column sum adds up to all rows of a block, then a block in 8 at a time
    adds = T + 64
    for name, (v, mag) in ref.items():
        got = getattr(lay, name)
        if name in ("dX", "dZ"):
            got = got if isinstance(got, torch.Tensor) else torch.cat(got)
            _within(name, got, v, mag, plain.BF16)
        else:
            n = L if name == "dgate" else T
            v, mag = v.view(-1, n, lay.hidden).sum(1), mag.view(-1, n, lay.hidden).sum(1)
            v, mag = (v, mag) if name == "dgate" else (v[0], mag[0])
            _within(name, got, v, mag, plain.F32, plain.STEPS + min(adds, n + 64))


CASES = [
    # T, h, gate_rows, post, pre
    (1, 8, 0, "rms", "rms"),
    (1, 12288, 1, "rms", "rms"),
    (2, 1000, 1, "layer", "layer"),
    (5, 2048, 5, "rms", "layer"),
    (37, 2056, 37, "layer", "rms"),
    (300, 256, 1, "rms", "rms"),          # a gate row for each token
    (333, 1040, 111, "layer", "layer"),
    (400, 4096, 100, "rms", "rms"),
    (130, 4104, 13, "layer", "layer"),    # just above one CTA's columns: a cluster of two
    (77, 8200, 7, "rms", "layer"),        # a cluster of four, its last CTA without columns
    (60, 16384, 60, "layer", "layer"),
    (200, 640, 0, "none", "rms"),
    (200, 640, 50, "none", "layer"),
    (128, 768, 32, "rms", "none"),
    (128, 768, 0, "none", "none"),
    (1000, 512, 4, "layer", "rms"),       # 250 gates: more than there are blocks
    (2000, 24, 500, "rms", "rms"),
]


@pytest.mark.parametrize("T,h,gate_rows,post,pre", CASES)
def test_norm(T, h, gate_rows, post, pre):
    d = _inputs(T, h, gate_rows, T + h)
    lay = _layer(d, T, h, post, pre, gate_rows, 0.75)
    g = GuardBands()
    g.guard(lay, ["_Out", "stats"] + (["_Xn"] if pre != "none" else []))
    grads = lay._gradients()
    for k, v in grads.items():
        grads[k] = [g.like(x, k) for x in v] if isinstance(v, list) else None if v is None else g.like(v, k)

    class Watched:
        pass
    w = Watched()
    w.__dict__.update({k: v for k, v in d.items() if v is not None})
    g.watch_inputs(w, list(w.__dict__))
    lay.forward(d["X"], d["Z"], gate=d["gate"])
    dXn = d["dXn"] if pre != "none" else None
    lay.backward(d["dOut"], dXn, d["Z"], lay.Out, gate=d["gate"])
    _sync()
    g.check()
    _check_forward(d, lay, lay.Out, lay.Xn, lay.stats)
    _check_backward(d, lay, lay.Out, lay.stats, d["dOut"], dXn)


@pytest.mark.parametrize("T,h", [(1, 4096), (9, 272), (130, 12288)])
@pytest.mark.parametrize("pre", ["rms", "layer"])
def test_norm_before_alone(T, h, pre):
    """No block before: Xn = N_pre(X), and its gradient with and without one of Out."""
    d = _inputs(T, h, 0, 5)
    lay = _layer(d, T, h, "none", pre, 0, 0.3)
    lay.forward(d["X"])
    _sync()
    _check_forward(d, lay, None, lay.Xn, lay.stats, z=False)
    for dOut in (None, d["dOut"]):
        lay.backward(dOut, d["dXn"], None, d["X"])
        _sync()
        _check_backward(d, lay, d["X"], lay.stats, dOut, d["dXn"], z=False)


def test_no_gradient_of_out():
    d = _inputs(50, 1024, 10, 6)
    lay = _layer(d, 50, 1024, "rms", "rms", 10, 1.0)
    lay.forward(d["X"], d["Z"], gate=d["gate"])
    lay.backward(None, d["dXn"], d["Z"], lay.Out, gate=d["gate"])
    _sync()
    _check_backward(d, lay, lay.Out, lay.stats, None, d["dXn"])


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("T,h", [(1, 16), (7, 4096), (65, 4112), (33, 9008)])
def test_norm_quantized(T, h, fmt):
    """Both forms of Xn from one call: the 8-bit one is the bf16 one, quantised."""
    from tensor_transformer_mlp_gemm_gb300 import binding, fp8
    d = _inputs(T, h, T, 8)
    lay = _layer(d, T, h, "rms", "layer", T, 0.5, quantize=fmt)
    lay.forward(d["X"], d["Z"], gate=d["gate"])
    q, s, out = lay.q.clone(), lay.q_scale.clone(), lay.Out.clone()
    Xn = torch.empty(T, h, dtype=torch.bfloat16, device="cuda")
    binding.tpmlp_norm_forward(lay.params, [d["X"]], [d["Z"]], lay.post_gamma, None, d["gate"],
                               lay.pre_gamma, lay.pre_beta, [lay.Out], [Xn], lay.q, lay.q_scale, None)
    want = fp8.quantize_tokens(Xn, fmt)
    _sync()
    assert bool((lay.Out == out).all())
    for a, b in ((q, lay.q), (want.rows, lay.q)):
        assert bool((a.view(torch.uint8) == b.view(torch.uint8)).all())
    for a, b in ((s, lay.q_scale), (want.row_scale, lay.q_scale)):
        assert bool((a == b).all())
    _check_forward(d, lay, lay.Out, Xn, lay.stats)


def test_norm_chunks():
    d = _inputs(96, 520, 24, 9)
    whole = _layer(d, 96, 520, "layer", "rms", 24, 0.9)
    parts = _layer(d, 96, 520, "layer", "rms", 24, 0.9, seq_chunks=4)
    c = lambda x: [t.clone() for t in x.chunk(4)]  # noqa: E731
    whole.forward(d["X"], d["Z"], gate=d["gate"])
    parts.forward(c(d["X"]), c(d["Z"]), gate=d["gate"])
    whole.backward(d["dOut"], d["dXn"], d["Z"], whole.Out, gate=d["gate"])
    parts.backward(c(d["dOut"]), c(d["dXn"]), c(d["Z"]), parts.Out, gate=d["gate"])
    _sync()
    for k in ("Out", "Xn", "dX", "dZ"):
        assert torch.equal(getattr(whole, k), torch.cat(getattr(parts, k)))
    for k in ("dgate", "dpost_gamma", "dpost_beta", "dpre_gamma"):
        assert torch.equal(getattr(whole, k), getattr(parts, k))


def test_norm_not_finite():
    """An infinity stays in its row (and in the sums of its columns)."""
    d = _inputs(40, 1024, 10, 10)
    lay = _layer(d, 40, 1024, "rms", "rms", 10, 1.0, quantize="e4m3")
    d["Z"][17, 5] = float("inf")
    lay.forward(d["X"], d["Z"], gate=d["gate"])
    lay.backward(d["dOut"], d["dXn"], d["Z"], lay.Out, gate=d["gate"])
    _sync()
    rows = torch.arange(40, device="cuda") != 17
    assert torch.isfinite(lay.Out[rows]).all() and not torch.isfinite(lay.Out[17]).all()
    assert torch.isnan(lay.q_scale[:, 17]).all() and not torch.isnan(lay.q_scale[:, rows]).any()
    assert (lay.q[17].float() == 0).all()
    assert torch.isfinite(lay.dX[rows]).all() and torch.isnan(lay.dX[17]).all()
    assert torch.isfinite(lay.dgate[[0, 2, 3]]).all() and torch.isnan(lay.dgate[1]).all()
    assert torch.isnan(lay.dpre_gamma).all()


def test_norm_empty():
    d = _inputs(0, 64, 0, 11)
    lay = _layer(d, 0, 64, "layer", "layer", 0, 1.0)
    for k in ("dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta"):
        getattr(lay, k).fill_(3.0)
    lay.forward(d["X"], d["Z"])
    lay.backward(d["dOut"], d["dXn"], d["Z"], lay.Out)
    _sync()
    for k in ("dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta"):
        assert torch.count_nonzero(getattr(lay, k)) == 0

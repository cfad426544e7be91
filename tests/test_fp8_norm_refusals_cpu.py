"""What the 8-bit calls and the norms refuse, without a GPU: the checks come before the
device is looked at, so pointers that are never followed stand in for the tensors."""
import ctypes

import pytest
import torch

from tensor_transformer_mlp_gemm_gb300.inputs import custom_linear

OK_PTR = 0x10000  # 16-byte aligned, never followed
BAD_PTR = OK_PTR + 8  # not on 16 bytes
BAD_SCALE = OK_PTR + 2
SCALES = ("s", "Xs", "Ws", "stats")


def bad_of(name):
    return BAD_SCALE if name in SCALES else BAD_PTR


@pytest.fixture(scope="module")
def b():
    from tensor_transformer_mlp_gemm_gb300.build import build
    build()
    from tensor_transformer_mlp_gemm_gb300 import binding
    return binding


def arr(*xs):
    return (ctypes.c_void_p * max(len(xs), 1))(*xs)


# ---- quantisation -------------------------------------------------------------------------

def _quantize(lib, rows=256, cols=128, ld=256, parts=1, fr=0, fc=0, src=None, q=None, s=None, qc=None,
              sc=None, row=True, col=False):
    d = lib.make_fp8_quant(rows, cols, ld, parts, fr, fc)
    n = max(parts, 1)
    one = arr(*([OK_PTR] * n))
    return lib.library().tpmlp_fp8_quantize(
        ctypes.byref(d), one if src is None else src, (one if q is None else q) if row else None,
        (one if s is None else s) if row else None, (one if qc is None else qc) if col else None,
        (one if sc is None else sc) if col else None, None)


def test_quantize(b):
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    assert b.library().tpmlp_fp8_quantize(None, None, None, None, None, None, None) == INV
    assert _quantize(b, rows=-1) == INV
    assert _quantize(b, cols=0) == INV
    assert _quantize(b, parts=0) == INV
    assert _quantize(b, fr=2) == INV and _quantize(b, fc=-1, col=True) == INV
    assert _quantize(b, row=False) == INV                 # neither grouping
    assert _quantize(b, ld=255) == INV                    # the scales' rows overlap
    assert _quantize(b, cols=136) == UNS                  # not a multiple of 16
    assert _quantize(b, parts=9) == UNS
    assert _quantize(b, rows=1 << 31, ld=1 << 31) == UNS
    assert _quantize(b, cols=1 << 31) == UNS
    assert _quantize(b, src=arr(None)) == INV and _quantize(b, src=arr(BAD_PTR)) == UNS
    for name in ("q", "s"):
        assert _quantize(b, **{name: arr(None)}) == INV
        assert _quantize(b, **{name: arr(bad_of(name))}) == UNS
        assert _quantize(b, col=True, **{name + "c": arr(None)}) == INV
        assert _quantize(b, col=True, **{name + "c": arr(bad_of(name))}) == UNS
    # one half of a pair
    d, one = b.make_fp8_quant(256, 128, 256, 1, 0, 0), arr(OK_PTR)
    call = b.library().tpmlp_fp8_quantize
    assert call(ctypes.byref(d), one, one, None, None, None, None) == INV
    assert call(ctypes.byref(d), one, None, None, None, one, None) == INV


def test_quantize_weight(b):
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    call = b.library().tpmlp_fp8_quantize_weight
    assert call(OK_PTR, 0, 128, 0, OK_PTR, OK_PTR, None) == INV
    assert call(OK_PTR, 128, -16, 0, OK_PTR, OK_PTR, None) == INV
    assert call(OK_PTR, 128, 128, 2, OK_PTR, OK_PTR, None) == INV
    assert call(OK_PTR, 128, 120, 0, OK_PTR, OK_PTR, None) == UNS
    assert call(OK_PTR, 1 << 31, 128, 0, OK_PTR, OK_PTR, None) == UNS
    for i in range(3):
        for bad, want in ((None, INV), (BAD_SCALE if i == 2 else BAD_PTR, UNS)):
            p = [OK_PTR] * 3
            p[i] = bad
            assert call(p[0], 128, 128, 0, p[1], p[2], None) == want


# ---- the linear layers ---------------------------------------------------------------------

def _linear(lib, split, back, dims=None, fmt=(0, 0, 0), **bad):
    """A call with valid stand-ins but for `bad` (argument name -> value)."""
    d = dims or lib.make_linear_dims(256, 256, 512, 2, 2)
    t, n, col = max(d.t, 1), max(d.seq_chunks, 1), split == "column"
    many = lambda k: arr(*([OK_PTR] * k))  # noqa: E731
    x = OK_PTR if col else many(t)
    a = {"Xq": x, "Xs": x, "Wq": many(t), "Ws": many(t), "b": OK_PTR, "Y": many(t if col else n),
         "dY": many(t if col else n), "dX": many(n if col else t), "dW": many(t), "db": OK_PTR, "ws": OK_PTR}
    a.update(bad)
    f = None if fmt is None else lib.make_fp8_formats(*fmt)
    args = [ctypes.byref(d), None if f is None else ctypes.byref(f)]
    names = (("dY", "Xq", "Xs", "Wq", "Ws", "dX", "dW", "db", "ws") if back
             else ("Xq", "Xs", "Wq", "Ws", "b", "Y", "ws"))
    fn = getattr(lib.library(), f"tpmlp_fp8_{split}_linear_{'backward' if back else 'forward'}")
    return fn(*args, *[a[k] for k in names], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("split", ["column", "row"])
def test_linear(b, split, back):
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    mk = b.make_linear_dims
    col = split == "column"
    call = lambda **kw: _linear(b, split, back, **kw)  # noqa: E731
    for dims in (mk(-1, 256, 512, 2), mk(256, 0, 512, 2), mk(256, 256, -512, 2), mk(256, 256, 512, 0),
                 mk(256, 256, 512, 2, 0), mk(257, 256, 512, 2, 2)):
        assert call(dims=dims) == INV
    assert call(dims=mk(256, 250, 250, 3)) == INV                        # t does not divide the shards
    for dims in (mk(256, 2304, 2304, 9), mk(128 * 9, 256, 512, 2, 9),    # more than 8
                 mk(256, 264, 264, 1), mk(256, 272, 272, 2),             # 16 does not divide
                 mk(192 * 2, 256, 512, 2, 2),                            # chunks of 192
                 mk(1 << 31, 256, 512, 2)):
        assert call(dims=dims) == UNS
    for i in range(3):
        f = [0, 0, 0]
        f[i] = 2
        assert call(fmt=tuple(f)) == INV
    assert call(fmt=None) == INV
    lists = ["Wq", "Ws"] + (["dY", "dX", "dW"] if back else ["Y"]) + ([] if col else ["Xq", "Xs"])
    for name in lists:
        assert call(**{name: None}) == INV
        assert call(**{name: arr(OK_PTR, None)}) == INV
        assert call(**{name: arr(OK_PTR, bad_of(name))}) == UNS
    for name in (["db", "ws"] if back else ["b", "ws"]) + (["Xq", "Xs"] if col else []):
        assert call(**{name: None}) == INV
        assert call(**{name: bad_of(name)}) == UNS


def test_linear_workspace(b):
    mk, size = b.make_linear_dims, b.tpmlp_fp8_linear_workspace_bytes
    assert size(mk(256, 264, 264, 1)) == 0
    # the 8-bit gradient by rows and by columns
    assert size(mk(2048, 4096, 4096, 8)) >= 2 * 2048 * 4096
    assert size(mk(0, 256, 512, 2)) > 0
    assert b.library().tpmlp_fp8_linear_workspace_bytes(None) == 0


# ---- the norms -------------------------------------------------------------------------------

FORWARD = ("X", "Z", "post_gamma", "post_beta", "gate", "pre_gamma", "pre_beta", "Out", "Xn", "Xq", "Xs",
           "stats")
BACKWARD = ("dOut", "dXn", "Z", "Out", "post_gamma", "post_beta", "gate", "pre_gamma", "stats", "dX", "dZ",
            "dpost_gamma", "dpost_beta", "dgate", "dpre_gamma", "dpre_beta", "ws")
CHUNKED = ("X", "Z", "Out", "Xn", "dOut", "dXn", "dX", "dZ")
KINDS = {"none": 0, "rms": 1, "layer": 2}


def _norm(lib, back, post="layer", pre="layer", tokens=256, hidden=512, gate_rows=64, chunks=2, fmt=0,
          eps=1e-5, alpha=1.0, **bad):
    d = lib.make_norm_params(tokens, hidden, KINDS.get(post, post), KINDS.get(pre, pre), gate_rows, chunks, fmt,
                           eps, alpha)
    n = max(chunks, 1)
    a = {k: arr(*([OK_PTR] * n)) if k in CHUNKED else OK_PTR for k in FORWARD + BACKWARD}
    unused = [f"{d_}{w}_{k}" for w, kind in (("post", post), ("pre", pre)) for d_ in ("", "d")
              for k, has in (("gamma", kind != "none"), ("beta", kind == "layer")) if not has]
    if not gate_rows:
        unused += ["gate", "dgate"]
    if pre == "none":
        unused += ["Xn", "Xq", "Xs", "dXn"] + (["Out"] if back else [])
    for k in unused:
        a[k] = None
    a.update(bad)
    fn = lib.library().tpmlp_norm_backward if back else lib.library().tpmlp_norm_forward
    return fn(ctypes.byref(d), *[a[k] for k in (BACKWARD if back else FORWARD)], None)


@pytest.mark.parametrize("back", [False, True])
def test_norm_params(b, back):
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    for kw in (dict(tokens=-2), dict(hidden=0), dict(chunks=0), dict(chunks=3, tokens=256), dict(gate_rows=-1),
               dict(gate_rows=96), dict(post=3), dict(pre=-1), dict(eps=-1e-6), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(alpha=float("nan")), dict(alpha=float("-inf"))):
        assert _norm(b, back, **kw) == INV, kw
    for kw in (dict(hidden=516), dict(hidden=16392), dict(chunks=9, tokens=9 * 64), dict(tokens=1 << 31)):
        assert _norm(b, back, **kw) == UNS, kw
    fn = b.library().tpmlp_norm_backward if back else b.library().tpmlp_norm_forward
    assert fn(None, *[None] * (len(BACKWARD if back else FORWARD) + 1)) == INV


@pytest.mark.parametrize("back", [False, True])
def test_norm_pointers(b, back):
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    may_miss = {"dOut"} if back else {"stats", "Xn"}
    for name in BACKWARD if back else FORWARD:
        if name not in may_miss and name not in ("Xq", "Xs"):
            assert _norm(b, back, **{name: None}) == INV, name
        if name in CHUNKED:
            assert _norm(b, back, **{name: arr(OK_PTR, None)}) == INV, name
            assert _norm(b, back, **{name: arr(OK_PTR, BAD_PTR)}) == UNS, name
        else:
            assert _norm(b, back, **{name: bad_of(name)}) == UNS, name
    # what a kind does not have must not be there
    rest = ("dpost_gamma", "dpost_beta", "dpre_gamma", "dpre_beta") if back else ("pre_beta",)
    for kw in ([dict(post="none", post_gamma=OK_PTR), dict(post="rms", post_beta=OK_PTR),
                dict(pre="none", pre_gamma=OK_PTR), dict(gate_rows=0, gate=OK_PTR)]
               + [dict(post="none", pre="none", **{k: OK_PTR}) for k in rest]):
        assert _norm(b, back, **kw) == INV, kw
    if back:
        assert _norm(b, back, gate_rows=0, dgate=OK_PTR) == INV
        assert _norm(b, back, pre="none", dXn=arr(OK_PTR, OK_PTR)) == INV
        assert _norm(b, back, pre="none", dOut=None) == INV       # no gradient at all
    else:
        assert _norm(b, back, Xq=None) == INV and _norm(b, back, Xs=None) == INV
        assert _norm(b, back, Xn=None, Xq=None, Xs=None) == INV   # a norm before and nowhere to put it
        assert _norm(b, back, pre="none", Xn=arr(OK_PTR, OK_PTR)) == INV
        assert _norm(b, back, fmt=2) == INV
        assert _norm(b, back, hidden=520) == UNS                  # 8-bit rows: multiples of 16
    # without Z there is the norm before alone
    for kw in (dict(), dict(post="none"), dict(post="none", gate_rows=0, pre="none")):
        assert _norm(b, back, Z=None, **kw) == INV, kw


def test_norm_workspace(b):
    size = b.tpmlp_norm_workspace_bytes
    assert size(b.make_norm_params(256, 512, 1, 1, 0, 1, 0, 1e-5, 1.0)) > 0
    assert size(b.make_norm_params(0, 512, 1, 1, 0, 1, 0, 1e-5, 1.0)) > 0
    assert size(b.make_norm_params(256, 516, 1, 1, 0, 1, 0, 1e-5, 1.0)) == 0
    assert b.library().tpmlp_norm_workspace_bytes(None) == 0


# ---- the layers in Python --------------------------------------------------------------------

def test_python_layers_refuse_the_cpu(b):
    from tensor_transformer_mlp_gemm_gb300 import fp8
    from tensor_transformer_mlp_gemm_gb300.norm import DeviceNormResidual
    x = torch.zeros(128, 256, dtype=torch.bfloat16)
    for call in (lambda: fp8.quantize_tokens(x), lambda: fp8.quantize_shards([x]),
                 lambda: fp8.quantize_weight(x), lambda: fp8.quantize_tokens(x, "e3m4"),
                 lambda: fp8.quantize_tokens([]), lambda: fp8.quantize_shards([x] * 9),
                 lambda: DeviceNormResidual(16, 64, "l2"), lambda: DeviceNormResidual(16, 20, "none", "none"),
                 lambda: DeviceNormResidual(16, 64, "none", "none", device="cpu"),
                 lambda: DeviceNormResidual(16, 24, quantize="e4m3", pre_gamma=x[0, :24], post_gamma=x[0, :24]),
                 lambda: DeviceNormResidual(16, 64, gate_rows=5)):
        with pytest.raises(ValueError):
            call()
    w = custom_linear(16, 256, 128, 1, "column")
    q, s = torch.zeros(256, 128, dtype=torch.float8_e4m3fn), torch.zeros(2, 1)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.DeviceFp8Linear(w, [q], [s], torch.zeros(128, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="unsupported"):
        fp8.DeviceFp8Linear(custom_linear(16, 256, 136, 1, "column"), [q], [s], x[0])

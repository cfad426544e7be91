"""What the 4-bit calls and the gradient calls refuse, without a GPU: the checks come before
the device is looked at, so pointers that are never followed stand in for the tensors."""
import ctypes
import math

import pytest

from test_fp8_norm_refusals_cpu import BAD_PTR, OK_PTR, arr, b  # noqa: F401  (b: the fixture)

BAD_SCALE = OK_PTR + 2


def bad_of(name):
    return BAD_SCALE if "scale" in name else BAD_PTR


# ---- quantisation -------------------------------------------------------------------------

def _quantize(lib, rows=256, cols=128, parts=1, gather=0, fmt=1, row=True, col=False, **bad):
    d = lib.make_fp4_quant(rows, cols, parts, gather, fmt)
    a = {k: arr(*([OK_PTR] * max(parts, 1))) for k in ("src", "q", "s", "qc", "sc")}
    a["scale"] = OK_PTR if fmt == 1 else None
    a.update(bad)
    return lib.library().tpmlp_fp4_quantize(
        ctypes.byref(d), a["src"], a["scale"], a["q"] if row else None, a["s"] if row else None,
        a["qc"] if col else None, a["sc"] if col else None, None)


def test_quantize(b):  # noqa: F811
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    assert b.library().tpmlp_fp4_quantize(None, None, None, None, None, None, None, None) == INV
    assert _quantize(b, rows=-1) == INV and _quantize(b, cols=0) == INV and _quantize(b, parts=0) == INV
    assert _quantize(b, fmt=2) == INV and _quantize(b, fmt=-1) == INV
    assert _quantize(b, row=False) == INV                 # neither grouping
    assert _quantize(b, scale=None) == INV                # nv has a scale
    assert _quantize(b, fmt=0, scale=OK_PTR) == INV       # mx has none
    assert _quantize(b, scale=BAD_SCALE) == UNS
    assert _quantize(b, cols=144) == UNS                  # not a multiple of 32
    assert _quantize(b, parts=9) == UNS
    assert _quantize(b, rows=1 << 31) == UNS and _quantize(b, cols=1 << 31) == UNS
    assert _quantize(b, rows=192, parts=2, gather=1) == UNS                # chunks of 192
    assert _quantize(b, rows=1 << 30, parts=2, gather=1) == UNS            # 2^31 rows together
    for name in ("src", "q", "s"):
        assert _quantize(b, **{name: arr(None)}) == INV and _quantize(b, **{name: arr(BAD_PTR)}) == UNS
        assert _quantize(b, **{name: None}) == INV
    for name in ("qc", "sc"):
        assert _quantize(b, col=True, **{name: arr(None)}) == INV
        assert _quantize(b, col=True, **{name: arr(BAD_PTR)}) == UNS
        assert _quantize(b, col=True, **{name: None}) == INV


def test_tensor_scale(b):  # noqa: F811
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    call = b.library().tpmlp_fp4_tensor_scale
    d = b.make_fp4_quant(256, 128, 1, 0, 1)
    assert call(None, arr(OK_PTR), OK_PTR, None) == INV
    assert call(ctypes.byref(b.make_fp4_quant(256, 128, 1, 0, 0)), arr(OK_PTR), OK_PTR, None) == INV
    assert call(ctypes.byref(b.make_fp4_quant(256, 100, 1, 0, 1)), arr(OK_PTR), OK_PTR, None) == UNS
    assert call(ctypes.byref(d), None, OK_PTR, None) == INV
    assert call(ctypes.byref(d), arr(BAD_PTR), OK_PTR, None) == UNS
    assert call(ctypes.byref(d), arr(OK_PTR), None, None) == INV
    assert call(ctypes.byref(d), arr(OK_PTR), BAD_SCALE, None) == UNS


def test_dequantize(b):  # noqa: F811
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    call = b.library().tpmlp_fp4_dequantize
    p = OK_PTR
    assert call(-1, 64, 0, p, p, None, p, None) == INV and call(4, -1, 0, p, p, None, p, None) == INV
    assert call(4, 64, 2, p, p, None, p, None) == INV
    assert call(4, 64, 0, p, p, p, p, None) == INV and call(4, 64, 1, p, p, None, p, None) == INV
    assert call(1 << 31, 64, 0, p, p, None, p, None) == UNS
    for i in (0, 1, 3):
        for bad, want in ((None, INV), (BAD_PTR, UNS)):
            a = [p, p, p, p]
            a[i] = bad
            assert call(4, 64, 1, a[0], a[1], a[2], a[3], None) == want


def test_sizes(b):  # noqa: F811
    assert b.tpmlp_fp4_packed_bytes(3, 33) == 3 * 32 and b.tpmlp_fp4_packed_bytes(0, 64) == 0
    assert b.tpmlp_fp4_scale_bytes(1, 1, 0) == 1024 and b.tpmlp_fp4_scale_bytes(129, 257, 1) == 4 * 2048
    assert b.tpmlp_fp4_scale_bytes(1, 1, 2) == 0 and b.tpmlp_fp4_packed_bytes(-1, 2) == 0


# ---- the linear layers ---------------------------------------------------------------------

def _linear(lib, split, back, dims=None, fmt=1, save=False, **bad):
    """A call with valid stand-ins but for `bad` (argument name -> value)."""
    d = dims or lib.make_linear_dims(256, 256, 512, 2, 2)
    t, n, col = max(d.t, 1), max(d.seq_chunks, 1), split == "column"
    many = lambda k: arr(*([OK_PTR] * k))  # noqa: E731
    kept = OK_PTR if col else many(t)
    g = OK_PTR if fmt == 1 else None
    a = {"X": many(n if col else t), "x_scale": g, "calibrated": 0, "Xq": kept if back or save else None,
         "Xs": kept if back or save else None, "Wq": many(t), "Ws": many(t), "w_scale": g, "b": OK_PTR,
         "Y": many(t if col else n), "dY": many(t if col else n), "dX": many(n if col else t),
         "dW": many(t), "db": OK_PTR, "ws": OK_PTR}
    a.update(bad)
    names = (("dY", "Xq", "Xs", "x_scale", "Wq", "Ws", "w_scale", "dX", "dW", "db", "ws") if back
             else ("X", "x_scale", "calibrated", "Xq", "Xs", "Wq", "Ws", "w_scale", "b", "Y", "ws"))
    fn = getattr(lib.library(), f"tpmlp_fp4_{split}_linear_{'backward' if back else 'forward'}")
    return fn(ctypes.byref(d), fmt, *[a[k] for k in names], None)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("split", ["column", "row"])
def test_linear(b, split, back):  # noqa: F811
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    mk = b.make_linear_dims
    col = split == "column"
    call = lambda **kw: _linear(b, split, back, **kw)  # noqa: E731
    for dims in (mk(-1, 256, 512, 2), mk(256, 0, 512, 2), mk(256, 256, -512, 2), mk(256, 256, 512, 0),
                 mk(256, 256, 512, 2, 0), mk(257, 256, 512, 2, 2)):
        assert call(dims=dims) == INV
    assert call(dims=mk(256, 250, 250, 3)) == INV                        # t does not divide the shards
    most = 2 ** 31 - 256
    for dims in (mk(256, 2304, 2304, 9), mk(128 * 9, 256, 512, 2, 9),    # more than 8
                 mk(256, 272, 272, 1), mk(256, 288, 288, 2),             # 32 does not divide
                 mk(192 * 2, 256, 512, 2, 2),                            # chunks of 192
                 mk(1 << 31, 256, 512, 2), mk(most + 1, 256, 512, 2), mk(256, most + 32, 512, 2)):
        assert call(dims=dims) == UNS
    assert call(fmt=2) == INV and call(fmt=-1) == INV
    lists = ["Wq", "Ws"] + (["dY", "dX", "dW"] if back else ["Y", "X"])
    if not col:
        lists += ["Xq", "Xs"]
    for name in lists:
        kw = {"save": True} if name in ("Xq", "Xs") else {}
        assert call(**kw, **{name: None}) == INV
        assert call(**kw, **{name: arr(OK_PTR, None)}) == INV
        assert call(**kw, **{name: arr(OK_PTR, BAD_PTR)}) == UNS
    for name in (["db", "ws"] if back else ["b", "ws"]) + ["x_scale", "w_scale"]:
        assert call(**{name: None}) == INV
        assert call(**{name: bad_of(name)}) == UNS
        if "scale" in name:
            assert call(fmt=0, **{name: OK_PTR}) == INV
    if col:
        for name in ("Xq", "Xs"):
            assert call(save=True, **{name: None}) == INV
            assert call(save=True, **{name: BAD_PTR}) == UNS


@pytest.mark.parametrize("which", range(3))
def test_largest_sizes(b, which):  # noqa: F811
    most = 2 ** 31 - 256
    size = b.tpmlp_fp4_linear_workspace_bytes
    for n, fits in ((most, True), (most + (1 if which == 0 else 32), False)):
        d = [32, 32, 32]
        d[which] = n
        for fmt in (0, 1):
            for back in (False, True):
                assert (size(b.make_linear_dims(*d, 1), fmt, back) > 0) == fits


def test_linear_workspace(b):  # noqa: F811
    mk, size = b.make_linear_dims, b.tpmlp_fp4_linear_workspace_bytes
    assert size(mk(256, 272, 272, 1), 0, True) == 0 and size(mk(256, 256, 256, 1), 2, True) == 0
    assert size(mk(2048, 4096, 4096, 8), 0, False) >= 2048 * 4096 * (0.5 + 1 / 32)
    assert size(mk(2048, 4096, 4096, 8), 1, True) >= 2 * 2048 * 4096 * (0.5 + 1 / 16)
    assert size(mk(0, 256, 512, 2), 0, True) > 0
    assert b.library().tpmlp_fp4_linear_workspace_bytes(None, 0, 1) == 0


# ---- gradients ------------------------------------------------------------------------------

def test_gradients(b):  # noqa: F811
    import torch
    INV, UNS = b.TPMLP_ERR_INVALID_ARG, b.TPMLP_ERR_UNSUPPORTED
    lib = b.library()

    def call(clip, tensors, n=None, max_norm=1.0, norm=OK_PTR, ws=OK_PTR):
        t = None if tensors is None else b.make_grad_tensors(tensors)
        n = len(tensors) if n is None else n
        return (lib.tpmlp_grad_clip(t, n, max_norm, norm, ws, None) if clip
                else lib.tpmlp_grad_norm(t, n, norm, ws, None))

    p = OK_PTR
    for clip in (False, True):
        assert call(clip, None, 1) == INV and call(clip, [(p, p, 4, 0)], -1) == INV
        assert call(clip, [(p, p, -1, 0)]) == INV
        assert call(clip, [(p, p, 4, 3)]) == INV and call(clip, [(p, p, 4, -1)]) == INV
        assert call(clip, [(None, p, 4, 0)]) == INV
        assert call(clip, [(p + 2, p, 4, 0)]) == UNS and call(clip, [(p + 1, p, 4, 1)]) == UNS
        assert call(clip, [(p, p, (1 << 40) + 1, 0)]) == UNS
        assert call(clip, [(p, p, 4, 0)], norm=None) == INV and call(clip, [(p, p, 4, 0)], norm=p + 2) == UNS
        assert call(clip, [(p, p, 4, 0)], ws=None) == INV and call(clip, [(p, p, 4, 0)], ws=p + 8) == UNS
        assert call(clip, [(p, p, 0, 0)], n=1 << 17) == UNS
    assert call(True, [(p, None, 4, 0)]) == INV and call(True, [(p, p + 2, 4, 0)]) == UNS
    for bad in (-1.0, math.nan, math.inf, -math.inf):
        assert call(True, [(p, p, 4, 0)], max_norm=bad) == INV
    size = b.tpmlp_grad_workspace_bytes
    assert size(1) > 0 and size(0) > 0 and size(65536) > 0 and size(65537) == 0 and size(-1) == 0
    assert torch.float64 not in b.GRAD_TYPES

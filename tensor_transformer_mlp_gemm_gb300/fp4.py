"""4-bit floating point quantisation (mxfp4, nvfp4) and device buffers for one
tensor-parallel linear layer on 4-bit operands.

PyTorch is used for device memory and streams only; every step runs in libtpmlp
through :mod:`binding`.  A 4-bit value is a sign, two exponent bits and one mantissa
bit; groups along the axis that a product sums over share a scale (include/tpmlp.h):
  mxfp4  groups of 32, scales powers of two
  nvfp4  groups of 16, scales e4m3, and a power of two for the whole tensor, shared by
         its shards
"""
from __future__ import annotations

import ctypes

import torch

from . import binding
from .fp8 import _ARRAYS, _check_like, _check_parts, _pointers, _strided, _up256
from .inputs import LinearWorkload


def _format(name: str) -> int:
    if name not in binding.FP4_FORMATS:
        raise ValueError(f"format must be one of {sorted(binding.FP4_FORMATS)}, got {name!r}")
    return binding.FP4_FORMATS[name]


def _check_scale(scale, fmt: str, device, what: str) -> None:
    if fmt == "mxfp4":
        if scale is not None:
            raise ValueError(f"mxfp4 has no scale for a tensor: {what} must be None")
    elif scale is not None:
        _check_like(scale, (1,), torch.float32, device, what)


class Fp4Matrix:
    """A matrix [rows, k] in 4 bits, summed over k: ``q`` uint8 [rows, ceil(k/32) * 16], two
    values a byte; ``s`` uint8, the scales as the tensor cores take them; ``scale`` fp32 [1]
    (nvfp4) or None; ``fmt``."""

    def __init__(self, q: torch.Tensor, s: torch.Tensor, scale: torch.Tensor | None, shape: tuple,
                 fmt: str):
        code = _format(fmt)
        rows, k = shape
        _check_like(q, (rows, -(-k // 32) * 16), torch.uint8, q.device, "q")
        _check_like(s, (binding.tpmlp_fp4_scale_bytes(rows, k, code),), torch.uint8, q.device, "s")
        _check_scale(scale, fmt, q.device, "scale")
        if fmt == "nvfp4" and scale is None:
            raise ValueError("nvfp4 needs the tensor's scale")
        self.q, self.s, self.scale, self.shape, self.fmt = q, s, scale, (rows, k), fmt

    @property
    def device(self):
        return self.q.device

    def values(self, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The values that it stands for, bf16 [rows, k] (exact)."""
        dev = self.q.device
        if out is None:
            with binding.allocate_on(dev, stream):
                out = torch.empty(self.shape, dtype=torch.bfloat16, device=dev)
        else:
            _check_like(out, self.shape, torch.bfloat16, dev, "out")
        with binding.on_device(dev):
            binding.tpmlp_fp4_dequantize(*self.shape, binding.FP4_FORMATS[self.fmt], self.q, self.s,
                                         self.scale, out, binding.stream_on(dev, stream))
        return out


class Fp4Tokens:
    """One matrix of activations in 4 bits: by rows [T, C], by columns [C, T], or both (None
    where it is not there)."""

    def __init__(self, rows: Fp4Matrix | None = None, cols: Fp4Matrix | None = None):
        self.rows, self.cols = rows, cols


class Fp4Weights:
    """The shards of one weight in 4 bits: ``forward`` [out_i, in_i] grouped along the inputs,
    ``backward`` [in_i, out_i] grouped along the outputs, or None; their ``scale``."""

    def __init__(self, forward: list, backward: list | None):
        self.forward, self.backward = list(forward), None if backward is None else list(backward)
        both = self.forward + (self.backward or [])
        if not both:
            raise ValueError("no shards")
        self.fmt, self.scale = both[0].fmt, both[0].scale
        if self.backward is not None and len(self.backward) != len(self.forward):
            raise ValueError("as many shards are needed forward and backward")
        for m in both:
            # one scale for all: the shards of a row-parallel layer are summed before it is applied
            if m.fmt != self.fmt or m.device != both[0].device or (
                    m.scale is not None and m.scale.data_ptr() != self.scale.data_ptr()):
                raise ValueError("the shards of a weight have one format, device and scale")


class _Space:
    """Room for n matrices [R, K] in 4 bits and their scales, in one buffer."""

    def __init__(self, n: int, R: int, K: int, fmt: str, device, stream=None):
        code = binding.FP4_FORMATS[fmt]
        self.n, self.shape, self.fmt = n, (R, K), fmt
        self.q = binding.tpmlp_fp4_packed_bytes(R, K)
        self.s = binding.tpmlp_fp4_scale_bytes(R, K, code)
        self.at = _up256(n * self.q)
        with binding.allocate_on(device, stream):
            self.buf = torch.empty(max(self.at + n * self.s, 256), dtype=torch.uint8, device=device)
        base = self.buf.data_ptr()
        self.q_ptrs, self.s_ptrs = _strided(base, self.q, n), _strided(base + self.at, self.s, n)

    def matrix(self, i: int, scale) -> Fp4Matrix:
        R, K = self.shape
        q = self.buf[i * self.q:(i + 1) * self.q].view(R, -(-K // 32) * 16)
        s = self.buf[self.at + i * self.s:self.at + (i + 1) * self.s]
        m = Fp4Matrix.__new__(Fp4Matrix)
        m.q, m.s, m.scale, m.shape, m.fmt = q, s, scale, self.shape, self.fmt
        return m


def tensor_scale(parts, stream=None) -> torch.Tensor:
    """The scale (fp32 [1]) of the nvfp4 tensor whose bf16 parts these are, of one shape."""
    parts = [parts] if isinstance(parts, torch.Tensor) else list(parts)
    _check_parts(parts, "part")
    dev = parts[0].device
    with binding.allocate_on(dev, stream):
        scale = torch.empty(1, dtype=torch.float32, device=dev)
    with binding.on_device(dev):
        binding.tpmlp_fp4_tensor_scale(binding.make_fp4_quant(*parts[0].shape, len(parts), False, 1),
                                       _pointers(parts), scale, binding.stream_on(dev, stream))
    return scale


def _quantize(parts, fmt: str, gather: bool, rows: bool, cols: bool, scale, stream):
    """(space by rows or None, space by columns or None, the scale used)."""
    code, dev, n = _format(fmt), parts[0].device, len(parts)
    if not (rows or cols):
        raise ValueError("choose rows, cols or both")
    _check_scale(scale, fmt, dev, "scale")
    if fmt == "nvfp4" and scale is None:
        scale = tensor_scale(parts, stream)
    R, C = parts[0].shape
    outs, T = (1, R * n) if gather else (n, R)
    by_rows = _Space(outs, T, C, fmt, dev, stream) if rows else None
    by_cols = _Space(outs, C, T, fmt, dev, stream) if cols else None
    with binding.on_device(dev):
        binding.tpmlp_fp4_quantize(
            binding.make_fp4_quant(R, C, n, gather, code), _pointers(parts), scale,
            by_rows and by_rows.q_ptrs, by_rows and by_rows.s_ptrs, by_cols and by_cols.q_ptrs,
            by_cols and by_cols.s_ptrs, binding.stream_on(dev, stream))
    return by_rows, by_cols, scale


def quantize_tokens(X, fmt: str = "mxfp4", rows: bool = True, cols: bool = False,
                    scale: torch.Tensor | None = None, stream=None) -> Fp4Tokens:
    """X: a bf16 tensor [T, C], or the list of its token chunks (multiples of 128 tokens),
    which are gathered on the way.  rows and cols choose the groupings (one read makes both);
    scale (nvfp4): the tensor's, or None to compute it first."""
    chunks = [X] if isinstance(X, torch.Tensor) else list(X)
    _check_parts(chunks, "token chunk")
    if len(chunks) > 1 and chunks[0].shape[0] % 128:
        raise ValueError("token chunks must be a multiple of 128 tokens")
    r, c, scale = _quantize(chunks, fmt, True, rows, cols, scale, stream)
    return Fp4Tokens(r and r.matrix(0, scale), c and c.matrix(0, scale))


def quantize_weight(W, fmt: str = "mxfp4", backward: bool = False, scale: torch.Tensor | None = None,
                    stream=None) -> Fp4Weights:
    """W: the bf16 shards [in_i, out_i] of one weight (a tensor: one shard).  backward: make
    the form for the backward pass too, in the same read."""
    shards = [W] if isinstance(W, torch.Tensor) else list(W)
    _check_parts(shards, "weight shard")
    r, c, scale = _quantize(shards, fmt, False, backward, True, scale, stream)
    return Fp4Weights([c.matrix(i, scale) for i in range(len(shards))],
                      [r.matrix(i, scale) for i in range(len(shards))] if backward else None)


class DeviceFp4Linear:
    """One linear layer on 4-bit weight shards (``quantize_weight``): the 4-bit counterpart of
    ``linear.DeviceLinear`` for the same workloads.  It takes bf16 activations and gradients
    and quantises them on the way.

    x_scale (nvfp4): the activations' scale from a calibration, fp32 [1]; None computes it
    from each input.  The backward pass needs weights with both forms."""

    def __init__(self, w: LinearWorkload, weights: Fp4Weights, b: torch.Tensor,
                 x_scale: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
        if w.split not in ("column", "row"):
            raise ValueError("split must be 'column' or 'row'")
        self.w, self._weights, self.fmt = w, weights, weights.fmt
        self.column = w.split == "column"
        self._code = _format(self.fmt)
        T, din, dout, t, n = w.tokens, w.in_features, w.out_features, w.t, w.seq_chunks
        self.dims = binding.make_linear_dims(T, din, dout, t, n)
        need = binding.tpmlp_fp4_linear_workspace_bytes(self.dims, self._code, weights.backward is not None)
        if need == 0:
            raise ValueError(f"unsupported dims for a 4-bit linear layer: {w}")
        if not b.is_cuda:
            raise ValueError(f"the layer's tensors must be CUDA tensors, got b on {b.device}")
        self.device = dev = b.device
        _check_like(b, (dout,), torch.bfloat16, dev, "b")
        s = w.shard
        wshape = (din, s) if self.column else (s, dout)
        if len(weights.forward) != t:
            raise ValueError(f"{t} weight shards are needed, got {len(weights.forward)}")
        for m, shape in ([(m, wshape[::-1]) for m in weights.forward]
                         + [(m, wshape) for m in weights.backward or []]):
            if m.shape != shape or m.device != dev:
                raise ValueError(f"a 4-bit weight shard of shape {shape} on {dev} is needed, got "
                                 f"{m.shape} on {m.device}")
        self._bias = b
        self.x_scale = x_scale
        bf = torch.bfloat16
        # the shapes of X_i, Y_i (or Z) and their gradients, and how many of each
        self._x = ((T // n, din), n) if self.column else ((T, s), t)
        self._y = ((T, s), t) if self.column else ((T // n, dout), n)
        self.Y = [torch.empty(self._y[0], dtype=bf, device=dev) for _ in range(self._y[1])]
        self._dX = self._dx_ptrs = self._grads = self._saved = None
        self._has_saved, self._saved_scale = False, None
        if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()
                                      or workspace.numel() * workspace.element_size() < need):
            raise ValueError(f"the workspace needs {need} contiguous bytes on {dev}")
        self.ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8,
                                                                      device=dev)
        # (what stays the same in every call is marshalled once, and kept)
        split = "column" if self.column else "row"
        self._call = binding.prepared(f"tpmlp_fp4_{split}_linear_forward")
        self._call_back = binding.prepared(f"tpmlp_fp4_{split}_linear_backward")
        self._dims = ctypes.byref(self.dims)
        self._b = b.data_ptr()
        self._w_scale = None if weights.scale is None else weights.scale.data_ptr()
        self._forward = (_pointers([m.q for m in weights.forward]), _pointers([m.s for m in weights.forward]))
        self._backward = weights.backward and (_pointers([m.q for m in weights.backward]),
                                               _pointers([m.s for m in weights.backward]))
        # where a forward call without a calibration writes the scale: one that keeps nothing, and
        # one that keeps X for the backward pass
        self._scales = torch.empty(2, 1, dtype=torch.float32, device=dev) if self.fmt == "nvfp4" else None

    weights = property(lambda self: self._weights)
    b = property(lambda self: self._bias)

    @property
    def x_scale(self):
        return self._x_scale

    @x_scale.setter
    def x_scale(self, scale):
        _check_scale(scale, self.fmt, self.device, "x_scale")
        self._x_scale = scale

    @property
    def Y(self):
        return list(self._Y)

    @Y.setter
    def Y(self, xs):
        self._Y = tuple(self._list(xs, self._y, "Y"))
        self._y_ptrs = _pointers(self._Y)

    # Gradients are made by the first backward call, so that a layer that only goes forward
    # does not hold them.
    def _input_grads(self, stream=None):
        if self._dX is None:
            with binding.allocate_on(self.device, stream):
                self.dX = [torch.empty(self._x[0], dtype=torch.bfloat16, device=self.device)
                           for _ in range(self._x[1])]
        return self._dx_ptrs

    @property
    def dX(self):
        self._input_grads()
        return list(self._dX)

    @dX.setter
    def dX(self, xs):
        self._dX = tuple(self._list(xs, self._x, "dX"))
        self._dx_ptrs = _pointers(self._dX)

    def _weight_grads(self, stream=None):
        if self._grads is None:
            s = self.w.shard
            shape = (self.w.in_features, s) if self.column else (s, self.w.out_features)
            with binding.allocate_on(self.device, stream):
                dW = [torch.empty(shape, dtype=torch.float32, device=self.device) for _ in range(self.w.t)]
                db = torch.empty(self.w.out_features, dtype=torch.float32, device=self.device)
            self._grads = (dW, db, _pointers(dW))
        return self._grads

    @property
    def dW(self):
        return list(self._weight_grads()[0])

    @property
    def db(self):
        return self._weight_grads()[1]

    def _save(self, stream):
        """Room for X by columns, kept by the layer from its first saving call on."""
        if self._saved is None:
            n, C = (1, self.w.in_features) if self.column else (self.w.t, self.w.shard)
            self._saved = _Space(n, C, self.w.tokens, self.fmt, self.device, stream)
        return self._saved

    def _list(self, xs, spec, what):
        xs = [xs] if isinstance(xs, torch.Tensor) else list(xs)
        if len(xs) != spec[1]:
            raise ValueError(f"{what}: {spec[1]} tensors are needed, got {len(xs)}")
        for x in xs:
            _check_like(x, spec[0], torch.bfloat16, self.device, what)
        return xs

    def _ptrs(self, xs, spec, what):
        """Pointers of the bf16 tensors xs, which are looked over."""
        if isinstance(xs, torch.Tensor):
            xs = (xs,)
        shape, n = spec
        dev, bf = self.device, torch.bfloat16
        if len(xs) != n:
            self._list(xs, spec, what)
        got = []
        for x in xs:
            if x.dtype is not bf or x.shape != shape or not x.is_contiguous() or x.device != dev:
                self._list(xs, spec, what)
            got.append(x.data_ptr())
        return _ARRAYS[n](*got)

    def forward(self, X, save: bool = False, Y=None, stream=None) -> None:
        """X: bf16 (column: its token chunks, row: t shards).  save: keep X in 4 bits for the
        next backward call."""
        X = self._ptrs(X, self._x, "X")
        Y = self._y_ptrs if Y is None else self._ptrs(Y, self._y, "Y")
        q = s = scale = None
        if save:
            if self._backward is None:
                raise ValueError("the weights have no form for the backward pass")
            kept = self._save(stream)
            q, s = (kept.q_ptrs[0], kept.s_ptrs[0]) if self.column else (kept.q_ptrs, kept.s_ptrs)
        calibrated = self._x_scale is not None
        if calibrated:
            scale = self._x_scale.data_ptr()
        elif self._scales is not None:
            scale = self._scales[int(save)].data_ptr()
        dev = self.device
        with binding.on_device(dev):
            self._call(self._dims, self._code, X, scale, calibrated, q, s, *self._forward, self._w_scale,
                       self._b, Y, self.ws.data_ptr(), binding.stream_on(dev, stream))
        if save:
            # (of a calibration the tensor, in case another one is set before the backward call)
            self._saved_scale = (self._x_scale if calibrated else None, scale)
            self._has_saved = True

    def backward(self, dY, dX=None, stream=None) -> None:
        """dY: bf16 (column: t shards, row: token chunks), for the X that the last forward call
        with save=True kept."""
        if self._backward is None:
            raise ValueError("the weights have no form for the backward pass")
        if not self._has_saved:
            raise ValueError("there is no forward call with save=True to go back through")
        dY = self._ptrs(dY, self._y, "dY")
        dX = self._input_grads(stream) if dX is None else self._ptrs(dX, self._x, "dX")
        _, db, dW = self._weight_grads(stream)
        kept = self._saved
        q, s = (kept.q_ptrs[0], kept.s_ptrs[0]) if self.column else (kept.q_ptrs, kept.s_ptrs)
        dev = self.device
        with binding.on_device(dev):
            self._call_back(self._dims, self._code, dY, q, s, self._saved_scale[1], *self._backward,
                            self._w_scale, dX, dW, db.data_ptr(), self.ws.data_ptr(),
                            binding.stream_on(dev, stream))

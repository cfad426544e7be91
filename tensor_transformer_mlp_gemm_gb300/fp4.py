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
import functools

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


def _ld(k: int) -> int:
    """Bytes of a row of k values."""
    return -(-k // 32) * 16


def _scale_bytes(rows: int, k: int, code: int) -> int:
    return -(-rows // 128) * -(-k // 256) * (2048 if code else 1024)


class Fp4Matrix:
    """A matrix [rows, k] in 4 bits, summed over k: ``q`` uint8 [rows, ceil(k/32) * 16], two
    values a byte; ``s`` uint8, the scales as the tensor cores take them; ``scale`` fp32 [1]
    (nvfp4) or None; ``fmt``."""

    def __init__(self, q: torch.Tensor, s: torch.Tensor, scale: torch.Tensor | None, shape: tuple,
                 fmt: str):
        code = _format(fmt)
        rows, k = shape
        if not q.is_cuda:
            raise ValueError(f"q must be a CUDA tensor, got one on {q.device}")
        _check_like(q, (rows, _ld(k)), torch.uint8, q.device, "q")
        _check_like(s, (_scale_bytes(rows, k, code),), torch.uint8, q.device, "s")
        _check_scale(scale, fmt, q.device, "scale")
        if fmt == "nvfp4" and scale is None:
            raise ValueError("nvfp4 needs the tensor's scale")
        self._q, self._s, self._scale = q, s, scale
        self._ptrs = (q.data_ptr(), s.data_ptr(), None if scale is None else scale.data_ptr())
        self.shape, self.fmt, self.device = (rows, k), fmt, q.device

    @classmethod
    def _of(cls, space: "_Space", i: int, scale) -> "Fp4Matrix":
        """Matrix i of a space, whose tensors are made when asked for."""
        m = cls.__new__(cls)
        m._q = m._s = None
        m._scale, m._space, m._i = scale, space, i
        m._ptrs = (space.q_ptrs[i], space.s_ptrs[i], space.scale_ptr)
        m.shape, m.fmt, m.device = space.shape, space.fmt, space.device
        return m

    @property
    def q(self) -> torch.Tensor:
        if self._q is None:
            self._q = self._space.bytes(self._ptrs[0], self._space.q).view(self.shape[0], _ld(self.shape[1]))
        return self._q

    @property
    def s(self) -> torch.Tensor:
        if self._s is None:
            self._s = self._space.bytes(self._ptrs[1], self._space.s)
        return self._s

    @property
    def scale(self) -> torch.Tensor | None:
        if self._scale is None and self.fmt == "nvfp4":
            self._scale = self._space.bytes(self._ptrs[2], 4).view(torch.float32)
        return self._scale

    def values(self, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
        """The values that it stands for, bf16 [rows, k] (exact)."""
        dev = self.device
        if out is None:
            with binding.allocate_on(dev, stream):
                out = torch.empty(self.shape, dtype=torch.bfloat16, device=dev)
        else:
            _check_like(out, self.shape, torch.bfloat16, dev, "out")
        with binding.on_device(dev):
            _dequantize(*self.shape, binding.FP4_FORMATS[self.fmt], *self._ptrs, out.data_ptr(),
                        binding.stream_on(dev, stream))
        return out


class Fp4Tokens:
    """One matrix of activations in 4 bits: by rows [T, C], by columns [C, T], or both (None
    where it is not there)."""

    def __init__(self, rows: Fp4Matrix | None = None, cols: Fp4Matrix | None = None):
        self.rows, self.cols = rows, cols


class Fp4Weights:
    """The shards of one weight in 4 bits: ``forward`` [out_i, in_i] grouped along the inputs,
    ``backward`` [in_i, out_i] grouped along the outputs, or None; their ``scale``.  They stay the
    same: a layer holds their addresses."""

    def __init__(self, forward: list, backward: list | None):
        self._forward, self._backward = tuple(forward), None if backward is None else tuple(backward)
        both = self._forward + (self._backward or ())
        if not both:
            raise ValueError("no shards")
        first = both[0]
        self.fmt = first.fmt
        if self._backward is not None and len(self._backward) != len(self._forward):
            raise ValueError("as many shards are needed forward and backward")
        for m in both:
            # one scale for all: the shards of a row-parallel layer are summed before it is applied
            if m.fmt != first.fmt or m.device != first.device or m._ptrs[2] != first._ptrs[2]:
                raise ValueError("the shards of a weight have one format, device and scale")

    forward = property(lambda self: self._forward)
    backward = property(lambda self: self._backward)
    scale = property(lambda self: self._forward[0].scale)


class _Space:
    """Room for n matrices [R, K] in 4 bits and their scales in a buffer, from byte `at` on."""

    def __init__(self, n: int, R: int, K: int, fmt: str):
        self.n, self.shape, self.fmt = n, (R, K), fmt
        self.q, self.s = R * _ld(K), _scale_bytes(R, K, binding.FP4_FORMATS[fmt])
        self.size = _up256(n * self.q) + _up256(n * self.s)
        self.scale_ptr = None

    def place(self, buf: torch.Tensor, at: int) -> "_Space":
        self.buf, self.device, self.start = buf, buf.device, buf.data_ptr()
        base = self.start + at
        self.q_ptrs = _strided(base, self.q, self.n)
        self.s_ptrs = _strided(base + _up256(self.n * self.q), self.s, self.n)
        return self

    def bytes(self, ptr: int, size: int) -> torch.Tensor:
        return self.buf[ptr - self.start:ptr - self.start + size]


_dequantize = binding.prepared("tpmlp_fp4_dequantize")
_quantize_call = binding.prepared("tpmlp_fp4_quantize")
_tensor_scale_call = binding.prepared("tpmlp_fp4_tensor_scale")
# (R, C, parts, gather, format) -> a call's description
_quant = functools.lru_cache(maxsize=256)(lambda *a: ctypes.byref(binding.make_fp4_quant(*a)))


def tensor_scale(parts, stream=None) -> torch.Tensor:
    """The scale (fp32 [1]) of the nvfp4 tensor whose bf16 parts these are, of one shape."""
    parts = [parts] if isinstance(parts, torch.Tensor) else list(parts)
    _check_parts(parts, "part")
    dev = parts[0].device
    with binding.allocate_on(dev, stream):
        scale = torch.empty(1, dtype=torch.float32, device=dev)
    with binding.on_device(dev):
        _tensor_scale_call(_quant(*parts[0].shape, len(parts), False, 1), _pointers(parts), scale.data_ptr(),
                           binding.stream_on(dev, stream))
    return scale


def _quantize(parts, fmt: str, gather: bool, rows: bool, cols: bool, scale, stream):
    """(matrices by rows or None, matrices by columns or None), in one buffer with the scale
    where that is computed here (an allocation costs more host time than a launch)."""
    code, dev, n = _format(fmt), parts[0].device, len(parts)
    if not (rows or cols):
        raise ValueError("choose rows, cols or both")
    _check_scale(scale, fmt, dev, "scale")
    R, C = parts[0].shape
    outs, T = (1, R * n) if gather else (n, R)
    spaces = [_Space(outs, *shape, fmt) if wanted else None
              for wanted, shape in ((rows, (T, C)), (cols, (C, T)))]
    at = 256 if fmt == "nvfp4" else 0
    with binding.allocate_on(dev, stream):
        buf = torch.empty(max(at + sum(x.size for x in spaces if x), 256), dtype=torch.uint8, device=dev)
    for x in spaces:
        if x is not None:
            x.place(buf, at)
            at += x.size
    scale_ptr = None
    if fmt == "nvfp4":
        scale_ptr = buf.data_ptr() if scale is None else scale.data_ptr()
    ptrs = _pointers(parts)
    r, c = spaces
    with binding.on_device(dev):
        raw = binding.stream_on(dev, stream)
        if fmt == "nvfp4" and scale is None:
            _tensor_scale_call(_quant(R, C, n, False, 1), ptrs, scale_ptr, raw)
        _quantize_call(_quant(R, C, n, gather, code), ptrs, scale_ptr, r and r.q_ptrs, r and r.s_ptrs,
                       c and c.q_ptrs, c and c.s_ptrs, raw)
    for x in spaces:
        if x is not None:
            x.scale_ptr = scale_ptr
    return tuple(x and [Fp4Matrix._of(x, i, scale) for i in range(outs)] for x in spaces)


def quantize_tokens(X, fmt: str = "mxfp4", rows: bool = True, cols: bool = False,
                    scale: torch.Tensor | None = None, stream=None) -> Fp4Tokens:
    """X: a bf16 tensor [T, C], or the list of its token chunks (multiples of 128 tokens),
    which are gathered on the way.  rows and cols choose the groupings (one read makes both);
    scale (nvfp4): the tensor's, or None to compute it first."""
    chunks = [X] if isinstance(X, torch.Tensor) else list(X)
    _check_parts(chunks, "token chunk")
    if len(chunks) > 1 and chunks[0].shape[0] % 128:
        raise ValueError("token chunks must be a multiple of 128 tokens")
    r, c = _quantize(chunks, fmt, True, rows, cols, scale, stream)
    return Fp4Tokens(r and r[0], c and c[0])


def quantize_weight(W, fmt: str = "mxfp4", backward: bool = False, scale: torch.Tensor | None = None,
                    stream=None) -> Fp4Weights:
    """W: the bf16 shards [in_i, out_i] of one weight (a tensor: one shard).  backward: make
    the form for the backward pass too, in the same read."""
    shards = [W] if isinstance(W, torch.Tensor) else list(W)
    _check_parts(shards, "weight shard")
    r, c = _quantize(shards, fmt, False, backward, True, scale, stream)
    return Fp4Weights(c, r)


class DeviceFp4Linear:
    """One linear layer on 4-bit weight shards (``quantize_weight``): the 4-bit counterpart of
    ``linear.DeviceLinear`` for the same workloads.  It takes bf16 activations and gradients
    and quantises them on the way.

    x_scale (nvfp4): the activations' scale from a calibration, fp32 [1]; None computes it
    from each input.  (One that a saving forward call took keeps its value until the backward
    call.)  The backward pass needs weights with both forms."""

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
                         + [(m, wshape) for m in weights.backward or ()]):
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
        self._w_scale = weights.forward[0]._ptrs[2]
        def pointers(ms):
            return tuple(_ARRAYS[t](*[m._ptrs[k] for m in ms]) for k in (0, 1))
        self._forward = pointers(weights.forward)
        self._backward = weights.backward and pointers(weights.backward)
        # where a forward call without a calibration writes the scale: one that keeps nothing, and
        # one that keeps X for the backward pass
        self._scales = torch.empty(2, 1, dtype=torch.float32, device=dev) if self.fmt == "nvfp4" else None
        self._scale_ptrs = self._scales is not None and tuple(x.data_ptr() for x in self._scales)

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
            space = _Space(n, C, self.w.tokens, self.fmt)
            with binding.allocate_on(self.device, stream):
                buf = torch.empty(max(space.size, 256), dtype=torch.uint8, device=self.device)
            self._saved = space.place(buf, 0)
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
        elif not isinstance(xs, (list, tuple)):
            xs = list(xs)
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
        save = bool(save)
        if save:
            if self._backward is None:
                raise ValueError("the weights have no form for the backward pass")
            kept = self._save(stream)
            q, s = (kept.q_ptrs[0], kept.s_ptrs[0]) if self.column else (kept.q_ptrs, kept.s_ptrs)
        calibrated = self._x_scale is not None
        if calibrated:
            scale = self._x_scale.data_ptr()
        elif self._scale_ptrs:
            scale = self._scale_ptrs[save]
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

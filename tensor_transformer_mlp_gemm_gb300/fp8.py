"""8-bit quantisation with a scale for each group of 128, and device buffers for
one tensor-parallel linear layer on 8-bit operands.

PyTorch is used for device memory and streams only; every step runs in libtpmlp
through :mod:`binding`.  Layouts follow the C ABI (include/tpmlp.h):
  activations  q [T, C] float8; row_scale fp32 [ceil(C/128), T] (groups along
               features, for a product over features); col_scale fp32
               [ceil(T/128), C] (groups along tokens, for the weight gradient)
  weights      q [in, out] float8, scale fp32 [ceil(in/128), ceil(out/128)]
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import binding
from .inputs import LinearWorkload

DTYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _up128(n: int) -> int:
    return -(-n // 128)


def _up256(n: int) -> int:
    return -(-n // 256) * 256


class _Packed:
    """n matrices [T, C] in 8 bits with their scales, side by side in one buffer (an
    allocation costs more host time than a launch)."""

    def __init__(self, n: int, T: int, C: int, fmt: str, rows: bool, cols: bool, device,
                 stream=None):
        self.n, self.T, self.C, self.fmt, self.device = n, T, C, fmt, device
        self.q = T * C                                       # bytes of one matrix
        # of its scales; every matrix's start on 16 bytes
        self.steps = (-(-_up128(C) * T // 4) * 16, _up128(T) * C * 4)
        # where each part starts: q and scales by rows, then by columns (None: not made)
        at, self.at = 0, [None, None, None, None]
        for k, (wanted, size) in enumerate(((rows, self.q), (rows, self.steps[0]),
                                            (cols, self.q), (cols, self.steps[1]))):
            if wanted:
                self.at[k] = at
                at += _up256(n * size)
        with binding.allocate_on(device, stream):
            self.buf = torch.empty(max(at, 256), dtype=torch.uint8, device=device)
        self.base = self.buf.data_ptr()
        self._typed = [None, None]                           # the buffer as 8-bit values, as fp32

    def pointers(self, cols: bool):
        """(q, scale) pointer arrays by rows or by columns."""
        return (_strided(self.base + self.at[2 * cols], self.q, self.n),
                _strided(self.base + self.at[2 * cols + 1], self.steps[cols], self.n))

    def view(self, k: int, i: int):
        """Part k of matrix i as a tensor, or None."""
        if self.at[k] is None:
            return None
        T, C, scales = self.T, self.C, k % 2
        typed = self._typed[scales]
        if typed is None:
            typed = self._typed[scales] = self.buf.view(torch.float32 if scales else DTYPES[self.fmt])
        if not scales:
            return typed.as_strided((T, C), (C, 1), self.at[k] + i * self.q)
        shape = (_up128(C), T) if k == 1 else (_up128(T), C)
        return typed.as_strided(shape, (shape[1], 1), (self.at[k] + i * self.steps[k // 2]) // 4)


class Fp8Tokens:
    """One matrix of activations in 8 bits: by rows, by columns, or both.  The tensors
    rows, row_scale, cols and col_scale are None where that grouping is not there."""

    def __init__(self, rows: torch.Tensor | None = None, row_scale: torch.Tensor | None = None,
                 cols: torch.Tensor | None = None, col_scale: torch.Tensor | None = None):
        self._pack, self._i = None, 0
        self._views = {0: rows, 1: row_scale, 2: cols, 3: col_scale}

    @classmethod
    def _of(cls, pack: _Packed, i: int) -> "Fp8Tokens":
        x = cls.__new__(cls)
        x._pack, x._i, x._views = pack, i, {}
        return x

    def _view(self, k: int):
        if k not in self._views:
            self._views[k] = self._pack.view(k, self._i)
        return self._views[k]

    rows = property(lambda self: self._view(0))
    row_scale = property(lambda self: self._view(1))
    cols = property(lambda self: self._view(2))
    col_scale = property(lambda self: self._view(3))


class Fp8Shards:
    """The shards of one tensor in 8 bits: a sequence of Fp8Tokens."""

    def __init__(self, pack: _Packed):
        self._pack = pack

    def __len__(self) -> int:
        return self._pack.n

    def __getitem__(self, i: int) -> Fp8Tokens:
        if not 0 <= i < self._pack.n:
            raise IndexError(i)
        return Fp8Tokens._of(self._pack, i)


def _format(name: str) -> int:
    if name not in binding.FP8_FORMATS:
        raise ValueError(f"format must be one of {sorted(binding.FP8_FORMATS)}, got {name!r}")
    return binding.FP8_FORMATS[name]


def _check_bf16(x: torch.Tensor, what: str) -> None:
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous() or not x.is_cuda:
        raise ValueError(f"{what} must be a contiguous 2-d bf16 CUDA tensor, got "
                         f"{x.dtype} {tuple(x.shape)} on {x.device}")


def _check_like(x: torch.Tensor, shape: tuple, dtype, device, what: str) -> None:
    if x.shape != shape or x.dtype != dtype or not x.is_contiguous() or x.device != device:
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on "
                         f"{device}, got {x.dtype} {tuple(x.shape)} on {x.device}")


_ARRAYS = [ctypes.c_void_p * n for n in range(9)]


def _pointers(xs):
    return _ARRAYS[len(xs)](*[x.data_ptr() for x in xs])


def _strided(start: int, step: int, n: int):
    """The pointers start, start + step, ... (n of them)."""
    return _ARRAYS[n](*range(start, start + n * step, step)) if step else _ARRAYS[n](*[start] * n)


_quant = functools.lru_cache(maxsize=256)(
    lambda T, C, ld, n, code: binding.make_fp8_quant(T, C, ld, n, code, code))


def _quantize(parts, code: int, scale_ld: int, rows, cols, stream) -> None:
    """One launch over `parts` [T, C]; rows, cols: (q, scale) pointer arrays or None."""
    T, C = parts[0].shape
    dev = parts[0].device
    quant = _quant(T, C, scale_ld, len(parts), code)
    q_rows, s_rows = rows or (None, None)
    q_cols, s_cols = cols or (None, None)
    with binding.on_device(dev):
        binding.tpmlp_fp8_quantize(quant, _pointers(parts), q_rows, s_rows, q_cols,
                                   s_cols, binding.stream_on(dev, stream))


def _check_parts(parts, what: str) -> None:
    if not 1 <= len(parts) <= 8:
        raise ValueError(f"1 to 8 {what}s are taken in a call, got {len(parts)}")
    first = parts[0]
    _check_bf16(first, what)
    shape, dev = first.shape, first.device
    for x in parts[1:]:
        if (x.dtype is not torch.bfloat16 or x.shape != shape or x.device != dev
                or not x.is_contiguous()):
            _check_bf16(x, what)
            raise ValueError(f"{what}s must have one shape and device")


def quantize_tokens(X, fmt: str = "e4m3", rows: bool = True, cols: bool = False,
                    out: Fp8Tokens | None = None, stream=None) -> Fp8Tokens:
    """X: a bf16 tensor [T, C], or the list of its token chunks, which are
    gathered on the way.  rows and cols choose the groupings (one read makes
    both); out: buffers to reuse, as returned by an earlier call."""
    chunks = [X] if isinstance(X, torch.Tensor) else list(X)
    code = _format(fmt)
    _check_parts(chunks, "token chunk")
    first, n = chunks[0], len(chunks)
    tc, C = first.shape
    if n > 1 and tc % 128:
        raise ValueError("token chunks must be a multiple of 128 tokens")
    if not (rows or cols):
        raise ValueError("choose rows, cols or both")
    T, dev = tc * n, first.device
    if out is None:
        pack = _Packed(1, T, C, fmt, rows, cols, dev, stream)
        out = Fp8Tokens._of(pack, 0)
        at = [None if a is None else pack.base + a for a in pack.at]
    else:
        at = [None] * 4
        for wanted, k, shape in ((rows, 0, (_up128(C), T)), (cols, 2, (_up128(T), C))):
            if wanted:
                q, scale = out._view(k), out._view(k + 1)
                if q is None or scale is None:
                    raise ValueError("out has no buffers for a grouping that is wanted")
                _check_like(q, (T, C), DTYPES[fmt], dev, "out")
                _check_like(scale, shape, torch.float32, dev, "out's scales")
                at[k], at[k + 1] = q.data_ptr(), scale.data_ptr()

    # token chunk j's part of each output
    _quantize(chunks, code, max(T, 1),
              (_strided(at[0], tc * C, n), _strided(at[1], tc * 4, n)) if rows else None,
              (_strided(at[2], tc * C, n), _strided(at[3], tc // 128 * C * 4, n)) if cols else None,
              stream)
    return out


def quantize_shards(shards, fmt: str = "e4m3", rows: bool = True, cols: bool = False,
                    stream=None) -> Fp8Shards:
    """Each of up to eight bf16 tensors [T, C] of one shape, in one launch."""
    shards = list(shards)
    code = _format(fmt)
    _check_parts(shards, "shard")
    if not (rows or cols):
        raise ValueError("choose rows, cols or both")
    T, C = shards[0].shape
    pack = _Packed(len(shards), T, C, fmt, rows, cols, shards[0].device, stream)
    _quantize(shards, code, max(T, 1), pack.pointers(False) if rows else None,
              pack.pointers(True) if cols else None, stream)
    return Fp8Shards(pack)


def quantize_weight(W: torch.Tensor, fmt: str = "e4m3", stream=None) -> tuple:
    """(q, scale) of one bf16 weight shard [in, out] in 128 x 128 blocks."""
    code = _format(fmt)
    _check_bf16(W, "W")
    r, c = W.shape
    with binding.allocate_on(W.device, stream):
        q = torch.empty(r, c, dtype=DTYPES[fmt], device=W.device)
        s = torch.empty(_up128(r), _up128(c), dtype=torch.float32, device=W.device)
    with binding.on_device(W.device):
        binding.tpmlp_fp8_quantize_weight(W, r, c, code, q, s, binding.stream_on(W.device, stream))
    return q, s


class DeviceFp8Linear:
    """One linear layer on quantised weight shards (``quantize_weight``): the
    8-bit counterpart of ``linear.DeviceLinear`` for the same workloads.

    forward takes activations by rows, backward the same activations by
    columns; ``quantize(X, cols=True)`` makes both in one pass."""

    def __init__(self, w: LinearWorkload, Wq, Ws, b: torch.Tensor, x_format: str = "e4m3",
                 w_format: str = "e4m3", dy_format: str = "e4m3",
                 workspace: torch.Tensor | None = None):
        if w.split not in ("column", "row"):
            raise ValueError("split must be 'column' or 'row'")
        self.w = w
        self.column = w.split == "column"
        self.x_format = x_format
        self._x_dtype = DTYPES.get(x_format)
        self.formats = binding.make_fp8_formats(_format(x_format), _format(w_format),
                                                _format(dy_format))
        T, din, dout, t, n = w.tokens, w.in_features, w.out_features, w.t, w.seq_chunks
        self.dims = binding.make_linear_dims(T, din, dout, t, n)
        need = binding.tpmlp_fp8_linear_workspace_bytes(self.dims)
        if need == 0:
            raise ValueError(f"unsupported dims for an 8-bit linear layer: {w}")
        # (pointers of the layer's own buffers are marshalled once, so it keeps them)
        self._Wq, self._Ws, self.b = tuple(Wq), tuple(Ws), b
        if not b.is_cuda:
            raise ValueError(f"the layer's tensors must be CUDA tensors, got b on {b.device}")
        self.device = dev = b.device
        s = w.shard
        wshape = (din, s) if self.column else (s, dout)
        if len(self.Wq) != t or len(self.Ws) != t:
            raise ValueError(f"{t} weight shards and scales are needed")
        for q, sc in zip(self.Wq, self.Ws):
            _check_like(q, wshape, DTYPES[w_format], dev, "a weight shard")
            _check_like(sc, (_up128(wshape[0]), _up128(wshape[1])), torch.float32, dev,
                        "a weight shard's scale")
        _check_like(b, (dout,), torch.bfloat16, dev, "b")
        bf, f32 = torch.bfloat16, torch.float32
        # the shapes of X_i, Y_i (or Z) and their gradients, and how many of each
        self._x = ((T, din), 1) if self.column else ((T, s), t)
        self._y = ((T, s), t) if self.column else ((T // n, dout), n)
        self._dx = ((T // n, din), n) if self.column else ((T, s), t)
        self.Y = [torch.empty(self._y[0], dtype=bf, device=dev) for _ in range(self._y[1])]
        self._dX = self._dx_ptrs = self._grads = None
        if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()
                                      or workspace.numel() * workspace.element_size() < need):
            raise ValueError(f"the workspace needs {need} contiguous bytes on {dev}")
        self.ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8,
                                                                      device=dev)
        self._weights = (_pointers(self.Wq), _pointers(self.Ws))

    # lists of their own: to exchange a buffer, set the attribute
    Wq = property(lambda self: list(self._Wq))
    Ws = property(lambda self: list(self._Ws))

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
                self.dX = [torch.empty(self._dx[0], dtype=torch.bfloat16, device=self.device)
                           for _ in range(self._dx[1])]
        return self._dx_ptrs

    @property
    def dX(self):
        self._input_grads()
        return list(self._dX)

    @dX.setter
    def dX(self, xs):
        self._dX = tuple(self._list(xs, self._dx, "dX"))
        self._dx_ptrs = _pointers(self._dX)

    def _weight_grads(self, stream=None):
        # fp32, four times the weights' bytes
        if self._grads is None:
            shape = self._Wq[0].shape
            with binding.allocate_on(self.device, stream):
                self._grads = ([torch.empty(shape, dtype=torch.float32, device=self.device)
                                for _ in range(self.w.t)],
                               torch.empty(self.w.out_features, dtype=torch.float32,
                                           device=self.device))
        return self._grads

    @property
    def dW(self):
        return self._weight_grads()[0]

    @property
    def db(self):
        return self._weight_grads()[1]

    def quantize(self, X, cols: bool = False, stream=None):
        """The layer's bf16 input (column: [T, in] or its token chunks; row: the
        t shards) as forward and backward take it."""
        if self.column:
            return quantize_tokens(X, self.x_format, True, cols, stream=stream)
        return quantize_shards(X, self.x_format, True, cols, stream=stream)

    def _tokens(self, x, cols: bool):
        shape, n = self._x
        pack = x._pack if isinstance(x, (Fp8Shards, Fp8Tokens)) else None
        if pack is not None and pack.n == n and (n == 1 or isinstance(x, Fp8Shards)):
            if ((pack.T, pack.C) != shape or pack.fmt != self.x_format or pack.device != self.device
                    or pack.at[2 * cols] is None):
                raise ValueError(f"an input quantised by {'columns' if cols else 'rows'} in "
                                 f"{self.x_format}, {shape} on {self.device}, is needed")
            return pack.pointers(cols)
        x = [x] if isinstance(x, Fp8Tokens) else list(x)
        if len(x) != n:
            raise ValueError(f"{n} quantised inputs are needed, got {len(x)}")
        T, C = shape
        sshape = (_up128(T), C) if cols else (_up128(C), T)
        q = [v.cols if cols else v.rows for v in x]
        s = [v.col_scale if cols else v.row_scale for v in x]
        for a, b in zip(q, s):
            if a is None or b is None:
                raise ValueError("the input is not quantised by " + ("columns" if cols else "rows"))
            _check_like(a, shape, self._x_dtype, self.device, "a quantised input")
            _check_like(b, sshape, torch.float32, self.device, "its scale")
        return _pointers(q), _pointers(s)

    def _list(self, xs, spec, what):
        xs = [xs] if isinstance(xs, torch.Tensor) else list(xs)
        if len(xs) != spec[1]:
            raise ValueError(f"{what}: {spec[1]} tensors are needed, got {len(xs)}")
        for x in xs:
            _check_like(x, spec[0], torch.bfloat16, self.device, what)
        return xs

    def forward(self, x, Y=None, stream=None) -> None:
        """x: by rows, as ``quantize`` makes it (column: Fp8Tokens, row: t of them)."""
        q, s = self._tokens(x, cols=False)
        Y = self._y_ptrs if Y is None else _pointers(self._list(Y, self._y, "Y"))
        with binding.on_device(self.device):
            stream = binding.stream_on(self.device, stream)
            if self.column:
                binding.tpmlp_fp8_column_linear_forward(self.dims, self.formats, q[0], s[0],
                                                        *self._weights, self.b, Y, self.ws, stream)
            else:
                binding.tpmlp_fp8_row_linear_forward(self.dims, self.formats, q, s, *self._weights,
                                                     self.b, Y, self.ws, stream)

    def backward(self, dY, x, dX=None, stream=None) -> None:
        """dY: bf16 (column: t shards, row: token chunks); x: by columns, as
        ``quantize`` makes it."""
        q, s = self._tokens(x, cols=True)
        dY = _pointers(self._list(dY, self._y, "dY"))
        dX = self._input_grads(stream) if dX is None else _pointers(self._list(dX, self._dx, "dX"))
        dW, db = self._weight_grads(stream)
        with binding.on_device(self.device):
            stream = binding.stream_on(self.device, stream)
            if self.column:
                binding.tpmlp_fp8_column_linear_backward(
                    self.dims, self.formats, dY, q[0], s[0], *self._weights, dX, dW, db, self.ws, stream)
            else:
                binding.tpmlp_fp8_row_linear_backward(
                    self.dims, self.formats, dY, q, s, *self._weights, dX, dW, db, self.ws, stream)

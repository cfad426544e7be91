"""Device buffers for the norms before and after a block, with its gate and
residual scale, and the calls that run them.

PyTorch is used for device memory and streams only; both passes run in libtpmlp
through :mod:`binding`.  Per token row of width h (include/tpmlp.h):

  Out = residual_scale * X + gate[row // gate_rows] * N_post(Z)
  Xn  = N_pre(Out)        bf16, or 8-bit as ``fp8.DeviceFp8Linear`` takes it
"""
from __future__ import annotations

import torch

from . import binding
from .fp8 import DTYPES, Fp8Tokens, _check_like, _format, _pointers, _up128


class DeviceNormResidual:
    """The norms between two blocks of a residual stream of `tokens` rows.

    post, pre: "rms", "layer" or "none".  quantize: "e4m3" or "e5m2" to write Xn
    in 8 bits by rows (``q``, ``q_scale``) instead of bf16 (``Xn``).  X, Z and
    the gradients may be tensors [tokens, h] or, with seq_chunks, lists of token
    chunks; outputs come as a tensor, or as a list with seq_chunks > 1."""

    def __init__(self, tokens: int, hidden: int, post: str = "rms", pre: str = "rms",
                 gate_rows: int = 0, residual_scale: float = 1.0, eps: float = 1e-5,
                 post_gamma=None, post_beta=None, pre_gamma=None, pre_beta=None,
                 quantize: str | None = None, seq_chunks: int = 1, device=None):
        for kind in (post, pre):
            if kind not in binding.NORM_KINDS:
                raise ValueError(f"a norm is one of {sorted(binding.NORM_KINDS)}, got {kind!r}")
        self.post, self.pre = post, pre
        self.tokens, self.hidden, self.chunks = int(tokens), int(hidden), int(seq_chunks)
        self.gate_rows = int(gate_rows)
        self.quantize = quantize if pre != "none" else None
        self.params = binding.make_norm_params(
            tokens, hidden, binding.NORM_KINDS[post], binding.NORM_KINDS[pre], gate_rows, seq_chunks,
            _format(quantize) if quantize else 0, eps, residual_scale)
        # without Z: the same with no norm after and no gate
        self._before = binding.make_norm_params(
            tokens, hidden, 0, binding.NORM_KINDS[pre], 0, seq_chunks,
            _format(quantize) if quantize else 0, eps, residual_scale)
        need = binding.tpmlp_norm_workspace_bytes(self.params)
        if need == 0:
            raise ValueError(f"unsupported norm: {tokens} tokens x {hidden}, gate_rows {gate_rows}, "
                             f"{seq_chunks} chunks, eps {eps}, residual_scale {residual_scale}")
        if self.quantize and hidden % 16:
            raise ValueError("8-bit rows need a multiple of 16 columns")
        wanted = {"post_gamma": (post_gamma, post != "none"), "post_beta": (post_beta, post == "layer"),
                  "pre_gamma": (pre_gamma, pre != "none"), "pre_beta": (pre_beta, pre == "layer")}
        given = [w for w, used in wanted.values() if used and w is not None]
        self.device = torch.device(device) if device is not None else (
            given[0].device if given else torch.device("cuda:0"))
        if self.device.type != "cuda":
            raise ValueError(f"the norms run on a CUDA device, got {self.device}")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        for name, (w, used) in wanted.items():
            if used:
                if w is None:
                    raise ValueError(f"{name} is needed")
                _check_like(w, (self.hidden,), torch.bfloat16, self.device, name)
            # a weight that the kind does not have is left out
            setattr(self, name, w if used else None)
        self._need = need
        dev, bf = self.device, torch.bfloat16
        self._Out = self._rows()
        self.stats = torch.empty(4, self.tokens, dtype=torch.float32, device=dev)
        self._Xn = self.q = self.q_scale = None
        if pre != "none":
            if self.quantize:
                self.q = torch.empty(self.tokens, self.hidden, dtype=DTYPES[quantize], device=dev)
                self.q_scale = torch.empty(_up128(self.hidden), self.tokens, dtype=torch.float32,
                                           device=dev)
            else:
                self._Xn = self._rows()
        self._grads = None

    def _rows(self):
        return [torch.empty(self.tokens // self.chunks, self.hidden, dtype=torch.bfloat16,
                            device=self.device) for _ in range(self.chunks)]

    def _one(self, xs):
        return xs if xs is None or self.chunks > 1 else xs[0]

    @property
    def Out(self):
        return self._one(self._Out)

    @property
    def Xn(self):
        return self._one(self._Xn)

    @property
    def tokens_by_rows(self) -> Fp8Tokens:
        """The 8-bit Xn as the linear layers take it."""
        return Fp8Tokens(rows=self.q, row_scale=self.q_scale)

    def _list(self, x, what):
        xs = [x] if isinstance(x, torch.Tensor) else list(x)
        if len(xs) != self.chunks:
            raise ValueError(f"{what}: {self.chunks} token chunks are needed, got {len(xs)}")
        for t in xs:
            _check_like(t, (self.tokens // self.chunks, self.hidden), torch.bfloat16, self.device, what)
        return xs

    def _check_gate(self, gate, z):
        if not z:
            if gate is not None:
                raise ValueError("a gate needs Z")
            return
        if (gate is None) != (self.gate_rows == 0):
            raise ValueError("a gate and gate_rows go together")
        if gate is not None:
            _check_like(gate, (self.tokens // self.gate_rows, self.hidden), torch.bfloat16, self.device,
                        "gate")

    def forward(self, X, Z=None, gate=None, stream=None) -> None:
        """Out, Xn (or q, q_scale) and stats from X and the block's output Z; with
        Z = None only Xn = N_pre(X) (Out is X, post and gate do not count)."""
        z = Z is not None
        X = self._list(X, "X")
        Z = self._list(Z, "Z") if z else None
        self._check_gate(gate, z)
        with binding.on_device(self.device):
            binding.tpmlp_norm_forward(
                self.params if z else self._before, _pointers(X), Z and _pointers(Z),
                self.post_gamma if z else None, self.post_beta if z else None, gate, self.pre_gamma,
                self.pre_beta, _pointers(self._Out) if z else None, self._Xn and _pointers(self._Xn),
                self.q, self.q_scale, self.stats, binding.stream_on(self.device, stream))

    def _gradients(self, stream=None):
        # made by the first backward call
        if self._grads is None:
            vec = lambda: torch.empty(self.hidden, dtype=torch.float32, device=self.device)  # noqa: E731
            with binding.allocate_on(self.device, stream):
                self._grads = {
                    "dX": self._rows(), "dZ": self._rows(),
                    "dpost_gamma": vec() if self.post != "none" else None,
                    "dpost_beta": vec() if self.post == "layer" else None,
                    "dpre_gamma": vec() if self.pre != "none" else None,
                    "dpre_beta": vec() if self.pre == "layer" else None,
                    "dgate": torch.empty(self.tokens // self.gate_rows, self.hidden,
                                         dtype=torch.float32, device=self.device)
                    if self.gate_rows else None,
                    "ws": torch.empty(self._need, dtype=torch.uint8, device=self.device)}
        return self._grads

    dX = property(lambda self: self._one(self._gradients()["dX"]))
    dZ = property(lambda self: self._one(self._gradients()["dZ"]))
    dpost_gamma = property(lambda self: self._gradients()["dpost_gamma"])
    dpost_beta = property(lambda self: self._gradients()["dpost_beta"])
    dpre_gamma = property(lambda self: self._gradients()["dpre_gamma"])
    dpre_beta = property(lambda self: self._gradients()["dpre_beta"])
    dgate = property(lambda self: self._gradients()["dgate"])

    def backward(self, dOut, dXn, Z, Out, stats=None, gate=None, stream=None) -> None:
        """dX, dZ and the weights' gradients for the gradients of Out and Xn (either
        may be None).  Z: the block's output, or None for the norm before alone, Out
        then being X; stats: as the forward pass left them (default: this object's)."""
        z = Z is not None
        if self.pre == "none" and dXn is not None:
            raise ValueError("there is no norm before: dXn must be None")
        if self.pre != "none" and dXn is None:
            raise ValueError("dXn is needed")
        stats = self.stats if stats is None else stats
        _check_like(stats, (4, self.tokens), torch.float32, self.device, "stats")
        self._check_gate(gate, z)
        d = self._gradients(stream)
        opt = lambda x, what: None if x is None else _pointers(self._list(x, what))  # noqa: E731
        with binding.on_device(self.device):
            binding.tpmlp_norm_backward(
                self.params if z else self._before, opt(dOut, "dOut"), opt(dXn, "dXn"), opt(Z, "Z"),
                opt(Out, "Out") if self.pre != "none" else None,
                self.post_gamma if z else None, self.post_beta if z else None, gate, self.pre_gamma,
                stats, _pointers(d["dX"]), _pointers(d["dZ"]) if z else None,
                d["dpost_gamma"] if z else None, d["dpost_beta"] if z else None,
                d["dgate"] if z else None, d["dpre_gamma"], d["dpre_beta"], d["ws"],
                binding.stream_on(self.device, stream))

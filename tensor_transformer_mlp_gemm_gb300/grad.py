"""The norm of a list of gradients together, and clipping by it, before an optimiser's step.

PyTorch is used for device memory and streams only; both run in libtpmlp through
:mod:`binding` (include/tpmlp.h):

  norm = sqrt(sum over all tensors of grad^2)
  out  = grad * min(1, max_norm / (norm + 1e-6))
"""
from __future__ import annotations

import torch

from . import binding


def _refuse(x: torch.Tensor, what: str, device):
    raise ValueError(f"{what} must be contiguous fp32, bf16 or fp16 tensors on {device}, got {x.dtype} "
                     f"{tuple(x.shape)} {'' if x.is_contiguous() else 'not contiguous '}on {x.device}")


def _check_apart(spans) -> None:
    """Nothing is written over what another entry reads or writes."""
    spans.sort()
    for (_, end, i), (start, _, j) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError(f"gradients and outputs lie over each other (numbers {i} and {j} of the list)")


class DeviceGradients:
    """A list of gradients (fp32, bf16, fp16; any sizes) that are clipped together.

    out: where the clipped ones go, tensors of the same shapes and types, or None: in place.
    Both stay the same, with the addresses that they have now: for others another list is made.
    ``norm``: fp32 [1] on the device, written by both calls."""

    def __init__(self, grads, out=None):
        self._grads = grads = tuple(grads)
        self._out = out = grads if out is None else tuple(out)
        if not grads:
            raise ValueError("at least one gradient is needed")
        if len(out) != len(grads):
            raise ValueError(f"{len(grads)} outputs are needed, got {len(out)}")
        self.device = dev = grads[0].device
        if dev.type != "cuda":
            _refuse(grads[0], "gradients", "a CUDA device")
        # (one pass: a list has hundreds of tensors)
        entries, spans = [], []
        for i, (g, o) in enumerate(zip(grads, out)):
            dtype, count, at = g.dtype, g.numel(), g.data_ptr()
            code = binding.GRAD_TYPES.get(dtype)
            if code is None or not g.is_contiguous() or g.device != dev:
                _refuse(g, "gradients", dev)
            end, to = at + count * g.element_size(), at
            if o is not g:
                if not o.is_contiguous() or o.device != dev:
                    _refuse(o, "outputs", dev)
                if o.dtype != dtype or o.shape != g.shape:
                    raise ValueError(f"outputs have their gradients' shape and type: got {dtype} "
                                     f"{tuple(g.shape)} and {o.dtype} {tuple(o.shape)}")
                to = o.data_ptr()
            if count:
                spans.append((at, end, i))
                if to != at:
                    spans.append((to, to + end - at, i))
            entries.append((at, to, count, code))
        _check_apart(spans)
        self._n = n = len(grads)
        need = binding.tpmlp_grad_workspace_bytes(n)
        if need == 0:
            raise ValueError(f"too many gradients for a call: {n}")
        self._measure = binding.prepared("tpmlp_grad_norm")
        self._clip = binding.prepared("tpmlp_grad_clip")
        # (marshalled once, so the object keeps the tensors)
        self._tensors = binding.make_grad_tensors(entries)
        self.norm = torch.empty(1, dtype=torch.float32, device=dev)
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)

    grads = property(lambda self: self._grads)
    out = property(lambda self: self._out)

    def measure(self, stream=None) -> torch.Tensor:
        """The norm, without clipping."""
        with binding.on_device(self.device):
            self._measure(self._tensors, self._n, self.norm.data_ptr(), self.ws.data_ptr(),
                          binding.stream_on(self.device, stream))
        return self.norm

    def clip(self, max_norm: float, stream=None) -> torch.Tensor:
        """Writes the clipped gradients; returns the norm before clipping."""
        with binding.on_device(self.device):
            self._clip(self._tensors, self._n, max_norm, self.norm.data_ptr(), self.ws.data_ptr(),
                       binding.stream_on(self.device, stream))
        return self.norm

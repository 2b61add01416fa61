"""AdamW over many tensors at once (poetx_adamw_multi_step), with moments in fp32 or in e4m3.

Plumbing only: the tensors are checked and their addresses laid out once, and every step is one
library call (one launch for up to 448 tensors).  The arithmetic and the 8-bit format are
described at poetx_adamw_multi_step in include/poetx.h.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import (POETX_BF16, POETX_F32, POETX_MOMENT_BLOCK, POETX_MOMENT_E4M3, POETX_MOMENT_F32, poetx_adamw_cfg,
               poetx_adamw_multi_step, poetx_adamw_tensor)

_DTYPES = {torch.float32: POETX_F32, torch.bfloat16: POETX_BF16}
_CODES = (torch.float8_e4m3fn, torch.uint8)


class AdamWTensor(NamedTuple):
    """One parameter tensor, its gradient and its moments.  m and v: float32 of the parameter's
    length, or e4m3 codes (float8_e4m3fn or uint8) with scale float32 [ceil(n / 256), 2]."""
    param: torch.Tensor
    grad: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    scale: Optional[torch.Tensor] = None
    lr_scale: float = 1.0
    decay_scale: float = 1.0


def new_moments(param: torch.Tensor, moments: str = "e4m3"):
    """(m, v, scale) of a parameter before its first step: zeros, in "e4m3" or in "f32" (scale None)."""
    n, dev = param.numel(), param.device
    if moments == "f32":
        return torch.zeros(n, device=dev), torch.zeros(n, device=dev), None
    if moments != "e4m3":
        raise ValueError(f"moments: 'e4m3' or 'f32', got {moments!r}")
    codes = [torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
    return codes[0], codes[1], torch.zeros((n + POETX_MOMENT_BLOCK - 1) // POETX_MOMENT_BLOCK, 2, device=dev)


class MultiAdamW:
    """The tensors of one optimiser on one device.  Keeps references to them; their addresses must
    not change while it is used (gradients are written in place, as the layers and GradBuckets do).
    All of them share one step count: tensors whose moments restart at different times (theta, which a
    merge restarts, and norms or embeddings, which it does not) take an object each.  Its state, as a checkpoint
    keeps it, is every tensor's m, v and scale and the step count t."""

    def __init__(self, tensors):
        self.tensors = [x if isinstance(x, AdamWTensor) else AdamWTensor(*x) for x in tensors]
        self.t = 0
        self._device = None
        self._entries = (poetx_adamw_tensor * len(self.tensors))()
        spans = []
        for i, x in enumerate(self.tensors):
            self._entries[i] = self._entry(i, x, spans)
        # Every array of a step is read or written by one thread of one tensor only.
        spans.sort()
        for (_, end, a), (start, _, b) in zip(spans, spans[1:]):
            if start < end:
                raise ValueError(f"{a} and {b} overlap")

    @classmethod
    def from_params(cls, params, grads, moments: str = "e4m3"):
        """An optimiser with new moments for parameters and their gradient buffers."""
        params, grads = list(params), list(grads)
        if len(params) != len(grads):
            raise ValueError(f"{len(params)} parameters and {len(grads)} gradients")
        return cls([AdamWTensor(p, g, *new_moments(p, moments)) for p, g in zip(params, grads)])

    def _entry(self, i, x, spans):
        n = x.param.numel()
        e4m3 = x.m.dtype in _CODES
        want = [("param", x.param, n, tuple(_DTYPES)), ("grad", x.grad, n, tuple(_DTYPES)),
                ("m", x.m, n, _CODES if e4m3 else (torch.float32,)),
                ("v", x.v, n, _CODES if e4m3 else (torch.float32,))]
        if e4m3:
            if x.scale is None:
                raise ValueError(f"tensor {i}: e4m3 moments need their scales")
            want.append(("scale", x.scale, 2 * ((n + POETX_MOMENT_BLOCK - 1) // POETX_MOMENT_BLOCK), (torch.float32,)))
        elif x.m.dtype == torch.float32 and x.scale is not None:
            raise ValueError(f"tensor {i}: fp32 moments take no scales")
        for name, a, numel, dtypes in want:
            what = f"tensor {i}: {name}"
            if not a.is_cuda:
                raise ValueError(f"{what} must be a CUDA tensor")
            if self._device is None:
                self._device = a.device
            if a.device != self._device:
                raise ValueError(f"{what} is on {a.device}, not on {self._device}")
            if not a.is_contiguous():
                raise ValueError(f"{what} must be contiguous")
            if a.dtype not in dtypes:
                raise ValueError(f"{what}: expected {' or '.join(map(str, dtypes))}, got {a.dtype}")
            if a.numel() != numel:
                raise ValueError(f"{what}: needs {numel} elements, has {a.numel()}")
            if numel:
                start = a.data_ptr()
                spans.append((start, start + numel * a.element_size(), what))
        return poetx_adamw_tensor(
            x.param.data_ptr(), x.grad.data_ptr(), x.m.data_ptr(), x.v.data_ptr(),
            x.scale.data_ptr() if e4m3 else None, n, x.lr_scale, x.decay_scale, _DTYPES[x.param.dtype],
            _DTYPES[x.grad.dtype], POETX_MOMENT_E4M3 if e4m3 else POETX_MOMENT_F32)

    def step(self, cfg: poetx_adamw_cfg, t: Optional[int] = None, seed: int = 0, stream=None):
        """One step.  t: the moments' step count (default: one more than the last step's).  seed: 0
        rounds to nearest, another (a new one each step) rounds stochastically.  Under stream capture cfg, t
        and seed are kept by the graph: every replay is the same step."""
        t = self.t + 1 if t is None else t
        if self._device is not None and self._device.index != torch.cuda.current_device():
            with torch.cuda.device(self._device):
                poetx_adamw_multi_step(cfg, len(self.tensors), self._entries, t, seed, stream)
        else:
            poetx_adamw_multi_step(cfg, len(self.tensors), self._entries, t, seed, stream)
        self.t = t

    def reset(self, stream=None):
        """Zeroes the moments, as after a merge, in the order of `stream` (as step takes it); the step count
        starts again."""
        if self._device is not None:
            if isinstance(stream, int):
                stream = torch.cuda.ExternalStream(stream, self._device)
            with torch.cuda.device(self._device), torch.cuda.stream(stream):
                for x in self.tensors:
                    for a in (x.m, x.v, x.scale):
                        if a is not None:
                            (a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a).zero_()
        self.t = 0

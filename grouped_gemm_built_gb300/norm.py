"""Layer norm and RMS norm with the residual sum in front (``mok_norm_fwd`` and ``mok_norm_bwd``
in include/mok_ops.h), on torch tensors and the current CUDA stream."""
from __future__ import annotations

from typing import Optional

import torch

from . import mok
from .layer import _dev, _result_code, _results


class Norm:
    """``y = (h - m) r weight + bias`` per row of ``h = x + add``: m the row's mean (0 for
    ``kind="rms"``), r the inverse root of its mean square around m plus eps. weight [H] and
    bias [H] or None, bf16 or fp32; like ``AdaptedLinear`` the object keeps the tensors, and a
    call reads what they hold then."""

    KINDS = {"layer": mok.MOK_NORM_LAYER, "rms": mok.MOK_NORM_RMS}

    def __init__(self, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 kind: str = "rms", eps: float = 1e-6):
        if kind not in self.KINDS:
            raise ValueError(f"kind must be one of {sorted(self.KINDS)}, got {kind!r}")
        self.weight, self.bias, self.kind, self.eps = weight, bias, kind, float(eps)
        self.H = self._check_weights()
        mok.mok_norm_get_sizes(mok.MokNormDims(T=0, H=self.H, kind=self.KINDS[kind], eps=self.eps,
                                               x_type=0, y_type=0, w_type=0))

    def _check_weights(self) -> int:
        for name in ("weight", "bias"):
            t = getattr(self, name)
            if t is None and name == "bias":
                continue
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
            if t.dim() != 1:
                raise ValueError(f"{name} must have 1 dimension, got {tuple(t.shape)}")
        w = self.weight
        _result_code(w.dtype, "weight")
        H = getattr(self, "H", w.numel())
        _dev(w, "weight", w.dtype, H)
        _dev(self.bias, "bias", w.dtype, H, optional=True)
        return H

    def _rows(self, t, name: str, T=None, dtype=None) -> int:
        """The rows of a tensor [T, H], of a given number or type where one is named."""
        dt = t.dtype if isinstance(t, torch.Tensor) else None
        _result_code(dt, name)
        if t.dim() != 2 or t.shape[1] != self.H or T not in (None, t.shape[0]):
            raise ValueError(f"{name} must be [{'T' if T is None else T}, {self.H}], got {tuple(t.shape)}")
        _dev(t, name, dtype or dt, t.numel())
        return t.shape[0]

    def _check_forward(self, x, add):
        T = self._rows(x, "x")
        if add is not None:
            self._rows(add, "add", T, x.dtype)
        self._check_weights()

    def _check_backward(self, dY, h, stats, add):
        T = self._rows(h, "h")
        self._rows(dY, "dY", T)
        _dev(stats, "stats", torch.float32, 2 * T)
        if add is not None:
            self._rows(add, "add", T, h.dtype)
        self._check_weights()

    def forward(self, x: torch.Tensor, add: Optional[torch.Tensor] = None,
                out: Optional[torch.dtype] = None):
        """(y [T,H], h [T,H], stats) from x [T,H] bf16 or fp32 and ``add`` like it (the residual
        stream); y in the type ``out`` (x's by default). Without ``add``, h is x itself. ``h``
        and ``stats`` are what ``backward`` takes."""
        code = _result_code(out or getattr(x, "dtype", None), "y")
        got = mok.torch_calls().norm_fwd(self.KINDS[self.kind], self.eps, self.weight, self.bias, x,
                                         add, code)
        if type(got) is tuple:
            return got
        return _results(got, "mok_norm_fwd", lambda: self._check_forward(x, add))

    def backward(self, dY: torch.Tensor, h: torch.Tensor, stats: torch.Tensor,
                 add: Optional[torch.Tensor] = None):
        """{"dX", "dW"[, "dB"]} for dY [T,H] (y's type), after ``forward`` gave h and stats;
        dW and dB in the parameters' type. ``add`` [T,H] (h's type): the gradient that reaches h
        along the residual stream. dX is the gradient of x and of forward's ``add``."""
        got = mok.torch_calls().norm_bwd(self.KINDS[self.kind], self.eps, self.weight, self.bias,
                                         h, dY, stats, add)
        if type(got) is not tuple:
            _results(got, "mok_norm_bwd", lambda: self._check_backward(dY, h, stats, add))
        return dict(zip(("dX", "dW", "dB"), got))

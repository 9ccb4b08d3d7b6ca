"""Dropout whose mask is a function of (seed, offset, element) and is never stored
(``mok_dropout`` in include/mok_ops.h), on torch tensors and the current CUDA stream."""
from __future__ import annotations

from typing import Optional

import torch

from . import mok
from .layer import _dev, _result_code, _results


def _check(x, add, y):
    dt = x.dtype if isinstance(x, torch.Tensor) else None
    _result_code(dt, "x")
    n = x.numel()
    _dev(x, "x", dt, n)
    _dev(add, "add", dt, n, optional=True)
    _dev(y, "y", dt, n, optional=True)


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0,
            add: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """``(add or 0) + x * mask / keep`` for bf16 or fp32 ``x``; each element is dropped with
    probability round(65536 p) / 65536. The backward is the same call on the gradient. Calls
    that need masks of their own take different seeds, or offsets at least
    ``(x.numel() + 7) // 8`` apart. ``y`` may be ``x`` or ``add``."""
    got = mok.torch_calls().dropout(x, p, seed, offset, add, y)
    out = _results(got, "mok_dropout", lambda: _check(x, add, y))[0]
    return out if y is None else y

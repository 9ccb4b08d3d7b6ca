"""Dropout whose mask is a function of (seed, offset, element) and is never stored
(``mok_dropout`` in include/mok_ops.h), on torch tensors and the current CUDA stream."""
from __future__ import annotations

from typing import Optional

import torch

from . import mok
from .layer import _dev, _on_current_stream, _result_code


def dropout(x: torch.Tensor, p: float, seed: int, offset: int = 0,
            add: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None):
    """``(add or 0) + x * mask / keep`` for bf16 or fp32 ``x``; each element is dropped with
    probability round(65536 p) / 65536. The backward is the same call on the gradient. Calls
    that need masks of their own take different seeds, or offsets at least
    ``(x.numel() + 7) // 8`` apart. ``y`` may be ``x`` or ``add``."""
    dt = x.dtype if isinstance(x, torch.Tensor) else None
    code = _result_code(dt, "x")
    n = x.numel()
    px = _dev(x, "x", dt, n)
    pa = _dev(add, "add", dt, n, optional=True)
    if y is None:
        y = torch.empty_like(x)
    py = _dev(y, "y", dt, n)
    _on_current_stream(x.get_device(), mok.mok_dropout, px, pa, py, n, p, seed, offset, code)
    return y

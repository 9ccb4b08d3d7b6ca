"""Balance loss, penalty on large logits and expert counts of a router, with the gradient
(``mok_balance_fwd`` and ``mok_balance_bwd`` in include/mok_ops.h), on torch tensors.

Beside a ``Routing`` over the same logits::

    idx, gates = R.forward(logits, bias)
    losses, counts, saved = B.forward(logits, idx)
    ...
    dlogits = R.backward(logits, idx, dgates)
    dlogits = B.backward(logits, saved, add=dlogits)
"""
from __future__ import annotations

from typing import Optional

import torch

from . import mok
from .layer import _dev, _result_code, _results
from .routing import Routing


class Balance:
    """The loss of a router over E experts that chooses k; see ``mok_balance_fwd``."""

    def __init__(self, E: int, k: int, score: str = "softmax", coef: float = 1e-2,
                 z_coef: float = 0.0):
        if score not in Routing.SCORES:
            raise ValueError(f"score must be one of {sorted(Routing.SCORES)}, got {score!r}")
        self.E, self.k = E, k
        self.rule = mok.MokBalance(E=E, k=k, score=Routing.SCORES[score], coef=coef, z_coef=z_coef)
        mok.mok_balance_get_sizes(self.rule, 0)     # checks it

    def _check(self, logits, seqs):
        dt = logits.dtype if isinstance(logits, torch.Tensor) else None
        _result_code(dt, "logits")
        if logits.dim() != 2 or logits.shape[1] != self.E:
            raise ValueError(f"logits must be [T, {self.E}], got {tuple(logits.shape)}")
        _dev(logits, "logits", dt, logits.numel())
        if seqs is not None:
            if not isinstance(seqs, torch.Tensor) or seqs.dim() != 1 or seqs.numel() < 2:
                raise ValueError("seqs must be a tensor of at least two row offsets")
            _dev(seqs, "seqs", torch.int32, seqs.numel())
        return logits.shape[0], 1 if seqs is None else seqs.numel() - 1

    @staticmethod
    def _shape(t, name, *shape):
        if t.shape != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")

    def _check_forward(self, logits, topk_idx, seqs):
        T, _ = self._check(logits, seqs)
        _dev(topk_idx, "topk_idx", torch.int32, T * self.k)
        self._shape(topk_idx, "topk_idx", T, self.k)

    def _check_backward(self, logits, saved, seqs, dlosses, add, dtype):
        T, S = self._check(logits, seqs)
        _dev(saved, "saved", torch.uint8, mok.mok_balance_get_sizes(self.rule, T, S))
        _dev(dlosses, "dlosses", torch.float32, 2, optional=True)
        _dev(add, "add", dtype, T * self.E, optional=True)
        if add is not None:
            self._shape(add, "add", T, self.E)

    def forward(self, logits: torch.Tensor, topk_idx: torch.Tensor,
                seqs: Optional[torch.Tensor] = None):
        """(losses [2] fp32: balance and logit penalty, counts [E] int32, saved) of logits [T,E]
        bf16 or fp32 whose router chose topk_idx [T,k] int32. ``seqs`` [S + 1] int32 on the
        device: row offsets of sequences that are balanced one by one; rows outside take no
        part. ``saved`` is what ``backward`` takes."""
        got = mok.torch_calls().balance_fwd(self.rule, logits, topk_idx, seqs)
        if type(got) is tuple:
            return got
        return _results(got, "mok_balance_fwd", lambda: self._check_forward(logits, topk_idx, seqs))

    def backward(self, logits: torch.Tensor, saved: torch.Tensor,
                 seqs: Optional[torch.Tensor] = None, dlosses: Optional[torch.Tensor] = None,
                 add: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None):
        """dlogits [T,E] (``dtype``, by default ``add``'s type or the logits') of the losses
        weighted by dlosses [2] fp32 (None: ones), plus ``add`` [T,E]; after ``forward`` with
        the same logits and seqs."""
        dtype = dtype or getattr(logits if add is None else add, "dtype", None)
        got = mok.torch_calls().balance_bwd(self.rule, logits, seqs, saved, dlosses, add,
                                            _result_code(dtype, "dlogits"))
        if type(got) is tuple:
            return got[0]
        return _results(got, "mok_balance_bwd", lambda: self._check_backward(
            logits, saved, seqs, dlosses, add, dtype))[0]

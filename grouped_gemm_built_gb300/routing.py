"""Routing to experts on torch tensors (``mok_route`` and ``mok_route_bwd`` in
include/mok_ops.h): softmax or sigmoid scores, a balance bias that steers the choice only,
expert groups, top-k, and the gradient of the gates with respect to the logits.

The results feed a layer without a router of its own (``MoELayer(router=False)``):
``plan(topk_idx=idx, gates=gates)``, then ``backward`` gives the ``dgates`` that
``Routing.backward`` takes.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import mok
from .layer import _dev, _result_code, _results


class Routing:
    """A routing rule over E experts; see ``mok_routing`` for what each field means."""

    SCORES = {"softmax": mok.MOK_SCORE_SOFTMAX, "sigmoid": mok.MOK_SCORE_SIGMOID}
    GROUP_SCORES = {"max": mok.MOK_GROUP_MAX, "top2": mok.MOK_GROUP_TOP2}

    def __init__(self, E: int, k: int, score: str = "softmax", groups: int = 1,
                 top_groups: int = 1, group_score: str = "max", renormalize: bool = True,
                 scale: float = 1.0):
        if score not in self.SCORES:
            raise ValueError(f"score must be one of {sorted(self.SCORES)}, got {score!r}")
        if group_score not in self.GROUP_SCORES:
            raise ValueError(f"group_score must be one of {sorted(self.GROUP_SCORES)}, "
                             f"got {group_score!r}")
        self.E, self.k = E, k
        self.rule = mok.MokRouting(E=E, k=k, score=self.SCORES[score], groups=groups,
                                   top_groups=top_groups,
                                   group_score=self.GROUP_SCORES[group_score],
                                   renormalize=1 if renormalize else 0, scale=scale)
        mok.mok_route(self.rule, 0, None, mok.MOK_OUT_F32, None, None, None, None)  # checks it

    def _check(self, logits, bias=None, topk_idx=None, dgates=None, backward=False):
        dt = logits.dtype if isinstance(logits, torch.Tensor) else None
        _result_code(dt, "logits")
        if logits.dim() != 2 or logits.shape[1] != self.E:
            raise ValueError(f"logits must be [T, {self.E}], got {tuple(logits.shape)}")
        T = logits.shape[0]
        _dev(logits, "logits", dt, T * self.E)
        _dev(bias, "bias", torch.float32, self.E, optional=True)
        if backward:
            _dev(topk_idx, "topk_idx", torch.int32, T * self.k)
            _dev(dgates, "dgates", torch.float32, T * self.k)

    def forward(self, logits: torch.Tensor, bias: Optional[torch.Tensor] = None):
        """(topk_idx [T,k] int32, gates [T,k] fp32) from logits [T,E] bf16 or fp32 and the
        selection bias [E] fp32."""
        return _results(mok.torch_calls().route(self.rule, logits, bias), "mok_route",
                        lambda: self._check(logits, bias))

    def backward(self, logits: torch.Tensor, topk_idx: torch.Tensor, dgates: torch.Tensor,
                 dtype: Optional[torch.dtype] = None):
        """dlogits [T,E] (``dtype``, the logits' type by default) from dgates [T,k] fp32, at
        the choice that ``forward`` made from these logits."""
        dtype = dtype or getattr(logits, "dtype", None)
        got = mok.torch_calls().route_bwd(self.rule, logits, topk_idx, dgates,
                                          _result_code(dtype, "dlogits"))
        return _results(got, "mok_route_bwd", lambda: self._check(
            logits, topk_idx=topk_idx, dgates=dgates, backward=True))[0]

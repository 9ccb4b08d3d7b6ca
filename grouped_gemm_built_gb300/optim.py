"""The norm of all gradients and the AdamW step over many tensors (``mok_grad_norm`` and
``mok_adamw`` in include/mok_ops.h), on torch tensors and the current CUDA stream::

    opt = AdamW(params, weight_decay=0.1, bits=8)
    norm, coef = grad_norm(grads, max_norm=1.0)     # coef stays on the device
    opt.step(grads, lr=3e-4, coef=coef)             # skipped where the norm is not finite
"""
from __future__ import annotations

from typing import Optional, Sequence, Union

import torch

from . import mok
from .layer import _dev, _result_code, _results


def _check_grads(grads):
    if not isinstance(grads, (list, tuple)):
        raise TypeError(f"grads must be a list or tuple of tensors, got {type(grads).__name__}")
    for i, g in enumerate(grads):
        if g is not None:
            if not isinstance(g, torch.Tensor):
                raise TypeError(f"grads[{i}] must be a torch.Tensor, got {type(g).__name__}")
            _result_code(g.dtype, f"grads[{i}]")
            _dev(g, f"grads[{i}]", g.dtype, g.numel())


def grad_norm(grads: Sequence[Optional[torch.Tensor]], max_norm: float = float("inf"),
              scale: float = 1.0):
    """(norm, coef), fp32 tensors of one value: norm = scale * the 2-norm of all gradients (bf16
    or fp32 tensors on one device, None for none), coef = scale * min(1, max_norm / norm), NaN
    when the norm is not finite."""
    got = mok.torch_calls().grad_norm(grads, max_norm, scale)
    if type(got) is tuple:
        return got

    def check():
        _check_grads(grads)
        if all(g is None for g in grads):
            raise ValueError("grads must hold at least one tensor")

    return _results(got, "mok_grad_norm", check)


class AdamW:
    """AdamW for a fixed list of tensors, bf16 or fp32, on one device. ``weight_decay``: one
    number, or one per tensor. ``bits``: 32 or 8, of the moments. The state is
    ``master`` (fp32 values of bf16 tensors, or None), ``m``, ``v``, ``scales`` (8-bit moments'
    block scales, or None): one tensor each for all parameters, in the layout of
    ``mok_adamw_state``; ``steps`` counts the steps taken. To restore a state, copy into them
    and set ``steps``; after changing a bf16 parameter by hand, call ``read_params``."""

    def __init__(self, params: Sequence[torch.Tensor], betas=(0.9, 0.95), eps: float = 1e-8,
                 weight_decay: Union[float, Sequence[float]] = 0.0, bits: int = 32, seed: int = 0):
        self.params = tuple(params)
        if not self.params:
            raise ValueError("params must hold at least one tensor")
        for i, p in enumerate(self.params):
            if not isinstance(p, torch.Tensor):
                raise TypeError(f"params[{i}] must be a torch.Tensor, got {type(p).__name__}")
            _result_code(p.dtype, f"params[{i}]")
            _dev(p, f"params[{i}]", p.dtype, p.numel())
            if p.device != self.params[0].device:
                raise ValueError(f"params[{i}] must be on params[0]'s device "
                                 f"{self.params[0].device}, got {p.device}")
        if isinstance(weight_decay, (int, float)):
            weight_decay = [weight_decay] * len(self.params)
        weight_decay = [float(d) for d in weight_decay]
        if len(weight_decay) != len(self.params):
            raise ValueError(f"weight_decay must be one number or {len(self.params)}, "
                             f"got {len(weight_decay)}")
        if bits not in (8, 32):
            raise ValueError(f"bits must be 8 or 32, got {bits!r}")
        self.rule = mok.MokAdamwRule(beta1=betas[0], beta2=betas[1], eps=eps, bits=bits)
        mok.mok_adamw(self.rule, [], mok.MokAdamwState(), 0.0, None, 1, None, None, 0, None)
        self.bits, self.seed, self.steps = bits, int(seed), 0
        sizes = [p.numel() for p in self.params]
        self._what = (mok.MokAdamwTensor * len(sizes))(
            *(mok.MokAdamwTensor(n=n, decay=d, p_type=_result_code(p.dtype, "p"))
              for n, p, d in zip(sizes, self.params, weight_decay)))
        self.elements = mok.mok_adamw_get_sizes(sizes)
        self.device = self.params[0].device
        kind = torch.uint8 if bits == 8 else torch.float32
        self.m = torch.zeros(self.elements, dtype=kind, device=self.device)
        self.v = torch.zeros_like(self.m)
        self.scales = (torch.zeros(self.elements // 256, 2, dtype=kind, device=self.device)
                       if bits == 8 else None)
        self.master = None
        if any(p.dtype == torch.bfloat16 for p in self.params):
            self.master = torch.zeros(self.elements, dtype=torch.float32, device=self.device)
            self.read_params()

    @torch.no_grad()
    def read_params(self) -> None:
        """Sets ``master`` to the values of the bf16 parameters."""
        at = 0
        for p in self.params:
            n = p.numel()
            if p.dtype == torch.bfloat16:
                self.master[at:at + n].copy_(p.reshape(-1))
            at += -(-n // 256) * 256

    def _check(self, grads, lr, t, coef):
        _check_grads(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"grads must hold {len(self.params)} tensors, got {len(grads)}")
        for i, (p, g, what) in enumerate(zip(self.params, grads, self._what)):
            kind = torch.float32 if what.p_type == mok.MOK_OUT_F32 else torch.bfloat16
            _dev(p, f"params[{i}]", kind, what.n)
            if g is not None:
                _dev(g, f"grads[{i}]", g.dtype, what.n)
                if g.shape != p.shape and min(g.dim(), p.dim()) > 1:
                    raise ValueError(f"grads[{i}] must be {list(p.shape)} or flat, got {tuple(g.shape)}")
        if isinstance(lr, torch.Tensor):
            _dev(lr, "lr", torch.float32, 1)
        if isinstance(t, torch.Tensor):
            _dev(t, "step", torch.int32, 1)
        _dev(coef, "coef", torch.float32, 1, optional=True)
        kind = torch.uint8 if self.bits == 8 else torch.float32
        _dev(self.m, "m", kind, self.elements)
        _dev(self.v, "v", kind, self.elements)
        _dev(self.scales, "scales", torch.uint8, self.elements // 128, optional=self.bits == 32)
        _dev(self.master, "master", torch.float32, self.elements, optional=True)

    def step(self, grads: Sequence[Optional[torch.Tensor]], lr: Union[float, torch.Tensor],
             coef: Optional[torch.Tensor] = None, step: Optional[torch.Tensor] = None) -> None:
        """One step with a gradient (bf16 or fp32, of the tensor's shape or flat) per tensor, None
        to leave a tensor as it is.
        ``coef``: factor of all gradients on the device (``grad_norm``'s); the step is skipped
        where it is not finite. A step captured in a graph takes its number from ``step``, an
        int32 tensor of one value that the graph advances, and a changing ``lr`` from an fp32
        tensor; without ``step`` the object counts, skipped steps too."""
        t = self.steps + 1 if step is None else step
        got = mok.torch_calls().adamw(self.rule, self.params, self._what,
                                      (self.master, self.m, self.v, self.scales), self.elements,
                                      grads, lr, t, coef, self.seed)
        if type(got) is not tuple:
            _results(got, "mok_adamw", lambda: self._check(grads, lr, t, coef))
        if step is None:
            self.steps += 1

    def moments(self):
        """(m, v) of all tensors in the state's layout: the fp32 tensors themselves, or the
        values of 8-bit moments in bf16, which holds them exactly (an m below 2^-117, the
        largest of its block, to 2^-134)."""
        if self.bits == 32:
            return self.m, self.v
        return _results(mok.torch_calls().adamw_moments(self.m, self.v, self.scales),
                        "mok_adamw_moments", lambda: None)

"""Low-rank adapters of many requests beside a shared projection, on torch tensors
(``mok_lora_fwd`` and ``mok_lora_bwd`` in include/mok_ops.h)."""
from __future__ import annotations

from typing import Optional

import torch

from . import mok
from .layer import _dev, _on_current_stream, _result_code


class AdaptedLinear:
    """``y = x W + scale[a] (x A_a^T) B_a`` with ``a = ids[t]`` for each row t of x: one frozen
    projection W [K,N], n adapters A [n,r,K] and B [n,r,N] (bf16), scale [n] fp32. The object
    keeps the tensors, not copies: updated weights are what the next call reads."""

    _sized = (-1, None, None)     # rows of the last call, and its dims and buffer sizes

    def __init__(self, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor):
        for name, t, nd in (("W", W, 2), ("A", A, 3), ("B", B, 3)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
            if t.dim() != nd:
                raise ValueError(f"{name} must have {nd} dimensions, got {tuple(t.shape)}")
        self.K, self.N = W.shape
        self.n, self.r = A.shape[:2]
        if A.shape[2] != self.K or tuple(B.shape) != (self.n, self.r, self.N):
            raise ValueError(f"W {tuple(W.shape)}, A {tuple(A.shape)} and B {tuple(B.shape)} "
                             "must be [K,N], [n,r,K] and [n,r,N]")
        bf = torch.bfloat16
        self.w = mok.MokLoraWeights(W=_dev(W, "W", bf, W.numel()), A=_dev(A, "A", bf, A.numel()),
                                    B=_dev(B, "B", bf, B.numel()),
                                    scale=_dev(scale, "scale", torch.float32, self.n))
        self.W, self.A, self.B, self.scale = W, A, B, scale
        self.device = W.device
        self._status = torch.zeros(1, dtype=torch.int32, device=W.device)
        self._dims(1)           # checks the sizes

    def _dims(self, T):
        if self._sized[0] != T:
            d = mok.MokLoraDims(T=T, K=self.K, N=self.N, n=self.n, r=self.r)
            self._sized = (T, d, mok.mok_lora_get_sizes(d))
        return self._sized[1:]

    def _rows(self, x, ids, x_ad):
        if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != self.K:
            raise ValueError(f"x must be a tensor [T, {self.K}]")
        T, bf = x.shape[0], torch.bfloat16
        return (T, _dev(x, "x", bf, T * self.K), _dev(ids, "ids", torch.int32, T),
                _dev(x_ad, "x_ad", bf, T * self.K, optional=True))

    def _scratch(self, nbytes):
        # a buffer of the current stream's allocator: calls on different streams share none
        return torch.empty(nbytes, dtype=torch.uint8, device=self.device)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, x_ad: Optional[torch.Tensor] = None,
                out: torch.dtype = torch.bfloat16):
        """(y [T,N], saved) from x [T,K] bf16 and ids [T] int32 (outside [0, n): no adapter).
        ``x_ad``: the adapters' own input when it is not x (x after dropout). ``saved`` is
        what ``backward`` takes."""
        T, px, pi, pa = self._rows(x, ids, x_ad)
        code = _result_code(out, "y")
        dims, sizes = self._dims(T)
        y = torch.empty((T, self.N), dtype=out, device=self.device)
        saved = self._scratch(sizes.saved_bytes)
        _on_current_stream(x.get_device(), mok.mok_lora_fwd, dims, self.w, px, pa, pi, y.data_ptr(),
                           code, saved.data_ptr(), self._status.data_ptr())
        return y, saved

    def backward(self, x: torch.Tensor, ids: torch.Tensor, saved: torch.Tensor,
                 dY: torch.Tensor, x_ad: Optional[torch.Tensor] = None,
                 out: torch.dtype = torch.bfloat16):
        """{"dX", "dA", "dB"} for dY [T,N] bf16, after ``forward`` with the same x, ids and
        x_ad; with x_ad, "dXa" holds its gradient and "dX" only the shared projection's."""
        T, px, pi, pa = self._rows(x, ids, x_ad)
        code = _result_code(out, "gradients")
        dims, sizes = self._dims(T)
        ps = _dev(saved, "saved", torch.uint8, sizes.saved_bytes)
        pdy = _dev(dY, "dY", torch.bfloat16, T * self.N)

        def new(*shape):
            return torch.empty(shape, dtype=out, device=self.device)

        g = {"dX": new(T, self.K), "dA": new(self.n, self.r, self.K),
             "dB": new(self.n, self.r, self.N)}
        if x_ad is not None:
            g["dXa"] = new(T, self.K)
        ws = self._scratch(sizes.workspace_bytes)
        _on_current_stream(x.get_device(), mok.mok_lora_bwd, dims, self.w, px, pa, pi, ps, pdy,
                           g["dX"].data_ptr(), g["dXa"].data_ptr() if x_ad is not None else None,
                           g["dA"].data_ptr(), g["dB"].data_ptr(), code, ws.data_ptr(),
                           self._status.data_ptr())
        return g

    def status(self) -> int:
        """Waits for the current stream; 0, or MOK_ERR_TIMEOUT after a device wait expired."""
        return _on_current_stream(self._status.get_device(), mok.mok_lora_get_status,
                                  self._status.data_ptr())

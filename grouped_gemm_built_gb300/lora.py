"""Low-rank adapters of many requests beside a shared projection, on torch tensors
(``mok_lora_fwd`` and ``mok_lora_bwd`` in include/mok_ops.h)."""
from __future__ import annotations

from typing import Optional

import torch

from . import mok
from .layer import _dev, _result_code, _results


class AdaptedLinear:
    """``y = x W + scale[a] (x A_a^T) B_a`` with ``a = ids[t]`` for each row t of x: one frozen
    projection W [K,N], n adapters A [n,r,K] and B [n,r,N] (bf16), scale [n] fp32. The object
    keeps the tensors, not copies or addresses: what W, A, B and scale hold at a call is what it
    reads, also after another tensor of the same shape has taken their place."""

    W = A = B = scale = _status = device = None
    _shape = (0, 0, 0, 0)       # K, N, n, r

    def __init__(self, W: torch.Tensor, A: torch.Tensor, B: torch.Tensor, scale: torch.Tensor):
        for name, t, nd in (("W", W, 2), ("A", A, 3), ("B", B, 3)):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
            if t.dim() != nd:
                raise ValueError(f"{name} must have {nd} dimensions, got {tuple(t.shape)}")
        self.K, self.N = W.shape
        self.n, self.r = A.shape[:2]
        self._shape = (self.K, self.N, self.n, self.r)
        if A.shape[2] != self.K or tuple(B.shape) != (self.n, self.r, self.N):
            raise ValueError(f"W {tuple(W.shape)}, A {tuple(A.shape)} and B {tuple(B.shape)} "
                             "must be [K,N], [n,r,K] and [n,r,N]")
        self.W, self.A, self.B, self.scale = W, A, B, scale
        self.device = W.device
        self._check_weights()
        mok.mok_lora_get_sizes(mok.MokLoraDims(T=1, K=self.K, N=self.N, n=self.n, r=self.r))
        self._status = torch.zeros(1, dtype=torch.int32, device=W.device)

    def _check_weights(self):
        K, N, n, r = self._shape
        for name, shape in (("W", (K, N)), ("A", (n, r, K)), ("B", (n, r, N)), ("scale", (n,))):
            t, kind = getattr(self, name), torch.float32 if name == "scale" else torch.bfloat16
            if isinstance(t, torch.Tensor) and t.is_cuda and t.device != self.device:
                raise ValueError(f"{name} must be on W's device {self.device}, got {t.device}")
            numel = 1
            for d in shape:
                numel *= d
            _dev(t, name, kind, numel)
            if name != "scale" and tuple(t.shape) != shape:
                raise ValueError(f"{name} must be {list(shape)}, got {tuple(t.shape)}")

    def _check(self, x, ids, x_ad, saved=None, dY=None, backward=False):
        if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.shape[1] != self.K:
            raise ValueError(f"x must be a tensor [T, {self.K}]")
        T, bf = x.shape[0], torch.bfloat16
        _dev(x, "x", bf, T * self.K)
        _dev(ids, "ids", torch.int32, T)
        _dev(x_ad, "x_ad", bf, T * self.K, optional=True)
        if backward:
            dims = mok.MokLoraDims(T=T, K=self.K, N=self.N, n=self.n, r=self.r)
            _dev(saved, "saved", torch.uint8, mok.mok_lora_get_sizes(dims).saved_bytes)
            _dev(dY, "dY", bf, T * self.N)
        if x.device != self.device:
            raise ValueError(f"x must be on the weights' device {self.device}, got {x.device}")
        self._check_weights()

    def _weights(self):
        return self.W, self.A, self.B, self.scale, self._status, self._shape

    def forward(self, x: torch.Tensor, ids: torch.Tensor, x_ad: Optional[torch.Tensor] = None,
                out: torch.dtype = torch.bfloat16):
        """(y [T,N], saved) from x [T,K] bf16 and ids [T] int32 (outside [0, n): no adapter).
        ``x_ad``: the adapters' own input when it is not x (x after dropout). ``saved`` is
        what ``backward`` takes."""
        code = _result_code(out, "y")
        return _results(mok.torch_calls().lora_fwd(self._weights(), x, ids, x_ad, code),
                        "mok_lora_fwd", lambda: self._check(x, ids, x_ad))

    def backward(self, x: torch.Tensor, ids: torch.Tensor, saved: torch.Tensor,
                 dY: torch.Tensor, x_ad: Optional[torch.Tensor] = None,
                 out: torch.dtype = torch.bfloat16):
        """{"dX", "dA", "dB"} for dY [T,N] bf16, after ``forward`` with the same x, ids, x_ad and
        weights; with x_ad, "dXa" holds its gradient and "dX" only the shared projection's."""
        code = _result_code(out, "gradients")
        got = _results(mok.torch_calls().lora_bwd(self._weights(), x, ids, x_ad, saved, dY, code),
                       "mok_lora_bwd", lambda: self._check(x, ids, x_ad, saved, dY, backward=True))
        return dict(zip(("dX", "dA", "dB", "dXa"), got))

    def status(self) -> int:
        """Waits for the current stream; 0, or MOK_ERR_TIMEOUT after a device wait expired."""
        with torch.cuda.device(self.device):
            return mok.mok_lora_get_status(self._status.data_ptr(),
                                           torch.cuda.current_stream().cuda_stream)

"""Infinities in the adapters' operands, on the GPU: results are infinite, with the right sign,
exactly where the formula's are (not NaN), and NaN where the formula's are NaN."""
import numpy as np
import pytest
import torch

from tests.test_gpu_lora import make, run

pytestmark = pytest.mark.gpu


def exact(v):
    """The values with no rounding error: multiples of 1/8 up to 2, none of them zero."""
    q = torch.clamp(torch.round(v.float() * 8), -16, 16)
    return torch.where(q == 0, 1.0, q).div(8).to(v.dtype)


def formula(x, W, A, B, scale, ids, dY):
    """u = scale x A^T, v = scale dY B^T; y = x W + u B, dX = dY W^T + v A, dA = v^T x, dB = u^T dY
    (ops_reference.lora multiplies by the scale last, which an infinite scale can tell apart)."""
    y, dX, dA, dB = x @ W, dY @ W.T, np.zeros(A.shape), np.zeros(B.shape)
    for a in range(len(A)):
        t = np.flatnonzero(ids == a)
        u, v = scale[a] * (x[t] @ A[a].T), scale[a] * (dY[t] @ B[a].T)
        y[t] += u @ B[a]
        dX[t] += v @ A[a]
        dA[a], dB[a] = v.T @ x[t], u.T @ dY[t]
    return {"y": y, "dX": dX, "dA": dA, "dB": dB}


@pytest.mark.parametrize("name,at", [("A", (1, 2, 7)), ("B", (1, 2, 5)), ("x", (1, 3)), ("dY", (1, 4)),
                                     ("scale", (1,))])
@pytest.mark.parametrize("T,r,two", [(5, 3, True), (5, 20, False), (300, 3, False), (300, 40, True),
                                     (300, 128, False)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinities_are_the_formulas(name, at, T, r, two, sign, rng):
    """Small exact values, so that u and v are exact in bf16 in part of the cases (two: only the
    first columns of A and B are not zero, a lo part of 0) and not in others."""
    c = make(rng, T, 64, 72, 2, r, "rows")
    c["ids"][:2] = 1
    for k in ("x", "A", "B", "dY"):
        c[k] = exact(c[k])
    c["scale"][:] = torch.tensor([0.5, 2.0])
    if two:       # sums of eight terms: exact in bf16
        c["A"][:, :, 8:] = 0.0
        c["B"][:, :, 8:] = 0.0
    c[name][at] = sign * float("inf")
    got = run(c, out=torch.float32)
    f = {k: v.double().numpy() for k, v in c.items() if k != "ids"}
    with np.errstate(invalid="ignore"):
        want = formula(ids=c["ids"].numpy(), **f)
    seen = 0
    for k in ("y", "dX", "dA", "dB"):
        g, w = got[k].double().cpu().numpy(), want[k]
        assert (np.isnan(g) == np.isnan(w)).all(), (k, np.isnan(g).sum(), np.isnan(w).sum())
        inf = np.isinf(w)
        assert (np.isinf(g) == inf).all() and (g[inf] == w[inf]).all(), k
        seen += inf.sum()
    assert seen > 0 or name == "scale"      # many ranks times inf: infinities of both signs, NaN

"""64-bit NumPy forms of the operators in include/mok_ops.h, for the tests: written from the
definitions, one token, adapter or counter at a time, sharing nothing with the kernels."""
import numpy as np


# ------------------------------------------------------------------------------ routing
def scores(l, score):
    """Scores of one token's logits (float64); masked logits (-inf, NaN) score 0."""
    l = np.asarray(l, np.float64).copy()
    l[np.isnan(l)] = -np.inf
    l[l == np.inf] = np.finfo(np.float32).max
    live = l > -np.inf
    s = np.zeros_like(l)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            s[live] = 1.0 / (1.0 + np.exp(-l[live]))
    elif live.any():
        e = np.exp(l[live] - l[live].max())
        s[live] = e / e.sum()
    return l, live, s


def choose(l, k, score, bias=None, groups=1, top_groups=1, group_score="max"):
    """The chosen ids of one token in slot order."""
    l, live, s = scores(l, score)
    E = len(l)
    graded = np.where(live, s + (0 if bias is None else np.asarray(bias, np.float64)), -np.inf)
    key = np.where(live, l, -np.inf) if score == "softmax" and bias is None else graded
    per = E // groups
    gs = []
    for g in range(groups):
        sl = slice(g * per, (g + 1) * per)
        if group_score == "max":
            gs.append(key[sl].max())
        else:
            best = sorted((v for v in graded[sl] if v > -np.inf), reverse=True)[:2]
            gs.append(sum(best) if best else -np.inf)
    kept = sorted(range(groups), key=lambda g: (-gs[g], g))[:top_groups]
    pool = [e for e in range(E) if e // per in kept]
    return sorted(pool, key=lambda e: (-key[e], e))[:k]


def gates(l, idx, score, renorm, scale):
    l, live, s = scores(l, score)
    if renorm and score == "softmax":      # the same ratios, without underflow
        c = l[idx]
        w = np.where(c > -np.inf, np.exp(c - c.max()), 0.0) if (c > -np.inf).any() else 0 * c
    else:
        w = s[idx]
    if renorm:
        w = w / w.sum() if w.sum() > 0 else 0 * w
    return scale * w


def gates_grad(l, idx, dg, score, renorm, scale):
    """d(sum_j dg_j gates_j) / d l through the Jacobian of the scores, choice fixed."""
    l, live, s = scores(l, score)
    sel = s[idx]
    if renorm:
        S = sel.sum()
        ds = (dg - (dg * sel).sum() / S) / S if S > 0 else np.zeros(len(idx))
    else:
        ds = np.asarray(dg, np.float64)
    J = np.diag(s * (1 - s)) if score == "sigmoid" else np.diag(s) - np.outer(s, s)
    return scale * (J[:, idx] @ ds)


# ------------------------------------------------------------------------------ dropout
def philox4x32(ctr, key, rounds=10):
    c, k = [int(v) for v in ctr], [int(v) for v in key]
    M = 2 ** 32
    for _ in range(rounds):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b // M) ^ c[1] ^ k[0], b % M, (a // M) ^ c[3] ^ k[1], a % M]
        k = [(k[0] + 0x9E3779B9) % M, (k[1] + 0xBB67AE85) % M]
    return c


def dropout_words(n, seed, offset):
    out = []
    for g in range((n + 7) // 8):
        ctr = (offset + g) % 2 ** 64
        for w in philox4x32([ctr % 2 ** 32, ctr // 2 ** 32, 0, 0], [seed % 2 ** 32, seed // 2 ** 32]):
            out += [w % 65536, w // 65536]
    return np.array(out[:n])


def dropout(x, p, seed, offset=0, add=None):
    t = round(p * 65536)
    keep = dropout_words(x.size, seed, offset).reshape(x.shape) >= t
    y = np.where(keep, x, 0.0) * (65536.0 / (65536 - t))
    return y if add is None else y + add


# ----------------------------------------------------------------------------- adapters
def lora(x, W, A, B, scale, ids, xa=None, dY=None):
    """Results and, for each, the same sums over absolute values (for error bounds)."""
    xa_ = x if xa is None else xa
    n = len(A)
    out = {"y": x @ W}
    mag = {"y": np.abs(x) @ np.abs(W)}
    if dY is not None:
        out.update(base=dY @ W.T, ad=np.zeros_like(x), dA=np.zeros(A.shape), dB=np.zeros(B.shape))
        mag.update(base=np.abs(dY) @ np.abs(W).T, ad=np.zeros_like(x), dA=np.zeros(A.shape),
                   dB=np.zeros(B.shape))
    for a in range(n):
        t = np.flatnonzero(ids == a)
        if not len(t):
            continue
        f, ab = float(scale[a]), np.abs
        out["y"][t] += f * ((xa_[t] @ A[a].T) @ B[a])
        mag["y"][t] += abs(f) * ((ab(xa_[t]) @ ab(A[a]).T) @ ab(B[a]))
        if dY is not None:
            out["ad"][t] = f * ((dY[t] @ B[a].T) @ A[a])
            mag["ad"][t] = abs(f) * ((ab(dY[t]) @ ab(B[a]).T) @ ab(A[a]))
            out["dA"][a] = f * ((dY[t] @ B[a].T).T @ xa_[t])
            mag["dA"][a] = abs(f) * ((ab(dY[t]) @ ab(B[a]).T).T @ ab(xa_[t]))
            out["dB"][a] = f * ((xa_[t] @ A[a].T).T @ dY[t])
            mag["dB"][a] = abs(f) * ((ab(xa_[t]) @ ab(A[a]).T).T @ ab(dY[t]))
    return out, mag

"""64-bit NumPy forms of the norm, the balance loss, the gradient norm and the AdamW step of
include/mok_ops.h, for the tests: written from the definitions, sharing nothing with the
kernels. The rounding of 8-bit moments, which is defined on fp32 bits, is done in fp32."""
import numpy as np

from tests.ops_reference import philox4x32, scores

U = 2.0 ** -24            # half a step of fp32, relative


# -------------------------------------------------------------------------------- norm
def norm(h, w, b, kind, eps):
    """(y, m, r) per row, float64."""
    h = np.asarray(h, np.float64)
    m = h.mean(1, keepdims=True) if kind == "layer" else np.zeros((len(h), 1))
    c = h - m
    with np.errstate(divide="ignore", invalid="ignore"):
        r = 1.0 / np.sqrt((c ** 2).mean(1, keepdims=True) + eps)
        y = c * r * w + (0.0 if b is None else b)
    return y, m, r


def norm_grad(h, w, dY, kind, eps):
    """(dX, dW, dB): dX through the Jacobian r (centring - xh xh^T / H) of each row."""
    _, m, r = norm(h, w, None, kind, eps)
    xh = (h - m) * r
    t = dY * w
    centred = t - t.mean(1, keepdims=True) if kind == "layer" else t
    dX = r * (centred - xh * (xh * t).mean(1, keepdims=True))
    return dX, (dY * xh).sum(0), dY.sum(0)


# ----------------------------------------------------------------------------- balance
def balance(logits, idx, score, coef, z_coef, seqs=None):
    """(losses, counts, dlosses[0]/dl, dlosses[1]/dl), one sequence and one row at a time."""
    T, E = logits.shape
    k = idx.shape[1]
    seqs = [0, T] if seqs is None else list(seqs)
    total = seqs[-1] - seqs[0]
    L, Z = 0.0, 0.0
    counts = np.zeros(E, np.int64)
    g0, g1 = np.zeros((T, E)), np.zeros((T, E))
    for lo, hi in zip(seqs, seqs[1:]):
        ids = idx[lo:hi].reshape(-1)
        c = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        counts += c
        for t in range(lo, hi):
            l, live, s = scores(logits[t], score)
            if not live.any():
                continue
            f = coef * E / (k * (hi - lo) * total) * c
            if score == "sigmoid" and s.sum() < 1e-30:      # the same ratios, without underflow
                s = np.where(live, np.exp(np.where(live, l, 0) - l[live].max()), 0.0)
                slope = s
            else:
                slope = s * (1 - s) if score == "sigmoid" else s
            S = s.sum()
            p = s / S
            L += p @ f
            if score == "sigmoid":
                g0[t] = slope / S * (f - p @ f)
            else:
                g0[t] = p * (f - p @ f)
            top = l[live].max()
            e = np.where(live, np.exp(np.where(live, l, top) - top), 0.0)
            lse = top + np.log(e.sum())
            Z += z_coef / total * lse ** 2
            g1[t] = 2 * z_coef / total * lse * e / e.sum()
    return np.array([L, Z]), counts, g0, g1


# ------------------------------------------------------------------------------- AdamW
def adamw(p, g, m, v, lr, beta1, beta2, eps, decay, t):
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    step = m / (1 - beta1 ** t) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p - lr * (step + decay * p), m, v


def e4m3_values():
    """The value of each E4M3 code (bias 7, no infinities, NaN at mantissa and exponent full)."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = (1 + f / 8) * 2.0 ** (e - 7) if e else f / 8 * 2.0 ** -6
        out[c] = np.nan if (c & 127) == 127 else -v if c & 128 else v
    return out


E4M3 = e4m3_values()


def moment_values(mc, vc, scales):
    """Values (float64) of codes [n] and scales [n / 256][2]."""
    a, b = (np.repeat(scales[:, i].astype(np.int64), 256) for i in (0, 1))
    c = vc.astype(np.int64)
    m = E4M3[mc] * 2.0 ** (a - 134.0)
    v = 2.0 ** (c // 8 - 30.0) * (1 + c % 8 / 8) * 2.0 ** (b - 127.0)
    return m, np.where(c > 0, v, 0.0)


def noise_words(first, n, seed, t):
    """16-bit words of positions first .. first + n - 1 (multiples of 8)."""
    out = []
    for q in range(first // 8, (first + n) // 8):
        for w in philox4x32([q % 2 ** 32, q // 2 ** 32, t % 2 ** 32, 0],
                            [seed % 2 ** 32, seed // 2 ** 32], rounds=7):
            out += [w % 65536, w // 65536]
    return np.array(out)


def random_code(x, word):
    """The code of 0 <= x < 256 rounded up or down by a 16-bit word, whose bits count in reverse
    order, the highest inverted. Codes are 2^20 apart: in the bits of an fp32 x from 2^-6 on, in
    steps of 2^-29 (those of x + 2^-6) below."""
    f, least = np.float32, np.float32(2.0 ** -6)
    if x < least:
        place = int((f(x) + least).view(np.uint32)) - (121 << 23)
    else:
        place = int(f(x).view(np.uint32)) - (120 << 23)
    u = int(f"{int(word):016b}"[::-1], 2) ^ 0x8000
    return (place + (u << 4)) >> 20


def moment_codes(m, v, words, beta1=0.9):
    """(codes of m, codes of v, scales) of fp32 moments [n], n a multiple of 256."""
    m, v = np.asarray(m, np.float32), np.asarray(v, np.float32)
    mc, vc = np.zeros(len(m), np.uint8), np.zeros(len(v), np.uint8)
    scales = np.zeros((len(m) // 256, 2), np.uint8)
    finite = E4M3[:127]                                   # codes 0 .. 126, ascending
    for blk in range(len(m) // 256):
        s = slice(256 * blk, 256 * blk + 256)
        ok = np.isfinite(m[s]) & np.isfinite(v[s])

        def field(x):
            top = np.where(ok, np.abs(x), 0).max().astype(np.float32)
            return int(top.view(np.uint32)) >> 23

        a, b = max(field(m[s]), 8), max(field(v[s]), 31)
        scales[blk] = a, b
        for i in range(256 * blk, 256 * blk + 256):
            if not ok[i - 256 * blk]:
                mc[i], vc[i] = 127, 255
                continue
            x = abs(float(m[i])) * 2.0 ** (134 - a)
            at = int(np.searchsorted(finite, x))          # finite[at - 1] < x <= finite[at]
            if at > 0 and (at == 127 or x - finite[at - 1] < finite[at] - x or
                           (x - finite[at - 1] == finite[at] - x and (at - 1) % 2 == 0)):
                at -= 1
            if beta1 > 0.9 or x < 2.0 ** -6:
                at = random_code(x, words[i])
            mc[i] = at + (128 if np.signbit(m[i]) else 0)
            if v[i] > 0:
                # the position among the codes, in steps of 2^-20 of a code
                steps = int(v[i].view(np.int32)) - ((b - 30) << 23)
                vc[i] = min(max((steps + (int(words[i]) << 4)) >> 20, 1), 255)
    return mc, vc, scales

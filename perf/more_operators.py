"""Timed cases of what a training step needs around the MoE layer: the norm before a block,
the router's balance loss, the norm of all gradients, and the AdamW step that applies them.

Every case runs in two forms on the same inputs: the plain form (``own = False``), made of
elementary torch operations in 32 bits and rounded once at the end, and the library's
kernels (``own = True``), called the way a training or serving program calls them.
``exact`` evaluates the definitions in 64 bits, separately from both.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BF16, F32, F64, I32, I64, U8 = (torch.bfloat16, torch.float32, torch.float64, torch.int32,
                                torch.int64, torch.uint8)
_TYPES = {"bf16": BF16, "fp32": F32}


# ------------------------------------------------------------------------------- cases
def listed():
    def norm(name, T, H, kind, x="bf16", y="bf16", w="bf16", add=True, bias=False, train=False):
        return dict(name=name, op="norm", T=T, H=H, kind=kind, x=x, y=y, w=w, add=add, bias=bias,
                    train=train)

    def balance(name, T, E, k, score, seqs=0, pad=0, coef=1e-2, z=0.0, dtype="fp32", add=False):
        return dict(name=name, op="balance", T=T, E=E, k=k, score=score, seqs=seqs, pad=pad,
                    coef=coef, z=z, dtype=dtype, add=add)

    def clip(name, tensors, lo, hi, shapes, dtype):
        return dict(name=name, op="clip", tensors=tensors, lo=lo, hi=hi, shapes=shapes, g=dtype)

    def adamw(name, tensors, lo, hi, shapes, bits, p, g):
        return dict(name=name, op="adamw", tensors=tensors, lo=lo, hi=hi, shapes=shapes,
                    bits=bits, p=p, g=g)

    return [
        # one generated token: residual sum and RMS norm before a block, latency only
        norm("norm_token", 1, 7168, "rms"),
        # a training batch: residual sum and norm forward, the backward with the gradient that
        # comes along the residual stream
        norm("norm_train", 8192, 7168, "rms", train=True),
        # a layer norm with bias of odd width, fp32 stream, a ragged batch
        norm("norm_train_odd", 2371, 1031, "layer", x="fp32", y="fp32", w="fp32", add=False,
             bias=True, train=True),
        # a micro-batch of one short prompt: the loss and its gradient, latency only
        balance("balance_small", 128, 256, 8, "sigmoid"),
        # packed documents, each balanced by itself, padding behind the last; the gradient is
        # added to the one that comes through the gates
        balance("balance_packed", 16384, 256, 8, "sigmoid", seqs=24, pad=301, add=True),
        # a large batch as one set, with the penalty on large logits
        balance("balance_batch", 65536, 384, 8, "softmax", z=1e-3, dtype="bf16"),
        # gradients of the adapters of a few projections
        clip("clip_adapters", 12, 40_000, 900_000, 3, "bf16"),
        # gradients of eight experts' three matrices
        clip("clip_experts", 24, 7168 * 2048, 7168 * 2048, 0, "bf16"),
        # a router's bias, norm weights and other small fp32 tensors: latency
        adamw("adamw_small", 9, 60, 7168, 5, 32, "fp32", "fp32"),
        # eight experts' three matrices in mixed precision, fp32 states
        adamw("adamw_experts", 24, 7168 * 2048, 7168 * 2048, 0, 32, "bf16", "bf16"),
        # the same matrices with states in 8 bits
        adamw("adamw_experts8", 24, 7168 * 2048, 7168 * 2048, 0, 8, "bf16", "bf16"),
        # many tensors of odd sizes with states in 8 bits, fp32 weights and gradients
        adamw("adamw_odd8", 60, 33, 400_000, 9, 8, "fp32", "fp32"),
    ]


def _log_int(rng, lo, hi):
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
        if lo <= v <= hi:
            return v


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["norm", "norm", "balance", "balance", "clip", "adamw", "adamw"])
    if op == "norm":
        x = rng.choice(["bf16", "fp32"])
        return dict(op=op, T=_log_int(rng, 1, 8192), H=_log_int(rng, 64, 7168) if x == "fp32"
                    else 8 * _log_int(rng, 8, 896) + rng.choice([0, 0, 0, 1]),
                    kind=rng.choice(["rms", "layer"]), x=x, y=rng.choice(["bf16", x]),
                    w=rng.choice(["bf16", "fp32"]), add=rng.random() < 0.6,
                    bias=rng.random() < 0.4, train=rng.random() < 0.6)
    if op == "balance":
        T = _log_int(rng, 1, 65536)
        seqs = rng.choice([0, 0, _log_int(rng, 1, 64)])
        return dict(op=op, T=T, E=_log_int(rng, 8, 512), k=rng.randint(1, 8),
                    score=rng.choice(["sigmoid", "softmax"]), seqs=seqs,
                    pad=rng.randint(0, T // 4) if seqs else 0, coef=1e-2,
                    z=rng.choice([0.0, 1e-3]), dtype=rng.choice(["fp32", "bf16"]),
                    add=rng.random() < 0.5)
    tensors = _log_int(rng, 1, 200)
    hi = _log_int(rng, 64, min(16_000_000, 300_000_000 // tensors))
    case = dict(op=op, tensors=tensors, lo=max(1, hi // rng.choice([1, 10, 1000])), hi=hi,
                shapes=rng.randint(1, 10**6))
    if op == "clip":
        return dict(case, g=rng.choice(["bf16", "fp32"]))
    p = rng.choice(["bf16", "fp32"])
    return dict(case, bits=rng.choice([8, 32]), p=p, g=rng.choice([p, "fp32"]))


def _sizes(case):
    """The tensors' sizes, spread over the logarithm of lo .. hi."""
    r = random.Random(case["shapes"])
    return [_log_int(r, case["lo"], case["hi"]) for _ in range(case["tensors"])]


def work(case):
    """Bytes (each input read once, each output written once) and operations of a pass."""
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "norm":
        n, x, y, w = case["T"] * case["H"], size[case["x"]], size[case["y"]], size[case["w"]]
        params = case["H"] * w * (2 if case["bias"] else 1)
        b = n * (x * (3 if case["add"] else 1) + y) + params
        if case["train"]:
            b += n * (y + x * (2 if case["add"] else 1)) + params
        return {"bytes": b, "flops": n * (20 if case["train"] else 8)}
    if case["op"] == "balance":
        n, s = case["T"] * case["E"], size[case["dtype"]]
        b = n * s * (3 if case["add"] else 2) + 4 * case["T"] * case["k"] + 4 * case["E"]
        return {"bytes": b, "flops": 16 * n}
    n = sum(_sizes(case))
    if case["op"] == "clip":
        return {"bytes": n * size[case["g"]], "flops": 2 * n}
    b = size[case["g"]] + 8 + (2 if case["p"] == "bf16" else 0) + (4 if case["bits"] == 8 else 16)
    if case["bits"] == 8:
        b += 4                        # the moments' values, which a pass returns
    return {"bytes": n * b, "flops": 16 * n}


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=F32, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _prepare_norm(case, g, st):
    T, H, xt, wt = case["T"], case["H"], _TYPES[case["x"]], _TYPES[case["w"]]
    st.update(x=_normal(g, (T, H), 1.0, xt), add=_normal(g, (T, H), 2.0, xt) if case["add"] else None,
              w=(1.0 + _normal(g, (H,), 0.2, F32)).to(wt),
              b=_normal(g, (H,), 0.2, wt) if case["bias"] else None, eps=1e-5)
    if case["train"]:
        st.update(dY=_normal(g, (T, H), 1.0, _TYPES[case["y"]]),
                  dh=_normal(g, (T, H), 1.0, xt) if case["add"] else None)
    if own:
        from grouped_gemm_built_gb300.norm import Norm
        st["handle"] = Norm(st["w"], st["b"], kind=case["kind"], eps=st["eps"])


def _prepare_balance(case, g, st, seed):
    T, E, k, dt = case["T"], case["E"], min(case["k"], case["E"]), _TYPES[case["dtype"]]
    logits = (_normal(g, (T, E), 1.5, F32) + _normal(g, (E,), 0.5, F32)).to(dt)
    idx = torch.argsort(logits.float(), dim=1, descending=True, stable=True)[:, :k]
    st.update(logits=logits, idx=idx.to(I32).contiguous(), seqs=None,
              add=_normal(g, (T, E), 1e-4, dt) if case["add"] else None)
    if case["seqs"]:
        r = random.Random(seed)
        last = T - case["pad"]
        cuts = sorted(r.randint(0, last) for _ in range(case["seqs"] - 1))
        st["seqs"] = torch.tensor([0] + cuts + [last], dtype=I32).cuda()
    if own:
        from grouped_gemm_built_gb300.balance import Balance
        st["handle"] = Balance(E, k, score=case["score"], coef=case["coef"], z_coef=case["z"])


_BLOCK = 256          # elements that share the scales of 8-bit states


def _prepare_tensors(case, g, st):
    """One buffer of gradients, each tensor at the next whole block: the views, where they
    start, and how many elements the buffer has."""
    sizes = _sizes(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // _BLOCK) * _BLOCK
    used = torch.zeros(total, dtype=torch.bool, device="cuda")
    for at, n in zip(starts, sizes):
        used[at:at + n] = True
    # gradients of a layer's matrices: small, a spread of scales over rows of a matrix
    rows = torch.exp(_normal(g, (total // _BLOCK, 1), 1.0, F32)) * 1e-3
    grad = (_normal(g, (total // _BLOCK, _BLOCK), 1.0, F32) * rows).reshape(-1)
    grad = torch.where(used, grad, 0.0).to(_TYPES[case["g"]])
    st.update(grad=grad, grads=[grad[at:at + n] for at, n in zip(starts, sizes)])
    return sizes, starts, total, used, rows


def _prepare_adamw(case, g, st):
    sizes, starts, total, used, rows = _prepare_tensors(case, g, st)
    blocks = total // _BLOCK
    master = torch.where(used, _normal(g, (total,), 0.02, F32), 0.0)
    p = master.to(_TYPES[case["p"]])
    params = [p[at:at + n] for at, n in zip(starts, sizes)]
    # matrices decay, the smallest tensors (norm weights, biases) do not
    most = max(sizes)
    decay = [0.0 if n < 100 else 0.1 if n * 4 > most else 0.05 for n in sizes]
    m = torch.where(used, (_normal(g, (blocks, _BLOCK), 0.3, F32) * rows).reshape(-1), 0.0)
    v = torch.exp(_normal(g, (blocks, _BLOCK), 0.7, F32)) * rows * rows
    v = torch.where(used, v.reshape(-1), 0.0)
    st.update(p=p, master=master if case["p"] == "bf16" else None, lr=3e-4, betas=(0.9, 0.95),
              eps=1e-8, seed=20240607, step=100,
              coef=torch.tensor([0.75], device="cuda"))
    if case["bits"] == 8:
        noise = torch.zeros(total, dtype=I32, device="cuda")
        st["m"], st["v"], st["scales"] = _plain_encode(m, v, noise)
    else:
        st["m"], st["v"], st["scales"] = m, v, None
    if own:
        from grouped_gemm_built_gb300.optim import AdamW
        opt = AdamW(params, betas=st["betas"], eps=st["eps"], weight_decay=decay,
                    bits=case["bits"], seed=st["seed"])
        opt.steps = st["step"]
        for name in ("master", "m", "v", "scales"):
            if st[name] is not None:
                getattr(opt, name).copy_(st[name])
                st[name] = None
        st["handle"] = opt
    else:
        of = torch.zeros(blocks, 1, dtype=F32, device="cuda")
        for at, n, d in zip(starts, sizes, decay):
            of[at // _BLOCK:-(-(at + n) // _BLOCK)] = d
        st["decay"] = of


def prepare(case, seed):
    """Inputs made from the seed, and the handles that a program keeps between calls."""
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "norm":
        _prepare_norm(case, g, st)
    elif case["op"] == "balance":
        _prepare_balance(case, g, st, seed)
    elif case["op"] == "clip":
        _prepare_tensors(case, g, st)
        st["max_norm"] = 1.0
    else:
        _prepare_adamw(case, g, st)
    return st


# --------------------------------------------------------------------- the plain forms
def _plain_norm(case, st):
    h = st["x"]
    if case["add"]:
        h = (h.float() + st["add"].float()).to(h.dtype)
    hf, w = h.float(), st["w"].float()
    if case["kind"] == "layer":
        hf = hf - hf.mean(-1, keepdim=True)
    r = torch.rsqrt((hf * hf).mean(-1, keepdim=True) + st["eps"])
    xh = hf * r
    y = xh * w
    if case["bias"]:
        y = y + st["b"].float()
    out = {"y": y.to(_TYPES[case["y"]])}
    if case["add"]:
        out["h"] = h
    if case["train"]:
        dY = st["dY"].float()
        t = dY * w
        dx = t - xh * (t * xh).mean(-1, keepdim=True)
        if case["kind"] == "layer":
            dx = dx - t.mean(-1, keepdim=True)
        dx = dx * r
        if case["add"]:
            dx = dx + st["dh"].float()
        out["dX"] = dx.to(h.dtype)
        out["dW"] = (dY * xh).sum(0).to(st["w"].dtype)
        if case["bias"]:
            out["dB"] = dY.sum(0).to(st["w"].dtype)
    return out


def _plain_balance(case, st):
    logits, idx = st["logits"], st["idx"].long()
    T, E = logits.shape
    k, rows = idx.shape[1], torch.arange(T, device="cuda")
    if st["seqs"] is None:
        ends = torch.tensor([0, T], device="cuda")
    else:
        ends = st["seqs"].long()
    S = ends.numel() - 1
    mine = (rows[:, None] >= ends[None, :]).sum(1) - 1           # S: behind the last sequence
    valid = mine < S
    mine = torch.where(valid, mine, S)
    counts = torch.zeros((S + 1) * E, dtype=F32, device="cuda")
    counts.index_add_(0, (mine[:, None] * E + idx).reshape(-1),
                      torch.ones(T * k, dtype=F32, device="cuda"))
    counts = counts.reshape(S + 1, E)
    length = (ends[1:] - ends[:-1]).float()
    total = length.sum()
    factor = case["coef"] * E / (k * length.clamp(min=1.0) * total.clamp(min=1.0))
    factor = torch.cat([factor, factor.new_zeros(1)])
    l = logits.float()
    top = l.amax(-1, keepdim=True)
    e = torch.exp(l - top)
    z = e.sum(-1, keepdim=True)
    soft, lse = e / z, top + torch.log(z)
    if case["score"] == "softmax":
        p, slope = soft, soft
    else:
        s = 1.0 / (1.0 + torch.exp(-l))
        whole = s.sum(-1, keepdim=True)
        p, slope = s / whole, s / (1.0 + torch.exp(l)) / whole
    # the counts relative to their mean, an integer: the gradient is the same, without cancellation
    mean = torch.floor(counts.sum(-1, keepdim=True) / E)
    upstream = (counts - mean)[mine] * factor[mine][:, None]
    dl = slope * (upstream - (p * upstream).sum(-1, keepdim=True))
    loss = ((p * counts[mine]).sum(-1) * factor[mine]).sum()
    scale = torch.where(valid, case["z"] / total.clamp(min=1.0), 0.0)[:, None]
    loss_z = (scale * lse * lse).sum()
    if case["z"]:
        dl = dl + 2.0 * scale * lse * soft
    if case["add"]:
        dl = dl + st["add"].float()
    return {"losses": torch.stack([loss, loss_z]), "counts": counts[:S].sum(0).to(I32),
            "dlogits": dl.to(logits.dtype)}


def _plain_clip(case, st):
    """Elements between the tensors are 0."""
    g = st["grad"].float()
    norm = torch.sqrt((g * g).sum())
    return {"norm": norm.reshape(1), "coef": torch.clamp(st["max_norm"] / norm, max=1.0).reshape(1)}


def _plain_words(count, seed, step):
    """Random 16-bit numbers, eight per counter: Philox4x32 with 7 rounds (Salmon et al.,
    "Parallel random numbers: as easy as 1, 2, 3", 2011) of (position, step), keyed by the seed."""
    m32 = 0xFFFFFFFF
    at = torch.arange(count // 8, device="cuda")
    c0, c1, c2, c3 = at & m32, at >> 32, torch.full_like(at, step & m32), torch.zeros_like(at)
    k0, k1 = seed & m32, (seed >> 32) & m32
    for _ in range(7):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & m32) ^ c1 ^ k0, p1 & m32,
                          ((p0 >> 32) & m32) ^ c3 ^ k1, p0 & m32)
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    halves = [h for w in (c0, c1, c2, c3) for h in (w & 0xFFFF, w >> 16)]
    return torch.stack(halves, -1).reshape(-1).to(I32)


def _plain_decode(m, v, scales):
    """m: E4M3 times 2^(a - 134); v: 5 bits of exponent and 3 of mantissa, counted from
    2^(b - 157); a, b: the exponent fields that a block's scales hold."""
    a, b = scales[:, 0:1].to(I32), scales[:, 1:2].to(I32)
    mf = m.view(torch.float8_e4m3fn).float().reshape(-1, _BLOCK)
    mf = mf * ((a - 7) << 23).view(F32)
    c = v.reshape(-1, _BLOCK).to(I32)
    vf = torch.where(c > 0, ((c << 20) + ((b - 30) << 23)).view(F32), 0.0)
    return mf.reshape(-1), vf.reshape(-1)


def _plain_encode(m, v, noise):
    m, v = m.reshape(-1, _BLOCK), v.reshape(-1, _BLOCK)
    a = (m.abs().amax(1, keepdim=True).view(I32) >> 23).clamp(min=8)
    b = (v.amax(1, keepdim=True).view(I32) >> 23).clamp(min=31)
    codes = (m * ((261 - a) << 23).view(F32)).to(torch.float8_e4m3fn).view(U8)
    # rounded up with the probability that the cut-off bits stand for; never to 0 from above
    c = (v.view(I32) - ((b - 30) << 23) + (noise.reshape(-1, _BLOCK) << 4)) >> 20
    c = torch.where(v > 0, c.clamp(1, 255), 0)
    return codes.reshape(-1), c.to(U8).reshape(-1), torch.cat([a, b], 1).to(U8)


def _plain_adamw(case, st):
    st["step"] += 1
    (b1, b2), t = st["betas"], st["step"]
    p = st["p"] if st["master"] is None else st["master"]
    g = st["grad"].float() * st["coef"]
    small = case["bits"] == 8
    m, v = _plain_decode(st["m"], st["v"], st["scales"]) if small else (st["m"], st["v"])
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + (g * g) * (1.0 - b2)
    denom = torch.sqrt(v) * (1.0 / math.sqrt(1.0 - b2 ** t)) + st["eps"]
    keep = (1.0 - st["lr"] * st["decay"])
    new = (p.reshape(-1, _BLOCK) * keep).reshape(-1) - (st["lr"] / (1.0 - b1 ** t)) * (m / denom)
    p.copy_(new)
    out = {"p": st["p"]}
    if st["master"] is not None:
        st["p"].copy_(new)
        out["master"] = st["master"]
    if small:
        codes = _plain_encode(m, v, _plain_words(m.numel(), st["seed"], t))
        for name, c in zip(("m", "v", "scales"), codes):
            st[name].copy_(c)
        m, v = _plain_decode(st["m"], st["v"], st["scales"])
        out["m"], out["v"] = m.to(BF16), v.to(BF16)      # 4 significant bits: exact
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
        out["m"], out["v"] = st["m"], st["v"]
    return out


# ------------------------------------------------------------------ the library's calls
def _own_norm(case, st):
    y, h, stats = st["handle"].forward(st["x"], add=st["add"], out=_TYPES[case["y"]])
    out = {"y": y}
    if case["add"]:
        out["h"] = h
    if case["train"]:
        out.update(st["handle"].backward(st["dY"], h, stats, add=st["dh"]))
    return out


def _own_balance(case, st):
    losses, counts, saved = st["handle"].forward(st["logits"], st["idx"], st["seqs"])
    dlogits = st["handle"].backward(st["logits"], saved, st["seqs"], add=st["add"])
    return {"losses": losses, "counts": counts, "dlogits": dlogits}


def _own_clip(case, st):
    from grouped_gemm_built_gb300.optim import grad_norm
    norm, coef = grad_norm(st["grads"], max_norm=st["max_norm"])
    return {"norm": norm, "coef": coef}


def _own_adamw(case, st):
    opt = st["handle"]
    opt.step(st["grads"], lr=st["lr"], coef=st["coef"])
    out = {"p": st["p"]}
    if case["p"] == "bf16":
        out["master"] = opt.master
    out["m"], out["v"] = opt.moments()
    return out


def run(state):
    """ONE pass through the state's operator."""
    case = state["case"]
    forms = {"norm": (_plain_norm, _own_norm), "balance": (_plain_balance, _own_balance),
             "clip": (_plain_clip, _own_clip), "adamw": (_plain_adamw, _own_adamw)}
    return forms[case["op"]][1 if own else 0](case, state)


# ------------------------------------------------------------------ 64-bit definitions
def _exact_norm(case, st):
    """From the means and the Jacobian of x / sqrt(mean x^2 + eps), in float64."""
    h = st["x"].to(F64)
    if case["add"]:
        h = (st["x"].to(F64) + st["add"].to(F64)).to(F32).to(st["x"].dtype).to(F64)
    H, w = case["H"], st["w"].to(F64)
    c = h - h.sum(1, keepdim=True) / H if case["kind"] == "layer" else h
    var = (c ** 2).sum(1, keepdim=True) / H + st["eps"]
    out = {"y": c / var.sqrt() * w}
    if case["bias"]:
        out["y"] = out["y"] + st["b"].to(F64)
    if case["add"]:
        out["h"] = h
    if case["train"]:
        dY = st["dY"].to(F64)
        dc = dY * w / var.sqrt() - c * (dY * w * c).sum(1, keepdim=True) / (H * var ** 1.5)
        dx = dc - dc.sum(1, keepdim=True) / H if case["kind"] == "layer" else dc
        out["dX"] = dx + st["dh"].to(F64) if case["add"] else dx
        out["dW"] = (dY * (c / var.sqrt())).sum(0)
        if case["bias"]:
            out["dB"] = dY.sum(0)
    return out


def _exact_balance(case, st):
    """Sequence by sequence: the share of the choices times the mean score of each expert."""
    l, idx = st["logits"].to(F64), st["idx"].cpu().long()
    T, E = l.shape
    k = idx.shape[1]
    ends = [0, T] if st["seqs"] is None else st["seqs"].tolist()
    total = ends[-1] - ends[0]
    losses, counts = [0.0, 0.0], torch.zeros(E, dtype=I64)
    dl = torch.zeros_like(l) if st["add"] is None else st["add"].to(F64).clone()
    for lo, hi in zip(ends, ends[1:]):
        if hi == lo:
            continue
        c = torch.bincount(idx[lo:hi].reshape(-1), minlength=E)
        counts += c
        x = l[lo:hi].clone().requires_grad_(True)
        score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
        p = score / score.sum(1, keepdim=True)
        share = c.to(F64).cuda() / (k * (hi - lo))
        a = case["coef"] * E * (share * p.mean(0)).sum() * ((hi - lo) / total)
        z = case["z"] * (torch.logsumexp(x, 1) ** 2).sum() / total
        losses[0] += float(a)
        losses[1] += float(z)
        dl[lo:hi] += torch.autograd.grad(a + z, x)[0]
    return {"losses": torch.tensor(losses, dtype=F64).cuda(), "counts": counts.to(I32).cuda(),
            "dlogits": dl}


def _exact_clip(case, st):
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g, dtype=F64)) ** 2 for g in st["grads"]))
    factor = min(1.0, st["max_norm"] / norm) if norm else 1.0
    return {"norm": torch.tensor([norm], dtype=F64), "coef": torch.tensor([factor], dtype=F64)}


def _exact_adamw(case, st):
    """The textbook step with bias-corrected moments. Moments in 8 bits have no value in 64:
    their rounding goes by the bits of the 32-bit result."""
    (b1, b2), t, lr = st["betas"], st["step"] + 1, st["lr"]
    g = st["grad"].to(F64) * float(st["coef"])
    m, v = st["m"], st["v"]
    if case["bits"] == 8:
        scale = torch.exp2(st["scales"].to(F64) - 127.0).repeat_interleave(_BLOCK, 0)
        m = st["m"].view(torch.float8_e4m3fn).to(F64) * scale[:, 0] / 128.0
        c = st["v"].to(I64)
        v = torch.exp2((c // 8 - 30).to(F64)) * (1.0 + (c % 8).to(F64) / 8.0) * scale[:, 1]
        v = torch.where(c > 0, v, 0.0)
    m = b1 * m.to(F64) + (1.0 - b1) * g
    v = b2 * v.to(F64) + (1.0 - b2) * g * g
    p = (st["p"] if st["master"] is None else st["master"]).to(F64)
    step = (m / (1.0 - b1 ** t)) / ((v / (1.0 - b2 ** t)).sqrt() + st["eps"])
    p = p - lr * (step + st["decay"].to(F64).expand(-1, _BLOCK).reshape(-1) * p)
    out = {"p": p, "m": m, "v": v}
    if st["master"] is not None:
        out["master"] = p
    if case["bits"] == 8:
        out["m"] = out["v"] = None
    return out


def exact(case, seed):
    """What ``run`` returns, from the operators' definitions in 64 bits."""
    global own
    mode, own = own, False          # the inputs alone, without the library's handles
    try:
        st = prepare(case, seed)
    finally:
        own = mode
    forms = {"norm": _exact_norm, "balance": _exact_balance, "clip": _exact_clip,
             "adamw": _exact_adamw}
    return forms[case["op"]](case, st)

"""Timed cases of the operators around the MoE layer: routing to experts, low-rank adapters
beside a shared projection, and counter-based dropout.

Every case runs in two forms on the same inputs: the plain form (``own = False``), made of
elementary torch operations in 32 bits and rounded once at the end, and the library's
kernels (``own = True``), called the way a training or serving program calls them.
``exact`` evaluates the definitions in 64 bits, separately from both.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
_TYPES = {"bf16": BF16, "fp32": F32}


# ------------------------------------------------------------------------------- cases
def listed():
    def route(name, T, E, k, score, renorm, groups=1, top_groups=1, group_score="max",
              bias=False, scale=1.0, dtype="fp32", train=False):
        return dict(name=name, op="route", T=T, E=E, k=k, score=score, renorm=renorm,
                    groups=groups, top_groups=top_groups, group_score=group_score, bias=bias,
                    scale=scale, dtype=dtype, train=train)

    def lora(name, T, K, N, n, r, order, train=False, p=0.0):
        return dict(name=name, op="lora", T=T, K=K, N=N, n=n, r=r, order=order, train=train, p=p)

    def drop(name, rows, cols, p, add, dtype):
        return dict(name=name, op="dropout", rows=rows, cols=cols, p=p, add=add, dtype=dtype)

    return [
        # one generated token through a 384-expert router: latency only
        route("route_token", 1, 384, 8, "softmax", True),
        # a decode batch through a router with expert groups and a balance bias
        route("route_decode", 64, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # the same router over a long prefill or a training batch's forward
        route("route_prefill", 16384, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5),
        # a training step of a 384-expert router whose gates stay unnormalised: every
        # expert's logit has a gradient; bf16 logits, so equal logits occur
        route("route_train", 8192, 384, 8, "softmax", False, dtype="bf16", train=True),
        # a ragged training batch, an expert count that is no power of two
        route("route_train_odd", 2371, 60, 6, "sigmoid", True, 6, 3, "max", True, 1.0,
              train=True),
        # one token of one request: the up projection of a shared expert with its adapter
        lora("lora_token", 1, 7168, 2048, 8, 16, "rows"),
        # a decode batch, every row a request with an adapter of its own or none
        lora("lora_decode", 96, 2048, 7168, 48, 16, "rows"),
        # a prefill batch: a dozen prompts of uneven length packed one after another
        lora("lora_prefill", 8192, 7168, 2048, 12, 32, "packed"),
        # one training step for the adapters of four tenants, base weights frozen
        lora("lora_train", 8192, 7168, 2048, 4, 16, "packed", train=True),
        # odd everything: rank 5, sizes off every tile, shuffled rows, adapter dropout
        lora("lora_train_odd", 1003, 1032, 520, 7, 5, "rows", train=True, p=0.1),
        # residual dropout over a full training batch
        drop("dropout_train", 8192, 7168, 0.1, True, "bf16"),
        # a small fp32 activation whose size is no multiple of a vector
        drop("dropout_small", 333, 1031, 0.25, False, "fp32"),
    ]


def _cost(case):
    w = work(case)
    return w["flops"] / 1.9e15 + w["bytes"] / 6.8e12


def _log_int(rng, lo, hi):
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))
        if lo <= v <= hi and v != 3072:
            return v


def draw(rng):
    """One more case of the ranges that the listed ones stand for."""
    op = rng.choice(["route", "route", "lora", "lora", "lora", "dropout"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 6, 8])
        per = _log_int(rng, 2, 512 // groups)
        if groups * per < 8:
            per = 8
        E = groups * per
        top_groups = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(8, top_groups * per))
        return dict(op=op, T=_log_int(rng, 1, 16384), E=E, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6,
                    groups=groups, top_groups=top_groups,
                    group_score=rng.choice(["max", "top2"]), bias=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "bf16"]),
                    train=rng.random() < 0.5)
    if op == "dropout":
        return dict(op=op, rows=_log_int(rng, 1, 8192), cols=_log_int(rng, 64, 7168),
                    p=rng.choice([0.05, 0.1, 0.25, 0.5]), add=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "fp32"]))
    most = max(_cost(c) for c in listed() if c["op"] == "lora")
    while True:
        K, N = (8 * _log_int(rng, 16, 896) for _ in range(2))
        case = dict(op=op, T=_log_int(rng, 1, 8192), K=K, N=N, n=_log_int(rng, 1, 48),
                    r=_log_int(rng, 1, 64), order=rng.choice(["rows", "packed"]),
                    train=rng.random() < 0.4, p=rng.choice([0.0, 0.0, 0.1]))
        if not case["train"]:
            case["p"] = 0.0
        if K != 3072 and N != 3072 and _cost(case) <= most:
            return case


def work(case):
    """Bytes (each input read once, each output written once) and operations of a pass."""
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        es = 2 if case["dtype"] == "bf16" else 4
        b = T * E * es + T * k * 8 + (4 * E if case["bias"] else 0)
        f = T * E * 6
        if case["train"]:
            b += T * k * 4 + T * E * es       # upstream gate gradients in, logit gradients out
            f += T * E * 4
        return {"bytes": b, "flops": f}
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * es * (3 if case["add"] else 2), "flops": 2 * n}
    T, K, N, n, r = (case[c] for c in "TKNnr")
    used = min(n, T)
    b = 2 * (T * K + K * N + used * r * (K + N) + T * N) + 4 * T
    f = 2 * T * K * N + 2 * T * r * (K + N)
    if case["train"]:
        b += 2 * (T * N + T * K + n * r * (K + N))          # dY in; dX, dA, dB out
        f += 2 * T * K * N + 4 * T * r * (K + N)
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype):
    return torch.empty(shape, dtype=F32, device="cuda").normal_(0.0, std, generator=g).to(dtype)


def _near_ties(case, logits, bias):
    """Rows in which two choice scores (or two group scores) that decide the routing differ,
    but by less than 32-bit arithmetic resolves: their experts are not defined to 32 bits."""
    if case["score"] == "softmax" and bias is None and (
            case["groups"] == 1 or case["group_score"] == "max"):
        return torch.zeros(case["T"], dtype=torch.bool, device="cuda")   # logits compare exactly
    l = logits.to(F64)
    c = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, -1)
    if bias is not None:
        c = c + bias.to(F64)
    elif case["score"] == "softmax":
        c = c.log()                 # selected on the logits: only the groups compare sums
    bad = torch.zeros(case["T"], dtype=torch.bool, device="cuda")
    G = case["groups"]

    def close(v, count):
        top = v.sort(-1, descending=True).values[:, :count + 1]
        gap = top[:, :-1] - top[:, 1:]
        return ((gap > 0) & (gap < 4e-6 * top.abs().amax(-1, keepdim=True).clamp(min=1e-3))).any(-1)

    if G > 1 and case["top_groups"] < G:
        per = c.reshape(case["T"], G, -1)
        s = per.exp() if (bias is None and case["score"] == "softmax") else per
        n = min(2 if case["group_score"] == "top2" else 1, s.shape[-1])
        gs = s.sort(-1, descending=True).values[..., :n].sum(-1)
        bad |= close(gs, case["top_groups"])
        kept = torch.sort(gs, dim=-1, descending=True, stable=True).indices
        kept = kept[:, :case["top_groups"]]
        live = torch.zeros_like(gs, dtype=torch.bool).scatter_(1, kept, True)
        c = per.masked_fill(~live[..., None], -1e9).reshape(case["T"], -1)
    if not (bias is None and case["score"] == "softmax"):
        n = min(case["k"], c.shape[1] - 1)
        bad |= close(c, n) if n > 0 else False
    return bad


def prepare(case, seed):
    """Inputs made from the seed, and the handles that a program keeps between calls."""
    g = _gen(seed)
    st = {"case": case}
    if case["op"] == "route":
        T, E, dt = case["T"], case["E"], _TYPES[case["dtype"]]
        tilt = _normal(g, (E,), 0.5, F32)                       # some experts are busier
        bias = (-0.1 * tilt + _normal(g, (E,), 0.01, F32)) if case["bias"] else None
        logits = (_normal(g, (T, E), 1.5, F32) + tilt).to(dt)
        for _ in range(8):
            bad = _near_ties(case, logits, bias)
            fresh = (_normal(g, (T, E), 1.5, F32) + tilt).to(dt)
            logits = torch.where(bad[:, None], fresh, logits)
        st.update(logits=logits, bias=bias,
                  dgates=_normal(g, (T, case["k"]), 1.0, F32) if case["train"] else None)
        if own:
            from grouped_gemm_built_gb300.routing import Routing
            st["handle"] = Routing(E, case["k"], score=case["score"], groups=case["groups"],
                                   top_groups=case["top_groups"],
                                   group_score=case["group_score"],
                                   renormalize=case["renorm"], scale=case["scale"])
        return st
    if case["op"] == "dropout":
        shape, dt = (case["rows"], case["cols"]), _TYPES[case["dtype"]]
        st.update(x=_normal(g, shape, 1.0, dt), seed=(seed * 0x9E3779B9 + 12345) % 2**63,
                  add=_normal(g, shape, 1.0, dt) if case["add"] else None)
        return st
    T, K, N, n, r = (case[c] for c in "TKNnr")
    rnd = torch.Generator().manual_seed(seed)
    if case["order"] == "rows":              # every row its own request; -1: no adapter
        ids = torch.randint(0, n, (T,), generator=rnd)
        ids[torch.rand(T, generator=rnd) < 0.125] = -1
    else:                                    # prompts packed one after another
        m = max(1, min(T, n))
        cuts = torch.sort(torch.randint(0, T + 1, (m - 1,), generator=rnd)).values.tolist()
        ids = torch.empty(T, dtype=torch.int64)
        for a, (lo, hi) in enumerate(zip([0] + cuts, cuts + [T])):
            ids[lo:hi] = a
        if m > 4:
            ids[ids == 1] = -1               # one prompt runs on the base model
    st.update(x=_normal(g, (T, K), 1.0, BF16), W=_normal(g, (K, N), 0.02, BF16),
              A=_normal(g, (n, r, K), 0.02, BF16), B=_normal(g, (n, r, N), 0.02, BF16),
              scale=0.5 + 1.5 * torch.rand(n, generator=g, device="cuda"),
              ids=ids.to(torch.int32).cuda(), seed=(seed * 7919 + 17) % 2**63,
              dY=_normal(g, (T, N), 1.0, BF16) if case["train"] else None)
    if own:
        from grouped_gemm_built_gb300.lora import AdaptedLinear
        st["handle"] = AdaptedLinear(st["W"], st["A"], st["B"], st["scale"])
    return st


# --------------------------------------------------------------------- the plain forms
def _plain_philox(counters, seed):
    """Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011):
    four 32-bit words per counter, as int64 tensors."""
    m32 = 0xFFFFFFFF
    c0, c1 = counters & m32, (counters >> 32) & m32
    c2 = torch.zeros_like(c0)
    c3 = torch.zeros_like(c0)
    k0, k1 = seed & m32, (seed >> 32) & m32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & m32) ^ c1 ^ k0, p1 & m32,
                          ((p0 >> 32) & m32) ^ c3 ^ k1, p0 & m32)
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    return c0, c1, c2, c3


def _plain_keep(shape, p, seed):
    """Dropout's mask: 16 random bits per element, kept where they reach 65536 p."""
    n = math.prod(shape)
    words = _plain_philox(torch.arange((n + 7) // 8, device="cuda"), seed)
    halves = [h for w in words for h in (w & 0xFFFF, w >> 16)]
    u = torch.stack(halves, -1).reshape(-1)[:n].reshape(shape)
    t = round(p * 65536)
    return u >= t, 65536.0 / (65536 - t)


def _plain_choice(case, logits, bias):
    """Scores in 32 bits, and the scores the experts are chosen by."""
    l = logits.float()
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
        c = s
    else:
        e = torch.exp(l - l.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
        c = l if bias is None else s
    return s, c if bias is None else c + bias, s if bias is None else s + bias


def _plain_first_max(v):
    """Index of the largest entry of each row, the lowest where several are equal."""
    where = torch.arange(v.shape[-1], device=v.device).expand_as(v)
    return torch.where(v == v.amax(-1, keepdim=True), where, v.shape[-1]).amin(-1, keepdim=True)


def _plain_route(case, logits, bias):
    s, c, graded = _plain_choice(case, logits, bias)
    T, E, G = case["T"], case["E"], case["groups"]
    low = -float("inf")
    if G > 1:
        per = (graded if case["group_score"] == "top2" else c).reshape(T, G, E // G)
        gs = per.amax(-1)
        if case["group_score"] == "top2" and E // G > 1:
            first = _plain_first_max(per)
            gs = gs + per.scatter(-1, first, low).amax(-1)
        live = torch.zeros(T, G, dtype=torch.bool, device=c.device)
        for _ in range(case["top_groups"]):
            live.scatter_(1, _plain_first_max(gs), True)
            gs = torch.where(live, low, gs)
        c = torch.where(live[..., None], c.reshape(T, G, E // G), low).reshape(T, E)
    chosen = []
    for _ in range(case["k"]):
        i = _plain_first_max(c)
        chosen.append(i)
        c = c.scatter(1, i, low)
    idx = torch.cat(chosen, 1)
    if case["renorm"] and case["score"] == "softmax":
        l = logits.float().gather(1, idx)
        w = torch.exp(l - l.amax(-1, keepdim=True))
    else:
        w = s.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return s, idx, w


def _plain_route_pass(case, st):
    s, idx, w = _plain_route(case, st["logits"], st["bias"])
    out = {"topk_idx": idx.to(torch.int32), "gates": w * case["scale"]}
    if case["train"]:
        dg = st["dgates"] * case["scale"]
        if case["renorm"]:
            d = w * (dg - (w * dg).sum(-1, keepdim=True))
            if case["score"] == "sigmoid":
                d = d / (1.0 + torch.exp(st["logits"].float().gather(1, idx)))
            full = torch.zeros_like(s).scatter_(1, idx, d)
        elif case["score"] == "sigmoid":
            d = dg * w / (1.0 + torch.exp(st["logits"].float().gather(1, idx)))
            full = torch.zeros_like(s).scatter_(1, idx, d)
        else:
            full = torch.zeros_like(s).scatter_(1, idx, dg)
            full = s * (full - (w * dg).sum(-1, keepdim=True))
        out["dlogits"] = full.to(st["logits"].dtype)
    return out


def _plain_lora_pass(case, st):
    """Every row against every adapter, the pairs that do not belong together set to zero:
    the same sums without a host round trip over the rows of each adapter."""
    n, r = case["n"], case["r"]
    x, W = st["x"].float(), st["W"].float()
    A, B = st["A"].float().reshape(n * r, -1), st["B"].float().reshape(n * r, -1)
    mine = torch.arange(n, device="cuda")[None, :] == st["ids"][:, None]          # [T, n]
    factor = torch.where(mine, st["scale"][None, :], 0.0).repeat_interleave(r, 1)  # [T, n r]
    xa = x
    if case["p"] > 0:
        keep, up = _plain_keep(x.shape, case["p"], st["seed"])
        xa = torch.where(keep, x * up, 0.0)
    u = (xa @ A.t()) * factor
    out = {"y": (x @ W + u @ B).to(BF16)}
    if case["train"]:
        dY = st["dY"].float()
        v = (dY @ B.t()) * factor
        back = v @ A
        if case["p"] > 0:
            back = torch.where(keep, back * up, 0.0)
        out["dX"] = (dY @ W.t() + back).to(BF16)
        out["dA"] = (v.t() @ xa).reshape(n, r, -1).to(BF16)
        out["dB"] = (u.t() @ dY).reshape(n, r, -1).to(BF16)
    return out


def _plain_dropout_pass(case, st):
    keep, up = _plain_keep(st["x"].shape, case["p"], st["seed"])
    y = torch.where(keep, st["x"].float() * up, 0.0)
    if st["add"] is not None:
        y = y + st["add"].float()
    return y.to(st["x"].dtype)


# ------------------------------------------------------------------ the library's calls
def _own_route_pass(case, st):
    h = st["handle"]
    idx, gates = h.forward(st["logits"], st["bias"])
    out = {"topk_idx": idx, "gates": gates}
    if case["train"]:
        out["dlogits"] = h.backward(st["logits"], idx, st["dgates"])
    return out


def _own_lora_pass(case, st):
    from grouped_gemm_built_gb300.dropout import dropout
    h, x, ids = st["handle"], st["x"], st["ids"]
    xa = dropout(x, case["p"], st["seed"]) if case["p"] > 0 else None
    y, saved = h.forward(x, ids, x_ad=xa)
    out = {"y": y}
    if case["train"]:
        g = h.backward(x, ids, saved, st["dY"], x_ad=xa)
        out.update(dX=g["dX"], dA=g["dA"], dB=g["dB"])
        if xa is not None:
            out["dX"] = dropout(g["dXa"], case["p"], st["seed"], add=g["dX"])
    return out


def _own_dropout_pass(case, st):
    from grouped_gemm_built_gb300.dropout import dropout
    return dropout(st["x"], case["p"], st["seed"], add=st["add"])


def run(state):
    """ONE pass through the state's operator."""
    case = state["case"]
    forms = {"route": (_plain_route_pass, _own_route_pass),
             "lora": (_plain_lora_pass, _own_lora_pass),
             "dropout": (_plain_dropout_pass, _own_dropout_pass)}
    return forms[case["op"]][1 if own else 0](case, state)


# ------------------------------------------------------------------ 64-bit definitions
def _exact_keep(n, p, seed):
    u32, u64 = np.uint32, np.uint64
    ctr = np.arange((n + 7) // 8, dtype=u64)
    c = [(ctr & u64(0xFFFFFFFF)).astype(u32), (ctr >> u64(32)).astype(u32),
         np.zeros(ctr.shape, u32), np.zeros(ctr.shape, u32)]
    k = [seed % 2**32, (seed // 2**32) % 2**32]
    for _ in range(10):
        a = c[0].astype(u64) * u64(0xD2511F53)
        b = c[2].astype(u64) * u64(0xCD9E8D57)
        ahi, alo = (a >> u64(32)).astype(u32), a.astype(u32)
        bhi, blo = (b >> u64(32)).astype(u32), b.astype(u32)
        c = [bhi ^ c[1] ^ u32(k[0]), blo, ahi ^ c[3] ^ u32(k[1]), alo]
        k = [(k[0] + 0x9E3779B9) % 2**32, (k[1] + 0xBB67AE85) % 2**32]
    words = np.stack(c, 1).astype("<u4")
    u = words.view("<u2").reshape(-1)[:n]
    return torch.from_numpy(u.astype(np.int32) >= round(p * 65536))


def _exact_route(case, st):
    """Row by row from the definition, in numpy: groups, choice, gates, gradient."""
    if case["T"] * case["E"] > 2**23:
        return None
    l = st["logits"].to(F64).cpu().numpy()
    bias = None if st["bias"] is None else st["bias"].to(F64).cpu().numpy()
    T, E = l.shape
    G, P, k = case["groups"], E // case["groups"], case["k"]
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + np.exp(-l))
    else:
        s = np.exp(l - l.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    biased = s if bias is None else s + bias
    key = l if (bias is None and case["score"] == "softmax") else biased
    live = np.ones((T, E), bool)
    if G > 1:
        if case["group_score"] == "max":
            gs = key.reshape(T, G, P).max(2)
        else:
            gs = np.sort(biased.reshape(T, G, P), axis=2)[:, :, -2:].sum(2)
        best = np.argsort(-gs, axis=1, kind="stable")[:, :case["top_groups"]]
        lg = np.zeros((T, G), bool)
        np.put_along_axis(lg, best, True, 1)
        live = np.repeat(lg, P, axis=1)
    order = np.argsort(np.where(live, -key, np.inf), axis=1, kind="stable")[:, :k]
    sel = np.take_along_axis(s, order, 1)
    gates = sel / sel.sum(1, keepdims=True) if case["renorm"] else sel
    out = {"topk_idx": torch.from_numpy(order.astype(np.int32)).cuda(),
           "gates": torch.from_numpy(gates * case["scale"]).cuda()}
    if case["train"]:
        # d gate_j / d score_i, then d score / d logit, as whole matrices per row
        dg = st["dgates"].to(F64).cpu().numpy() * case["scale"]
        if case["renorm"]:
            ds = (dg - (dg * gates).sum(1, keepdims=True)) / sel.sum(1, keepdims=True)
        else:
            ds = dg
        dS = np.zeros((T, E))
        np.put_along_axis(dS, order, ds, 1)
        if case["score"] == "sigmoid":
            dl = dS * s * (1.0 - s)
        else:
            dl = s * (dS - (dS * s).sum(1, keepdims=True))
        out["dlogits"] = torch.from_numpy(dl).cuda()
    return out


def _exact_lora(case, st):
    """Adapter by adapter over the rows that use it, in float64."""
    x, W, ids = st["x"].to(F64), st["W"].to(F64), st["ids"].cpu()
    xa = x
    if case["p"] > 0:
        t = round(case["p"] * 65536)
        mask = _exact_keep(x.numel(), case["p"], st["seed"]).reshape(x.shape).cuda()
        mask = mask.to(F64) * (65536.0 / (65536 - t))
        xa = x * mask
    y = x @ W
    out = {"y": y}
    if case["train"]:
        dY = st["dY"].to(F64)
        back = torch.zeros_like(x)
        out.update(dX=dY @ W.t(), dA=torch.zeros(st["A"].shape, dtype=F64, device="cuda"),
                   dB=torch.zeros(st["B"].shape, dtype=F64, device="cuda"))
    for a in range(case["n"]):
        rows = torch.nonzero(ids == a).flatten().cuda()
        if rows.numel() == 0:
            continue
        f, A, B = float(st["scale"][a]), st["A"][a].to(F64), st["B"][a].to(F64)
        low = xa[rows] @ A.t()
        y[rows] += f * (low @ B)
        if case["train"]:
            low_dy = dY[rows] @ B.t()
            back[rows] = f * (low_dy @ A)
            out["dA"][a] = f * (low_dy.t() @ xa[rows])
            out["dB"][a] = f * (low.t() @ dY[rows])
    if case["train"]:
        out["dX"] += back * mask if case["p"] > 0 else back
    return out


def exact(case, seed):
    """What ``run`` returns, from the operators' definitions in 64 bits."""
    st = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, st)
    if case["op"] == "lora":
        return _exact_lora(case, st)
    t = round(case["p"] * 65536)
    keep = _exact_keep(st["x"].numel(), case["p"], st["seed"]).reshape(st["x"].shape).cuda()
    y = st["x"].to(F64) * (65536.0 / (65536 - t)) * keep
    return y if st["add"] is None else y + st["add"].to(F64)

"""mok_route and mok_route_bwd on the GPU against the 64-bit form in ops_reference.py.

Logits lie on a grid of 1/16 and biases on a grid of 1/8 (both exact in bf16), with scores
drawn again until the scores that decide a choice are either equal inputs (a tie, which must
go to the lower id) or at least 1e-5 apart, far above fp32's 6e-8 per operation: the chosen
ids must then be equal. Gates and gradients are a few fp32 operations on values of relative
error 2^-22 (exp to 2 ulp, a sum of at most 512 terms in a tree): 1e-5 relative to the largest
value of the row bounds them with room; bf16 gradients add half a step, 2^-8 relative."""
import numpy as np
import pytest
import torch

from grouped_gemm_built_gb300.routing import Routing
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu

RULES = [
    dict(E=1, k=1),
    dict(E=8, k=2),
    dict(E=33, k=5, score="sigmoid"),
    dict(E=60, k=6, score="sigmoid", groups=6, top_groups=3, bias=True),
    dict(E=64, k=6, renormalize=False, scale=2.5),
    dict(E=96, k=8, groups=8, top_groups=3, group_score="top2"),
    dict(E=100, k=32, score="sigmoid", renormalize=False, groups=4, top_groups=2),
    dict(E=256, k=8, score="sigmoid", groups=8, top_groups=4, group_score="top2", bias=True,
         scale=2.5),
    dict(E=256, k=8, bias=True, renormalize=False),
    dict(E=384, k=8),
    dict(E=500, k=7, groups=4, top_groups=4, bias=True),
    dict(E=512, k=8, score="sigmoid", groups=32, top_groups=5, group_score="top2"),
    dict(E=32, k=4, groups=32, top_groups=7, group_score="top2", score="sigmoid", bias=True),
]


def defined(l, c):
    """The choice is defined to 32 bits: scores of the choice equal or 1e-5 apart."""
    def apart(v, n):
        v = np.sort(v)[::-1][:n + 1]
        gap = v[:-1] - v[1:]
        return bool(np.all((gap == 0) | (gap > 1e-5)))

    s = ref.scores(l, c["score"])[2]
    b = c["bias_values"]
    if c["score"] == "softmax" and b is None:
        if c["groups"] == 1 or c["group_score"] == "max":
            return True
    v = s if b is None else s + b
    per = v.reshape(c["groups"], -1)
    n = 2 if c["group_score"] == "top2" else 1
    ok = apart(np.sort(per, 1)[:, -n:].sum(1), c["top_groups"]) if c["groups"] > 1 else True
    if c["score"] == "softmax" and b is None:
        return ok
    kept = ref.choose(l, c["top_groups"] * per.shape[1], c["score"], b, c["groups"],
                      c["top_groups"], c["group_score"])
    return ok and apart(v[kept], c["k"])


def draw(rng, T, c):
    rows = []
    while len(rows) < T:
        l = np.round(rng.normal(0, 1.5, c["E"]) * 16) / 16
        if defined(l, c):
            rows.append(l)
    return np.array(rows)


def full(rule, rng):
    c = dict(score="softmax", groups=1, top_groups=1, group_score="max", renormalize=True,
             scale=1.0, bias=False)
    c.update(rule)
    c["bias_values"] = np.round(rng.normal(0, 0.3, c["E"]) * 8) / 8 if c["bias"] else None
    R = Routing(c["E"], c["k"], score=c["score"], groups=c["groups"], top_groups=c["top_groups"],
                group_score=c["group_score"], renormalize=c["renormalize"], scale=c["scale"])
    return c, R


def cuda(a, dtype=torch.float32):
    return None if a is None else torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


@pytest.mark.parametrize("rule", RULES, ids=lambda r: "-".join(f"{v}" for v in r.values()))
@pytest.mark.parametrize("T,dtype", [(1, torch.float32), (67, torch.bfloat16)])
def test_choice_gates_and_gradient(rule, T, dtype, rng):
    c, R = full(rule, rng)
    l = draw(rng, T, c)
    dg = rng.normal(size=(T, c["k"])).astype(np.float32)
    logits = cuda(l, dtype)
    idx, gates = R.forward(logits, cuda(c["bias_values"]))
    dl = R.backward(logits, idx, cuda(dg)).float().cpu().numpy()
    wide = R.backward(logits, idx, cuda(dg), dtype=torch.float32).cpu().numpy()
    narrow = R.backward(logits, idx, cuda(dg), dtype=torch.bfloat16).float().cpu().numpy()
    idx, gates = idx.cpu().numpy(), gates.cpu().numpy()
    for t in range(T):
        want = ref.choose(l[t], c["k"], c["score"], c["bias_values"], c["groups"],
                          c["top_groups"], c["group_score"])
        assert list(idx[t]) == want
        g = ref.gates(l[t], want, c["score"], c["renormalize"], c["scale"])
        assert np.abs(gates[t] - g).max() <= 1e-5 * np.abs(g).max()
        d = ref.gates_grad(l[t], want, dg[t].astype(np.float64), c["score"], c["renormalize"],
                           c["scale"])
        tol = 1e-5 * c["scale"] * np.abs(dg[t]).max()
        assert np.abs(wide[t] - d).max() <= tol
        assert (np.abs(narrow[t] - d) <= tol + 2.0 ** -8 * np.abs(d)).all()
        assert (np.abs(dl[t] - d) <= tol + 2.0 ** -8 * np.abs(d)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_come_last_with_gate_zero(score):
    """-inf and NaN mask; with fewer unmasked experts than slots the lowest masked ids fill up
    with gate 0, a fully masked row gives ids 0..k-1 and gates 0; +inf does not make NaN."""
    E, k, inf, nan = 40, 4, float("inf"), float("nan")
    l = torch.full((4, E), -inf)
    l[0, [39, 7]] = torch.tensor([1.0, 2.0])
    l[1] = nan
    l[2, 5], l[2, 11] = inf, 3.0
    l[3] = torch.linspace(-1, 1, E)
    l[3, 39] = nan
    dg = torch.tensor([[1.0, 2.0, inf, nan]] * 4)
    dg[2:] = torch.tensor([1.0, -2.0, 0.5, 0.25])
    for renorm in (True, False):
        R = Routing(E, k, score=score, renormalize=renorm)
        idx, g = R.forward(l.cuda())
        assert idx[0].tolist() == [7, 39, 0, 1] and idx[1].tolist() == [0, 1, 2, 3]
        assert idx[2].tolist() == [5, 11, 0, 1] and idx[3].tolist() == [38, 37, 36, 35]
        assert torch.isfinite(g).all() and (g[0, 2:] == 0).all() and (g[1] == 0).all()
        for t in (0, 2, 3):
            want = ref.gates(l[t].double().numpy(), idx[t].tolist(), score, renorm, 1.0)
            assert np.abs(g[t].cpu().numpy() - want).max() <= 1e-5
        dl = R.backward(l.cuda(), idx, dg.cuda())
        assert torch.isfinite(dl).all()
        assert (dl[0, [0, 1, 2]] == 0).all() and (dl[1] == 0).all() and dl[3, 39] == 0


def test_equal_logits_go_to_the_lower_id_and_signed_zeros_are_equal():
    l = torch.zeros(2, 64)
    l[0, ::2] = -0.0
    l[1, [60, 3, 31, 32]] = 5.0
    for score in ("softmax", "sigmoid"):
        idx, _ = Routing(64, 5, score=score).forward(l.cuda())
        assert idx.tolist() == [[0, 1, 2, 3, 4], [3, 31, 32, 60, 0]]


def test_extreme_logits_keep_renormalised_gates():
    """All chosen probabilities underflow in fp32, their ratios do not (a bias makes the choice
    leave the largest logits)."""
    l = torch.full((1, 32), -400.0)
    l[0, 0] = 0.0
    bias = torch.zeros(32)
    bias[[4, 9]] = 5.0
    l[0, 9] = -401.0
    idx, g = Routing(32, 2).forward(l.cuda(), bias.cuda())
    want = np.array([1.0, np.exp(-1.0)]) / (1 + np.exp(-1.0))
    assert idx.tolist() == [[4, 9]] and np.abs(g.cpu().numpy()[0] - want).max() < 1e-6


def test_ids_outside_the_experts_have_no_gradient():
    R = Routing(48, 3)
    l = torch.randn(5, 48, device="cuda")
    idx, _ = R.forward(l)
    bad = idx.clone()
    bad[:, 1] = torch.tensor([-1, 48, 2**31 - 1, -2**31, 4096], device="cuda", dtype=torch.int32)
    dl = R.backward(l, bad, torch.ones(5, 3, device="cuda"))
    assert torch.isfinite(dl).all() and (dl != 0).sum(1).max() <= 2


def test_repeats_bitwise_and_follows_the_current_stream():
    R = Routing(256, 8, score="sigmoid", groups=8, top_groups=4, group_score="top2", scale=2.5)
    side = torch.cuda.Stream()
    l = torch.randn(3001, 256, device="cuda")
    b = torch.randn(256, device="cuda") * 0.1
    first = R.forward(l, b)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)          # a result that ran elsewhere would come too early
        l2 = l * 1.0
        again = R.forward(l2, b)
    side.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_row_offsets_past_32_bits():
    T, E = 4_300_000, 512                      # 2.2e9 logits
    l = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    l[-1, 500], l[-1, 7] = 3.0, 2.0
    R = Routing(E, 2, renormalize=False)
    idx, _ = R.forward(l)
    dl = R.backward(l, idx, torch.ones(T, 2, device="cuda"))
    assert idx[-1].tolist() == [500, 7] and idx[-2].tolist() == [0, 1]
    want = ref.gates_grad(l[-1].double().cpu().numpy(), [500, 7], np.ones(2), "softmax", False, 1.0)
    assert np.abs(dl[-1].float().cpu().numpy() - want).max() <= 1e-5 + 2.0 ** -8 * np.abs(want).max()

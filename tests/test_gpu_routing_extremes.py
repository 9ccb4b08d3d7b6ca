"""Routing at logits far from zero, on the GPU, against the 64-bit form in ops_reference.py."""
import numpy as np
import pytest
import torch

from grouped_gemm_built_gb300.routing import Routing
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("top", [-10.0, -16.5, -17.5, -60.0, -86.0, -95.0, -150.0, -1e4])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_renormalised_sigmoid_gates_of_very_negative_logits(top, dtype):
    """Scores that are tiny in fp32, or 0, have ratios that are not. The logits of a row are `top`,
    and lower by 0.5 or 3 (by 64 and 128 at -1e4, where bf16's step is 64). Per gate: the scores to
    3 ulp each (2^-22 relative), a sum of three and a quotient: 2^-20. Gradients: sums of products
    of such gates with |dg| <= 1, 2^-19 of the scale."""
    E, k, scale = 40, 3, 2.5
    l = torch.full((1, E), -float("inf"))
    steps = [0.0, 0.5, 3.0] if top > -1e3 else [0.0, 64.0, 128.0]
    if dtype == torch.bfloat16 and top != -1e4:
        steps = [0.0, 1.0, 3.0]
    l[0, [31, 4, 17]] = torch.tensor([top - s for s in steps])
    l = l.to(dtype)
    x = l[0].double().numpy()
    # the same order as the scores', whichever way the choice compares them
    bias = torch.zeros(E)
    bias[[31, 4, 17]] = torch.tensor([3.0, 2.0, 1.0])
    R = Routing(E, k, score="sigmoid", scale=scale)
    idx, g = R.forward(l.cuda(), bias.cuda())
    assert idx.tolist() == [[31, 4, 17]]
    with np.errstate(over="ignore"):
        want = ref.gates(np.maximum(x, -700), [31, 4, 17], "sigmoid", True, scale)
    if top == -1e4:       # e^-64 and e^-128 of the largest
        want = np.array([scale, scale * np.exp(-64.0), 0.0])
    assert np.abs(g[0].cpu().numpy() - want).max() <= 2.0 ** -20 * scale
    dg = torch.tensor([[1.0, -0.5, 0.75]])
    dl = R.backward(l.cuda(), idx, dg.cuda(), dtype=torch.float32)[0].cpu().numpy()
    w = want / scale
    d = scale * w * (dg[0].double().numpy() - (w * dg[0].double().numpy()).sum())
    d = d / (1 + np.exp(x[[31, 4, 17]]))
    assert np.abs(dl[[31, 4, 17]] - d).max() <= 2.0 ** -19 * scale
    assert np.count_nonzero(np.delete(dl, [31, 4, 17])) == 0


@pytest.mark.parametrize("rule", [dict(k=5), dict(k=3, groups=8, top_groups=3),
                                  dict(k=4, groups=6, top_groups=2, E=60)])
@pytest.mark.parametrize("around", [[17.5, 20.0, 24.0, 18.0, 30.0, 22.0, 19.0],
                                    [-96.0, -91.0, -105.0, -100.0, -93.0, -88.5, -110.0]])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sigmoid_without_a_bias_keeps_the_order_of_its_logits(rule, around, dtype, rng):
    """Logits whose fp32 scores are all 1, or all 0, are still in order; the rest lies below."""
    E = rule.get("E", 64)
    rule = {k: v for k, v in rule.items() if k != "E"}
    for trial in range(8):
        l = np.full(E, min(around) - 8.0)
        l[rng.choice(E, len(around), replace=False)] = around
        logits = torch.tensor(l[None], dtype=dtype)
        assert (logits[0].double().numpy() == l).all()
        idx, _ = Routing(E, score="sigmoid", **rule).forward(logits.cuda())
        want = ref.choose(l, rule["k"], "softmax", None, rule.get("groups", 1),
                          rule.get("top_groups", 1), "max")     # softmax compares the logits
        assert idx[0].tolist() == want


def choice_score_errors(score, logits, bias, at, other):
    """For each exact score s of expert `at` in the rows of logits: does the choice between it and
    expert `other`, whose own score is 0 and whose bias is s off by 8 ulp, go the right way?"""
    wrong = []
    for l in logits:
        x = ref.scores(l.double().numpy(), score)[2][at]
        R = Routing(len(l), 1, score=score)
        for off, first in ((1 - 2.0 ** -20, at), (1 + 2.0 ** -20, other)):
            b = bias.clone()
            b[other] = float(np.float32(x * off))
            idx, _ = R.forward(l[None].cuda(), b.cuda())
            if idx.item() != first:
                wrong.append((l[at].item(), off))
    return wrong


def test_sigmoid_choice_scores_are_good_to_a_few_ulp(rng):
    """exp to 1 ulp, a sum to half, a quotient to 2: 3.5 ulp, where 8 (2^-20) decide."""
    at = torch.tensor(rng.uniform(-24.0, 6.0, 400), dtype=torch.float32)
    logits = torch.stack([at, torch.full((400,), -200.0)], 1)
    assert choice_score_errors("sigmoid", logits, torch.zeros(2), 0, 1) == []


def test_softmax_choice_scores_are_good_to_a_few_ulp(rng):
    """exp to 1 ulp, a sum of two terms and its inverse to half an ulp each, a product to half:
    2.5 ulp and the sum's share of exp's, where 8 (2^-20) decide. The largest logit is 0, so the
    differences are exact; a bias keeps its expert out of the choice."""
    at = torch.tensor(rng.uniform(-60.0, -1.0, 400), dtype=torch.float32)
    logits = torch.stack([torch.zeros(400), at, torch.full((400,), -200.0)], 1)
    assert choice_score_errors("softmax", logits, torch.tensor([-10.0, 0.0, 0.0]), 1, 2) == []


def test_dense_gradient_of_unchosen_experts_is_good_to_a_few_ulp(rng):
    """dl_e = -scale s_e sum_S s dg for e outside S: two of them have the ratio of their scores.
    Each entry is an exp to 1 ulp and two products to half an ulp, a ratio at most 2 x 2 ulp (2^-23
    each) off: 4 x 2^-23 and their products, so 2^-20 with room. Logits on a grid of 1/16 and a
    largest one of 0 make the differences exact; reference entry: the largest unchosen one."""
    E, k = 384, 2
    l = np.round(rng.uniform(-80.0, -2.0, E) * 16) / 16
    l[[7, 200]] = 0.0, -0.5
    l[100] = -1.0
    R = Routing(E, k, renormalize=False, scale=1.0)
    logits = torch.tensor(l[None], dtype=torch.float32, device="cuda")
    idx, _ = R.forward(logits)
    assert idx.tolist() == [[7, 200]]
    # 2^40: the smallest products stay normal numbers
    dl = R.backward(logits, idx, torch.full((1, k), 2.0 ** 40, device="cuda"))[0].double().cpu().numpy()
    rest = [e for e in range(E) if e not in (7, 200)]
    want = np.exp(l[rest] - l[100])
    assert np.abs(dl[rest] / dl[100] / want - 1).max() <= 2.0 ** -20


def test_the_largest_row_count():
    """T is an int: rows up to 2^31 - 1 are counted without overflow."""
    T = 2 ** 31 - 1
    l = torch.zeros(T, 1, dtype=torch.bfloat16, device="cuda")
    R = Routing(1, 1, renormalize=False, scale=0.5)
    idx, g = R.forward(l)
    assert (idx[-4:] == 0).all() and (g[-4:] == 0.5).all() and (g[:4] == 0.5).all()
    assert g.amin() == 0.5 and g.amax() == 0.5
    del idx, g
    torch.cuda.empty_cache()
    some = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    dl = R.backward(l, some, torch.ones(T, 1, device="cuda"))
    assert dl.abs().amax() == 0           # one expert: its softmax is 1 whatever the logit

"""How many digits the balance loss and the penalty keep where logits are large, or a row's log sum
of exponentials is near 0.

Bounds, u = 2^-24. One row's loss is a multiple of one score p = s / sum s. An exponential of x is
off by 6 u + |x| u / 20 (2 ulp of the instruction, two roundings, the constants' last bits), 9.5 u for
|x| <= 70; a sigmoid by 4 u more (sum, reciprocal). The sum of 8 adds 6 u, its reciprocal and the
product with it 3 u, counts and factor 3 u: 2 9.5 + 12 = 31 u, sigmoids 39 u. With one product with
log2 e in place of two the exponentials are off by up to 63 u.
A row with one logit l that counts has log sum e^l = l: the penalty's l^2 z / T is off by 4 u, its
gradient 2 z l / T by 6 u."""
import numpy as np
import pytest
import torch

from grouped_gemm_built_gb300.balance import Balance

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("centre", [0.0, 5.0, 20.0, 40.0, 60.0, 66.0, -5.0, -10.0, -20.0, -40.0, -60.0])
@pytest.mark.parametrize("rows", [1, 1100])
def test_loss_of_large_logits(score, centre, rows):
    """One row, by itself or as a sequence of its own among rows of no sequence: the two kernels."""
    B = Balance(8, 1, score=score, coef=0.125)
    g = torch.Generator().manual_seed(int(centre) + 100)
    bound = (31 if score == "softmax" else 39) * U
    for _ in range(100 if rows == 1 else 20):
        l = (torch.randn(rows, 8, generator=g) + centre).to(F32)
        x = l[0].double().numpy()
        s = np.exp(x - x.max()) if score == "softmax" else np.exp(-np.logaddexp(0, -x))
        c = int(s.argmin())
        idx = torch.full((rows, 1), c, dtype=torch.int32)
        seqs = None if rows == 1 else torch.tensor([0, 1], dtype=torch.int32).cuda()
        losses, _, _ = B.forward(l.cuda(), idx.cuda(), seqs)
        want = s[c] / s.sum()
        assert abs(float(losses[0]) - want) <= bound * want


@pytest.mark.parametrize("E", [1, 8, 40])
@pytest.mark.parametrize("rows", [1, 1100])
def test_penalty_of_a_sum_near_one(E, rows):
    for l0 in (1e-4, -1e-3, 0.01, 0.3, -0.6, 0.69):
        l = torch.full((rows, E), -50.0)
        l[:, E // 2] = l0
        l0 = float(l[0, E // 2])
        idx = torch.full((rows, 1), E // 2, dtype=torch.int32).cuda()
        seqs = None if rows == 1 else torch.tensor([0, 1], dtype=torch.int32).cuda()
        for score in ("softmax", "sigmoid"):
            B = Balance(E, 1, score=score, coef=0.0, z_coef=0.5)
            losses, _, saved = B.forward(l.cuda(), idx, seqs)
            assert abs(float(losses[1]) - 0.5 * l0 * l0) <= 4 * U * 0.5 * l0 * l0
            dl = B.backward(l.cuda(), saved, seqs)
            assert abs(float(dl[0, E // 2]) - l0) <= 6 * U * abs(l0)


@pytest.mark.parametrize("E", [8, 40, 250])
def test_masked_logits_beside_large_ones(E):
    """-inf, NaN and the row's end are 0 in the same pass: the losses are those of the row without them,
    to the bounds above for both; gradients of the masked ones are 0."""
    g = torch.Generator().manual_seed(E)
    l = torch.randn(300, E, generator=g) * 4
    idx = torch.randint(0, E, (300, 2), generator=g, dtype=torch.int32).cuda()
    for value in (-float("inf"), float("nan")):
        for score in ("softmax", "sigmoid"):
            B = Balance(E, 2, score=score, coef=1.0, z_coef=0.1)
            masked, low = l.clone(), l.clone()
            masked[:, 1::3], low[:, 1::3] = value, -500.0       # e^-500 is below every sum's last bit
            a, b = B.forward(masked.cuda(), idx), B.forward(low.cuda(), idx)
            torch.testing.assert_close(a[0], b[0], rtol=80 * U, atol=0)
            ga, gb = B.backward(masked.cuda(), a[2]), B.backward(low.cuda(), b[2])
            assert not ga[:, 1::3].any() and ga.isfinite().all()
            torch.testing.assert_close(ga, gb, rtol=2e-5, atol=float(gb.abs().max()) * 80 * U)

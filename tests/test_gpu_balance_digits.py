"""How many digits the penalty on large logits keeps where a row's log sum of exponentials is near 0.

u = 2^-24. A row with one logit l that counts has log sum e^l = l: the penalty's l^2 z / T is off by
4 u, its gradient 2 z l / T by 6 u."""
import pytest
import torch

from grouped_gemm_built_gb300.balance import Balance

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


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

"""The largest number of rows, with values that every row shows in."""
import pytest
import torch

from grouped_gemm_built_gb300.balance import Balance

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_no_row_of_the_longest_batch_is_lost():
    """One expert, logits of 1: each row adds 1 to the loss's sum and (log e)^2 = 1 to the penalty's.
    A term is off by 24 u at most (exponential 6 u, logarithm 3 ulp, its square), so that from a
    sum of 64 on, whose ulp is 128 u, rounding takes a warp's sum up by 1 exactly, but for half
    an ulp where the sum's exponent changes: 13 u by 441506, its rows. 4864 warps' sums are joined by
    17 more additions, and three products follow: 24 + 13 + 17 + 3 < 64 u. One of the 608 CTAs
    holds 27000 u of the sums, one row of a warp 0.002 u a warp."""
    T = 2 ** 31 - 1
    junk = torch.full((T, 1), 7.0, dtype=torch.bfloat16, device="cuda")
    l = torch.ones_like(junk)
    del junk                                         # the gradient's memory: no row comes out right by chance
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    B = Balance(1, 1, coef=0.5, z_coef=0.125)
    losses, counts, saved = B.forward(l, idx)
    assert int(counts) == T
    assert abs(float(losses[0]) - 0.5) <= 64 * U * 0.5
    assert abs(float(losses[1]) - 0.125) <= 64 * U * 0.125
    dl = B.backward(l, saved)
    want = 2 * 0.125 / T                             # of the penalty; the scores' own is 0 with one expert
    first = float(dl[0])
    assert abs(first - want) <= (2.0 ** -8 + 64 * U) * want
    for at in range(0, T, 2 ** 28):
        assert (dl[at:at + 2 ** 28] == first).all()

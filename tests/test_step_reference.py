"""Pins of tests/step_reference.py on the CPU: difference quotients, worked examples, and
library routines."""
import numpy as np
import pytest
import torch

from tests import step_reference as ref


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_agrees_with_difference_quotients_and_torch(kind, rng):
    h, w, dY = rng.normal(size=(3, 11)), rng.normal(size=11), rng.normal(size=(3, 11))
    b = rng.normal(size=11)
    y, m, r = ref.norm(h, w, b, kind, 1e-3)
    if kind == "layer":
        want = torch.nn.functional.layer_norm(*(torch.from_numpy(a) for a in (h,)), (11,),
                                              torch.from_numpy(w), torch.from_numpy(b), 1e-3)
        np.testing.assert_allclose(y, want.numpy(), rtol=1e-12)
    else:
        np.testing.assert_allclose(((y - b) / w) ** 2 @ np.ones(11) / 11,
                                   (h ** 2).mean(1) / ((h ** 2).mean(1) + 1e-3), rtol=1e-12)
    dX, dW, dB = ref.norm_grad(h, w, dY, kind, 1e-3)

    def f(h, w, b):
        return (ref.norm(h, w, b, kind, 1e-3)[0] * dY).sum()

    d = 1e-6
    for i in range(3):
        for j in range(11):
            e = np.zeros_like(h)
            e[i, j] = d
            assert abs((f(h + e, w, b) - f(h - e, w, b)) / (2 * d) - dX[i, j]) < 1e-7
    for j in range(11):
        e = np.zeros(11)
        e[j] = d
        assert abs((f(h, w + e, b) - f(h, w - e, b)) / (2 * d) - dW[j]) < 1e-7
        assert abs((f(h, w, b + e) - f(h, w, b - e)) / (2 * d) - dB[j]) < 1e-7


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_agrees_with_difference_quotients(score, rng):
    l = rng.normal(size=(9, 5))
    idx = rng.integers(-1, 6, size=(9, 2))
    seqs = [1, 4, 4, 8]                                  # an empty sequence, rows outside
    L, counts, g0, g1 = ref.balance(l, idx, score, 0.3, 0.2, seqs)
    assert counts.sum() == ((idx[1:8] >= 0) & (idx[1:8] < 5)).sum()
    d = 1e-6
    for t in range(9):
        for e in range(5):
            x = np.zeros_like(l)
            x[t, e] = d
            up, down = (ref.balance(l + s * x, idx, score, 0.3, 0.2, seqs)[0] for s in (1, -1))
            q = (up - down) / (2 * d)
            assert abs(q[0] - g0[t, e]) < 1e-8 and abs(q[1] - g1[t, e]) < 1e-8
    assert not g0[0].any() and not g1[8].any()


def test_even_choices_cost_the_coefficient():
    l = np.zeros((12, 6))
    idx = np.arange(24).reshape(12, 2) % 6
    L, counts, g0, _ = ref.balance(l, idx, "softmax", 0.7, 0.0)
    assert abs(L[0] - 0.7) < 1e-14 and (counts == 4).all() and np.abs(g0).max() < 1e-16
    one = np.zeros((12, 6))
    one[:, 3] = 50.0
    L = ref.balance(one, np.full((12, 1), 3), "softmax", 0.7, 0.0)[0]
    assert abs(L[0] - 0.7 * 6) < 1e-12                   # everything to one expert


def test_adamw_agrees_with_torch(rng):
    p0, g = rng.normal(size=40), rng.normal(size=(3, 40))
    p = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.9, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p0.copy(), np.zeros(40), np.zeros(40)
    for t in range(3):
        p.grad = torch.from_numpy(g[t])
        opt.step()
        q, m, v = ref.adamw(q, g[t], m, v, 0.01, 0.9, 0.95, 1e-6, 0.1, t + 1)
    np.testing.assert_allclose(q, p.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_e4m3_codes_agree_with_torch():
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.E4M3, got)


def test_moment_codes_round_trip(rng):
    m = (rng.normal(size=512) * np.exp(rng.normal(size=512) * 3)).astype(np.float32)
    v = np.exp(rng.normal(size=512) * 4).astype(np.float32)
    m[5] = v[6] = v[300] = 0
    none = np.zeros(512, np.int64)
    mc, vc, s = ref.moment_codes(m, v, none)
    mv, vv = ref.moment_values(mc, vc, s)
    # exact for the values that codes stand for
    mc2, vc2, s2 = ref.moment_codes(mv.astype(np.float32), vv.astype(np.float32), none)
    np.testing.assert_array_equal(ref.moment_values(mc2, vc2, s2)[0], mv)
    np.testing.assert_array_equal(ref.moment_values(mc2, vc2, s2)[1], vv)
    # torch's rounding of m, truncation of v to 3 bits
    for i in range(512):
        x = m[i] * 2.0 ** (134 - int(s[i // 256, 0]))
        assert float(torch.tensor([x]).to(torch.float8_e4m3fn).double()) == ref.E4M3[mc[i]]
    top = np.repeat(v.reshape(2, 256).max(1), 256)
    fine = (v > 0) & (v > top * 2.0 ** -28)
    assert (vv[fine] <= v[fine]).all() and (vv[fine] > v[fine] / (1 + 1 / 8)).all()
    assert vv[6] == 0 and (vv[v > 0] > 0).all()
    up = ref.moment_values(*ref.moment_codes(m, v, np.full(512, 65535)))[1]
    assert (up >= vv).all() and (up[fine] / vv[fine] <= 1.125 + 1e-9).all()


def test_a_value_that_is_not_finite_counts_for_no_scale():
    m, v = np.full(256, 0.5, np.float32), np.full(256, 0.25, np.float32)
    clean = ref.moment_codes(m, v, np.zeros(256, int))
    m[7], v[7], v[9] = np.nan, np.nan, np.inf
    mc, vc, s = ref.moment_codes(m, v, np.zeros(256, int))
    np.testing.assert_array_equal(s, clean[2])
    assert np.isnan(ref.E4M3[mc[7]]) and np.isnan(ref.E4M3[mc[9]])
    keep = [i for i in range(256) if i not in (7, 9)]
    np.testing.assert_array_equal(mc[keep], clean[0][keep])

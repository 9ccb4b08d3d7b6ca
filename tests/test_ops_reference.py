"""Pins of the 64-bit forms in ops_reference.py: published generator outputs, finite
differences, and worked examples. CPU only."""
import numpy as np
import pytest

from tests import ops_reference as ref


def test_philox_known_answers():
    """The known-answer vectors published with the generator (Random123, philox4x32-10)."""
    assert ref.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    f = 0xFFFFFFFF
    assert ref.philox4x32([f] * 4, [f] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


def test_choice_worked_example():
    l = np.array([0.0, 3.0, 1.0, 1.0, 2.0, -1.0])
    assert ref.choose(l, 3, "softmax") == [1, 4, 2]            # the tie 2, 3 goes to 2
    assert ref.choose(l, 2, "softmax", groups=3, top_groups=1) == [1, 0]
    assert ref.choose(l, 2, "sigmoid", bias=[9, 0, 0, 0, 0, 0]) == [0, 1]
    # two largest: sigma(0) + sigma(3) = 1.453, 2 sigma(1) = 1.462, sigma(2) + sigma(-1) = 1.15
    assert ref.choose(l, 1, "sigmoid", groups=3, top_groups=1, group_score="top2") == [2]
    l[[1, 4]] = [np.nan, -np.inf]
    assert ref.choose(l, 5, "softmax") == [2, 3, 0, 5, 1]
    assert list(ref.gates(l, [2, 1], "softmax", True, 2.0)) == [2.0, 0.0]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_is_the_difference_quotient(score, renorm, rng):
    l, dg, idx, h = rng.normal(size=9), rng.normal(size=3), [4, 0, 7], 1e-6
    got = ref.gates_grad(l, idx, dg, score, renorm, 2.5)
    for e in range(9):
        d = np.zeros(9)
        d[e] = h
        hi, lo = (ref.gates(l + s * d, idx, score, renorm, 2.5) @ dg for s in (1, -1))
        assert abs((hi - lo) / (2 * h) - got[e]) < 1e-8


def test_adapter_gradients_are_the_difference_quotients(rng):
    T, K, N, n, r, h = 5, 4, 3, 2, 2, 1e-6
    x, W = rng.normal(size=(T, K)), rng.normal(size=(K, N))
    A, B = rng.normal(size=(n, r, K)), rng.normal(size=(n, r, N))
    scale, ids, dY = np.array([0.5, 2.0]), np.array([1, 0, -1, 1, 7]), rng.normal(size=(T, N))
    out, _ = ref.lora(x, W, A, B, scale, ids, dY=dY)

    def loss(**over):
        v = dict(x=x, A=A, B=B)
        v.update(over)
        return (ref.lora(v["x"], W, v["A"], v["B"], scale, ids)[0]["y"] * dY).sum()

    grads = {"x": out["base"] + out["ad"], "A": out["dA"], "B": out["dB"]}
    for name, base in (("x", x), ("A", A), ("B", B)):
        for at in np.ndindex(base.shape):
            d = np.zeros(base.shape)
            d[at] = h
            diff = (loss(**{name: base + d}) - loss(**{name: base - d})) / (2 * h)
            assert abs(diff - grads[name][at]) < 1e-7

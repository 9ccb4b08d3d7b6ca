"""The course of 8-bit moments over many steps, in the codes' definition (tests/step_reference.py):
what a nearest rounding would freeze has to fade with the gradient."""
import numpy as np
import pytest

from tests import step_reference as ref

F = np.float32


def course(beta1, beta2, warm, idle, small, stopped, n=512):
    """Mean distance that the stopped elements travel, in units of lr, after their gradient ends."""
    r = np.random.default_rng(3)
    m, v, p = np.zeros(n, F), np.zeros(n, F), np.zeros(n)
    for t in range(1, warm + idle + 1):
        g = r.normal(size=n).astype(F)
        if t > warm:
            g[stopped] = 0
        if t == warm + 1:
            start = p.copy()
        m, v = m * F(beta1) + g * F(1 - beta1), v * F(beta2) + g * g * F(1 - beta2)
        p -= m / (1 - beta1 ** t) / (np.sqrt(v.astype(np.float64) / (1 - beta2 ** t)) + 1e-8)
        if small:
            codes = ref.moment_codes(m, v, ref.noise_words(0, n, 5, t), beta1)
            m, v = (x.astype(F) for x in ref.moment_values(*codes))
    return np.abs(p - start)[stopped].mean()


@pytest.mark.parametrize("beta1,beta2,idle,per_block", [(0.95, 0.95, 120, 256), (0.98, 0.999, 150, 256), (0.9, 0.95, 150, 64)])
def test_moments_in_8_bits_fade_like_moments_in_32(beta1, beta2, idle, per_block):
    """Bounds as derived in tests/test_gpu_optim_courses.py, 10% more for the fewer elements: five
    standard deviations of a mean of 512 (128) values, each off by 0.45 (0.3) of itself."""
    stopped = np.arange(512) % 256 < per_block
    few, many = (course(beta1, beta2, 60, idle, s, stopped) for s in (True, False))
    assert 0.8 <= few / many <= 1.35


def test_random_codes_keep_the_mean(rng):
    """Over all words each value is met on average, to half a step of 2^-16 codes."""
    words = np.arange(65536)
    for x in (0.0, 1e-5, 2.0 ** -9, 0.0123, 2.0 ** -6, 0.3, 1.0625, 7.2, 100.0, 255.9):
        codes = np.array([ref.random_code(x, w) for w in words[::37]])
        lo = ref.E4M3[codes.min()]
        up = ref.E4M3[codes.max()]
        assert lo <= x <= up and codes.max() - codes.min() <= 1
        # every 37th of 65536 words: each bit still even to 1 / 1771
        assert abs(ref.E4M3[codes].mean() - x) <= (ref.E4M3[codes.min() + 1] - lo) * 0.03 + 2.0 ** -30
        assert ref.random_code(x, 0) in (codes.min(), codes.max())
    nearest = [(0.3, 0.3125), (0.31, 0.3125), (1.05, 1.0), (1.07, 1.125), (0.0009, 0.0), (0.0011, 2.0 ** -9)]
    for x, want in nearest:                                    # a word of 0 rounds to nearest
        assert ref.E4M3[ref.random_code(x, 0)] == want

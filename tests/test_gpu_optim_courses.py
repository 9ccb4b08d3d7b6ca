"""8-bit moments over many steps on the GPU, beside moments in 32 bits with the same gradients.

The distance that an element travels when its gradient ends, after 60 steps of normal gradients:
sum over k of |m_k| / sqrt(v_k). Rounding at random keeps the mean of m, so that |m_k| fades by beta1 a
step on average; to nearest at beta1 = 0.9 seven codes halve it (16, 14, 13, 12, 11, 10, 9, 8), by 0.906 a
step: 1.08 times as far with v's 0.975 a step. v's rounding is off by at most 1/8 and by 1/16 on
the root of the mean square, so that the mean of v_k^(-1/2) is up by at most 3/8 1/256 (1.1) a step, 1.0017^k,
over the fading step 1.03 to 1.10 times. The start of the course, after 60 steps: m's own noise adds 1.5%
to the mean of |m|, v's 3% to that of v^(-1/2) (beta2 = 0.999). All together 1.15 at most. An element's own
distance is off by 0.3 to 0.45 of itself, a mean of 1024 of them by 1.5%, five times that 7%.
Downwards only v's smallest code counts, long after the step has faded. Frozen codes of m give 30 to 160 times."""
import pytest
import torch

from grouped_gemm_built_gb300.optim import AdamW
from tests import step_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def distance(bits, betas, idle, stopped, dtype):
    n = stopped.numel()
    g = torch.Generator(device="cuda").manual_seed(11)
    p = torch.zeros(n, dtype=dtype, device="cuda")
    opt = AdamW([p], betas=betas, bits=bits, seed=5)
    for k in range(60 + idle):
        grad = torch.randn(n, generator=g, device="cuda")
        if k >= 60:
            grad[stopped] = 0
        if k == 60:
            start = (p if dtype == F32 else opt.master).clone()
        opt.step([grad], lr=1e-3)
    assert all(t.isfinite().all() for t in opt.moments())
    return float(((p if dtype == F32 else opt.master) - start)[stopped].abs().double().mean())


@pytest.mark.parametrize("betas,idle,per_block", [
    ((0.95, 0.95), 200, 256), ((0.95, 0.99), 400, 256), ((0.98, 0.999), 800, 256), ((0.9, 0.95), 800, 256),
    ((0.9, 0.95), 800, 16), ((0.95, 0.95), 200, 16), ((0.9, 0.999), 800, 16)])
def test_moments_in_8_bits_fade_like_moments_in_32(betas, idle, per_block):
    stopped = torch.arange(1 << 14, device="cuda") % 256 < per_block
    few, many = (distance(bits, betas, idle, stopped, F32) for bits in (8, 32))
    assert 0.9 <= few / many <= 1.25


def test_moments_of_masters_fade_too():
    stopped = torch.arange(1 << 14, device="cuda") % 256 < 128
    few, many = (distance(bits, (0.95, 0.95), 200, stopped, BF) for bits in (8, 32))
    assert 0.9 <= few / many <= 1.25


@pytest.mark.parametrize("beta1", [0.0, 0.9, 0.9001, 0.95, 0.999])
def test_codes_bit_for_bit(beta1):
    """Elements from 1e-9 to 1 in a block: normal codes, small ones and none."""
    import numpy as np

    n, f = 1024, np.float32
    g = torch.Generator().manual_seed(2)
    opt = AdamW([torch.zeros(n, device="cuda")], betas=(beta1, 0.99), bits=8, seed=21)
    for t in range(1, 4):
        grad = torch.randn(n, generator=g) * 10.0 ** (-(torch.arange(n) % 10).float())
        grad[::11] = 0
        m0, v0 = (x.float().cpu().numpy() for x in opt.moments())
        opt.step([grad.cuda()], lr=0.0)
        g32 = grad.numpy()
        m = m0 * f(beta1) + g32 * f(1 - beta1)
        v = v0 * f(0.99) + (g32 * g32) * f(1 - 0.99)
        mc, vc, sc = ref.moment_codes(m, v, ref.noise_words(0, n, 21, t), beta1)
        np.testing.assert_array_equal(opt.m.cpu().numpy(), mc)
        np.testing.assert_array_equal(opt.v.cpu().numpy(), vc)
        np.testing.assert_array_equal(opt.scales.cpu().numpy(), sc)


def test_values_of_tiny_moments():
    """Blocks whose largest |m| goes down to 2^-130: bf16 holds the codes' values exactly from a = 10
    on (steps of 2^(a - 143), bf16's smallest is 2^-133), smaller ones to half of 2^-133."""
    import numpy as np

    n, f = 256 * 14, np.float32
    g = torch.randn(n, generator=torch.Generator().manual_seed(4)).clamp(-1.9, 1.9)
    g *= 2.0 ** -(116.0 + torch.arange(n) // 256)
    opt = AdamW([torch.zeros(n, device="cuda")], betas=(0.0, 0.95), bits=8, seed=3)
    opt.step([g.cuda()], lr=0.0)
    mv, vv = ref.moment_values(opt.m.cpu().numpy(), opt.v.cpu().numpy(), opt.scales.cpu().numpy())
    m, v = (x.double().cpu().numpy() for x in opt.moments())
    a = np.repeat(opt.scales[:, 0].cpu().numpy(), 256)
    assert a.min() == 8 and a.max() >= 11
    np.testing.assert_array_equal(m[a >= 10], mv[a >= 10])
    assert np.abs(m - mv).max() <= 2.0 ** -134 and (m != mv).any()
    np.testing.assert_array_equal(v, vv)

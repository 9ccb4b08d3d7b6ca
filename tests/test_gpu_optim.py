"""The gradient norm and the AdamW step on the GPU against float64.

Bounds, u = 2^-24. Norm: squares are summed in fp32 over runs of 32 (33 u), then in fp64: 17 u on
the root, u for storing; coef the same and 2 u. Moments: beta, 1 - beta, two products, a square
and a sum: 6 u of the summands' absolute values. The step m / c1 / (sqrt(v / c2) + eps): the
moments' errors (v's by half), and 12 u of itself for its roundings; from a step number on the
device, 10 u more for expm1. p: lr times that, 2 u of lr decay |p|, u of the result. 8-bit
moments are compared code by code: they are a function of the fp32 steps, taken one by one."""
import numpy as np
import pytest
import torch

from grouped_gemm_built_gb300 import mok
from grouped_gemm_built_gb300.optim import AdamW, grad_norm
from tests import step_reference as ref

pytestmark = pytest.mark.gpu
U = ref.U
BF, F32 = torch.bfloat16, torch.float32


def d(t):
    return t.double().cpu().numpy()


def draw(n, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * std).to(dtype).cuda()


# ---------------------------------------------------------------------- gradient norm
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("sizes", [[1], [7], [256], [8192], [8193, 1, 3], [100_001], [5] * 300, [3000] * 1300,
                                   [2_000_003, 17]])
def test_norm_of_all_gradients(dtype, sizes):
    grads = [draw(n, dtype, i, std=0.5 + i % 7) for i, n in enumerate(sizes)]
    want = np.sqrt(sum((d(g) ** 2).sum() for g in grads))
    norm, coef = grad_norm(grads, max_norm=0.5 * want, scale=0.25)
    assert abs(float(norm) - 0.25 * want) <= 18 * U * 0.25 * want
    assert float(coef) == 0.25                                # below the limit
    norm, coef = grad_norm(grads, max_norm=0.1 * want)
    assert abs(float(coef) - 0.1) <= 20 * U * 0.1


def test_mixed_types_missing_and_unaligned_gradients():
    flat = draw(40_000, BF, 1)
    grads = [flat[1:20_000], None, flat[20_003:], draw(999, F32, 2), torch.empty(0, device="cuda"), draw((7, 5), F32, 3)]
    want = np.sqrt(sum((d(g) ** 2).sum() for g in grads if g is not None))
    norm, coef = grad_norm(tuple(grads))
    assert abs(float(norm) - want) <= 18 * U * want and float(coef) == 1.0


@pytest.mark.parametrize("size", [1e-40, 1e-25, 1e-19, 3e19, 1e25, 2e37])
def test_squares_beyond_fp32(size):
    g = draw(5000, F32, 4) * size
    want = np.sqrt((d(g) ** 2).sum())
    norm, coef = grad_norm([g, torch.zeros(9000, device="cuda")])
    if want > np.finfo(np.float32).max:                       # 1.4e39, no fp32 number
        assert float(norm) == np.inf and np.isnan(float(coef))
    else:
        assert abs(float(norm) - want) <= 18 * U * want + 2.0 ** -149


def test_no_gradient_at_all_and_values_that_are_not_finite():
    norm, coef = grad_norm([torch.zeros(3000, device="cuda")], max_norm=1.0)
    assert float(norm) == 0.0 and float(coef) == 1.0
    for bad in (float("nan"), float("inf"), -float("inf")):
        for dtype in (BF, F32):
            g = draw(10_000, dtype, 1)
            g[7777] = bad
            norm, coef = grad_norm([draw(50, BF, 2), g], max_norm=1.0)
            assert not np.isfinite(float(norm)) and np.isnan(float(coef))


def test_norm_repeats_bit_for_bit_in_a_graph():
    grads = [draw(123_457, BF, i) for i in range(9)]
    want = grad_norm(grads, 1.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        grad_norm(grads, 1.0)
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = grad_norm(grads, 1.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------------------- AdamW
def starts(sizes):
    at, out = 0, []
    for n in sizes:
        out.append(at)
        at += -(-n // 256) * 256
    return out


class Twin:
    """An AdamW and its 64-bit (8-bit moments: 32-bit) course, step by step."""

    def __init__(self, sizes, p_types, bits, betas=(0.9, 0.95), eps=1e-8, decay=0.1, seed=77, views=False):
        self.sizes, self.at = sizes, starts(sizes)
        self.params = [draw(n, t, 100 + i) for i, (n, t) in enumerate(zip(sizes, p_types))]
        if views:                                            # off every 16-byte boundary
            self.params = [torch.cat([p[:1], p])[1:] for p in self.params]
        self.betas, self.eps, self.decay = betas, eps, [decay / (1 + i) for i in range(len(sizes))]
        self.opt = AdamW(self.params, betas=betas, eps=eps, weight_decay=self.decay, bits=bits, seed=seed)

    def step(self, grads, lr=0.01, coef=None, t=None, extra=0.0):
        o = self.opt
        number = o.steps + 1 if t is None else int(t)
        before = [(d(o.master[a:a + n]) if p.dtype == BF else d(p)) for p, a, n in zip(self.params, self.at, self.sizes)]
        if o.bits == 8:
            m0, v0 = ref.moment_values(o.m.cpu().numpy(), o.v.cpu().numpy(), o.scales.cpu().numpy())
        else:
            m0, v0 = d(o.m), d(o.v)
        o.step(grads, lr=torch.tensor([lr], device="cuda") if t is not None else lr,
               coef=None if coef is None else torch.tensor([coef], device="cuda"), step=t)
        c = 1.0 if coef is None else float(np.float32(coef))
        lr = float(np.float32(lr))
        (b1, b2), f = self.betas, np.float32
        new_m, new_v = np.zeros(o.elements, f), np.zeros(o.elements, f)
        for i, (p, g, a, n) in enumerate(zip(self.params, grads, self.at, self.sizes)):
            if g is None or n == 0:
                continue
            gd, s = d(g).reshape(-1) * c, slice(a, a + n)
            want, m, v = ref.adamw(before[i], gd, m0[s], v0[s], lr, b1, b2, self.eps, self.decay[i], number)
            dm = 6 * U * (b1 * np.abs(m0[s]) + (1 - b1) * np.abs(gd))
            step = m / (1 - b1 ** number) / (np.sqrt(v / (1 - b2 ** number)) + self.eps)
            scale = 1 / (1 - b1 ** number) / (np.sqrt(v / (1 - b2 ** number)) + self.eps)
            tol = lr * (dm * scale + (16 + extra) * U * np.abs(step) + 2 * U * self.decay[i] * np.abs(before[i]))
            tol = tol + 2 * U * np.abs(want)
            got = d(o.master[s]) if p.dtype == BF else d(p)
            bad = ~(np.abs(got - want) <= tol)
            assert not bad.any(), (i, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])
            if p.dtype == BF:
                assert torch.equal(p, o.master[s].to(BF))
            if o.bits == 32:
                np.testing.assert_array_less(np.abs(d(o.m[s]) - m), dm + 1e-44)
                np.testing.assert_array_less(np.abs(d(o.v[s]) - v), 6 * U * v + 1e-44)
            else:
                g32 = g.float().cpu().numpy().reshape(-1) * f(c)
                new_m[s] = m0[s].astype(f) * f(b1) + g32 * f(1 - b1)
                new_v[s] = v0[s].astype(f) * f(b2) + (g32 * g32) * f(1 - b2)
                blocks = slice(a, a + -(-n // 256) * 256)
                words = ref.noise_words(blocks.start, blocks.stop - blocks.start, o.seed, number)
                mc, vc, sc = ref.moment_codes(new_m[blocks], new_v[blocks], words)
                np.testing.assert_array_equal(o.m[blocks].cpu().numpy(), mc)
                np.testing.assert_array_equal(o.v[blocks].cpu().numpy(), vc)
                np.testing.assert_array_equal(o.scales[blocks.start // 256:blocks.stop // 256].cpu().numpy(), sc)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_type", [BF, F32])
@pytest.mark.parametrize("g_type", [BF, F32])
@pytest.mark.parametrize("views", [False, True])
def test_steps(bits, p_type, g_type, views):
    sizes = [1, 255, 256, 257, 2048, 2049, 4111]
    T = Twin(sizes, [p_type] * len(sizes), bits, views=views)
    for k in range(3):
        grads = [draw(n, g_type, 10 * k + i, std=0.1 * 3.0 ** (i - k)) for i, n in enumerate(sizes)]
        if views:
            grads = [torch.cat([g[:1], g])[1:] for g in grads]
        T.step(grads, coef=None if k == 1 else 0.3)


@pytest.mark.parametrize("bits", [32, 8])
def test_mixed_types_and_missing_gradients(bits):
    sizes = [300, 7, 0, 1000, 64]
    T = Twin(sizes, [BF, F32, F32, F32, BF], bits)
    T.step([draw(n, (BF, F32)[i % 2], i) for i, n in enumerate(sizes)])
    frozen = [t.clone() for t in (T.params[0], T.params[3], T.opt.master[:300], T.opt.m, T.opt.v)]
    grads = [draw(n, BF, 50 + i) for i, n in enumerate(sizes)]
    grads[0] = grads[3] = None
    T.step(grads)
    assert torch.equal(T.params[0], frozen[0]) and torch.equal(T.params[3], frozen[1])
    assert torch.equal(T.opt.master[:300], frozen[2])
    for now, was in ((T.opt.m, frozen[3]), (T.opt.v, frozen[4])):
        assert torch.equal(now[:512], was[:512]) and torch.equal(now[768:1792], was[768:1792])
        assert not torch.equal(now[512:768], was[512:768])


def test_shapes_beyond_vectors_and_many_tensors():
    """More tensors than one launch holds, of every small size."""
    sizes = [1 + i % 97 for i in range(1500)]
    T = Twin(sizes, [(BF, F32)[i % 3 == 0] for i in range(1500)], 32)
    T.step([draw(n, F32, i) for i, n in enumerate(sizes)])
    T = Twin(sizes[:700], [F32] * 700, 8)
    T.step([draw(n, BF, i) for i, n in enumerate(sizes[:700])])


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("betas,eps,decay", [((0.0, 0.0), 1e-8, 0.0), ((0.9, 0.999), 1e-3, 0.01), ((0.0, 0.99), 1e-30, 1.0)])
def test_hyper_parameters(bits, betas, eps, decay):
    T = Twin([700], [F32], bits, betas=betas, eps=eps, decay=decay)
    for k in range(2):
        T.step([draw(700, F32, k)], lr=0.1)


@pytest.mark.parametrize("bits", [32, 8])
def test_wide_ranges_in_a_block(bits):
    """Gradients from 1e-18 to 1e15 side by side; zeros among them."""
    g = draw(2048, F32, 1) * 10.0 ** (torch.arange(2048, device="cuda") % 34 - 18).double()
    g = g.float()
    g[::5] = 0
    T = Twin([2048], [F32], bits, eps=1e-12)
    for k in range(3):
        T.step([g * (1.0 - 0.7 * k)], lr=1e-3)


@pytest.mark.parametrize("t", [1, 2, 10, 1000, 10**6, 2**31 - 1])
def test_step_number_and_rate_on_the_device(t):
    T = Twin([600], [F32], 32)
    T.step([draw(600, F32, 1)], t=torch.tensor([t], dtype=torch.int32, device="cuda"), extra=10)
    assert T.opt.steps == 0
    T = Twin([600], [BF], 8)
    T.step([draw(600, F32, 1)], t=torch.tensor([t], dtype=torch.int32, device="cuda"), extra=10)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_factor_that_is_not_finite_skips_the_step(bits):
    T = Twin([500, 300], [BF, F32], bits)
    T.step([draw(500, BF, 1), draw(300, F32, 2)])
    state = [t for t in (*T.params, T.opt.master, T.opt.m, T.opt.v, T.opt.scales) if t is not None]
    was = [t.clone() for t in state]
    for bad in (float("nan"), float("inf")):
        T.opt.step([draw(500, BF, 3), draw(300, F32, 4)], lr=0.1, coef=torch.tensor([bad], device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(state, was))


def test_gradients_that_are_not_finite():
    """Without a factor that skips: NaN where the formula gives it, neighbours untouched."""
    for bits in (32, 8):
        g = draw(512, F32, 1)
        clean = Twin([512], [F32], bits)
        clean.opt.step([g], lr=0.1)
        T = Twin([512], [F32], bits)
        bad = g.clone()
        bad[3], bad[300] = float("nan"), float("inf")
        T.opt.step([bad], lr=0.1)
        keep = torch.ones(512, dtype=torch.bool, device="cuda")
        keep[[3, 300]] = False
        assert torch.equal(T.params[0][keep], clean.params[0][keep])
        assert torch.isnan(T.params[0][[3, 300]]).all()
        m, v = T.opt.moments()
        assert torch.isnan(m[3]) and not torch.isfinite(m[300])
        assert torch.isfinite(m[:512][keep]).all() and torch.isfinite(v[:512][keep]).all()
        T.opt.step([g], lr=0.1)
        assert torch.isnan(T.params[0][[3, 300]]).all() and torch.isfinite(T.params[0][keep]).all()


def test_moments_are_the_codes_values():
    T = Twin([5000], [F32], 8)
    for k in range(3):
        T.step([draw(5000, F32, k) * 10.0 ** (k - 1)])
    m, v = T.opt.moments()
    mv, vv = ref.moment_values(T.opt.m.cpu().numpy(), T.opt.v.cpu().numpy(), T.opt.scales.cpu().numpy())
    np.testing.assert_array_equal(d(m), mv)
    np.testing.assert_array_equal(d(v), vv)
    T = Twin([5], [F32], 32)
    assert T.opt.moments()[0] is T.opt.m


def test_slow_averages_move_in_8_bits():
    """v follows a change of the gradient's size by a factor of 2 with beta2 = 0.999, a step of
    0.3 %, far below a code's step of 6 to 12 %: its mean over 2^16 elements stays within five
    standard deviations of the 64-bit average's course. A rounding goes up or down a code, at most 1/8 of the
    value: its standard deviation is at most 1/16. Each is kept by 0.999 a step, so all together
    have 1/16 / sqrt(1 - 0.999^2) = 1/16 22.4, over 2^16 elements 1/16 22.4 / 256 = 0.55 %."""
    n = 1 << 16
    p = torch.zeros(n, device="cuda")
    opt = AdamW([p], betas=(0.9, 0.999), bits=8, seed=5)
    want = 0.0
    ones = torch.ones(n, device="cuda")
    for k in range(800):
        g = 1.0 if k < 400 else 2.0
        opt.step([ones * g], lr=0.0)
        want = 0.999 * want + 0.001 * g * g
    v = d(opt.moments()[1])
    assert abs(v.mean() / want - 1) < 5 * 0.0055


def test_a_captured_loop_equals_the_eager_one():
    def make():
        params = [draw(3000, BF, 1), draw(77, F32, 2)]
        return params, AdamW(params, weight_decay=0.1, bits=8, seed=3)

    params, opt = make()
    others, eager = make()
    grads = [draw(3000, BF, 5), draw(77, F32, 6)]
    t = torch.zeros(1, dtype=torch.int32, device="cuda")
    lr = torch.zeros(1, device="cuda")

    def once():
        t.add_(1)
        norm, coef = grad_norm(grads, max_norm=1.0)
        opt.step(grads, lr=lr, coef=coef, step=t)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            once()
    for k in range(3):
        grads[0].copy_(draw(3000, BF, 20 + k))
        lr.fill_(0.01 / (k + 1))
        graph.replay()
        norm, coef = grad_norm(grads, max_norm=1.0)
        eager.step(grads, lr=lr, coef=coef, step=torch.tensor([k + 1], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert int(t) == k + 1
        for a, b in zip((*params, opt.master, opt.m, opt.v, opt.scales),
                        (*others, eager.master, eager.m, eager.v, eager.scales)):
            assert torch.equal(a, b)


def test_restored_state_goes_on_as_before():
    T = Twin([900, 40], [BF, F32], 8)
    for k in range(2):
        T.step([draw(900, BF, k), draw(40, BF, k + 5)])
    copies = [p.clone() for p in T.params]
    again = AdamW(copies, betas=T.betas, eps=T.eps, weight_decay=T.decay, bits=8, seed=77)
    for name in ("master", "m", "v", "scales"):
        getattr(again, name).copy_(getattr(T.opt, name))
    again.steps = T.opt.steps
    grads = [draw(900, BF, 9), draw(40, BF, 10)]
    T.opt.step(grads, lr=0.1)
    again.step(grads, lr=0.1)
    assert all(torch.equal(a, b) for a, b in zip(copies, T.params)) and torch.equal(again.m, T.opt.m)


def test_overlapping_parameters_are_refused():
    flat = draw(1000, F32, 1)
    opt = AdamW([flat[:600], flat[500:]])
    with pytest.raises(mok.MokError):
        opt.step([torch.zeros(600, device="cuda"), torch.zeros(500, device="cuda")], lr=0.1)
    opt = AdamW([flat])
    with pytest.raises(mok.MokError):
        opt.step([flat], lr=0.1)


def test_offsets_past_32_bits():
    n = 2 ** 31 + 4096 + 7
    p = torch.zeros(n, device="cuda")
    g = torch.zeros(n, dtype=BF, device="cuda")
    tail = draw(4096, BF, 1)
    p[-4096:], g[-4096:] = 1.0, tail
    opt = AdamW([p, torch.zeros(300, device="cuda")], bits=8, seed=9)
    opt.step([g, draw(300, BF, 2)], lr=0.01)
    want, _, _ = ref.adamw(np.ones(4096), d(tail), 0.0, 0.0, 0.01, 0.9, 0.95, 1e-8, 0.0, 1)
    np.testing.assert_allclose(d(p[-4096:]), want, rtol=40 * U)
    assert not p[:100_000].any() and not p[2**31 - 100_000:2**31].any()
    at = -(-n // 256) * 256
    words = ref.noise_words(at, 512, 9, 1)
    g2 = np.zeros(512, np.float32)
    g2[:300] = draw(300, BF, 2).float().cpu().numpy()
    mc, vc, sc = ref.moment_codes(g2 * np.float32(1 - 0.9), (g2 * g2) * np.float32(1 - 0.95), words)
    np.testing.assert_array_equal(opt.m[at:].cpu().numpy(), mc)
    np.testing.assert_array_equal(opt.v[at:].cpu().numpy(), vc)
    norm, _ = grad_norm([g])
    assert abs(float(norm) - np.sqrt((d(tail) ** 2).sum())) <= 18 * U * float(norm)

"""The norm and its gradients on the GPU against float64.

Bounds, with u = 2^-24 and every value taken from the 64-bit evaluation: a row sum of H fp32
terms is off by at most n u times the sum of their absolute values, n = 80 (at most 32 terms one
after another in a thread, 5 shuffles, 32 warps, and the roundings of the terms themselves). So
the mean is off by dm = n u mean|h|, xh by e = r (dm + u |c|) + |xh| dr, with dr the relative
error of r: half of (n u + 2 dm mean|c| / (mean c^2 + eps)), plus 4 u for root, division and
storing. Results are rounded once to their type, by half a step."""
import numpy as np
import pytest
import torch

from grouped_gemm_built_gb300.norm import Norm
from tests import step_reference as ref

pytestmark = pytest.mark.gpu
U, N = ref.U, 80
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def d(t):
    return t.double().cpu().numpy()


def draw(shape, dtype, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(dtype).cuda()


def errors(h, kind, eps):
    """xh, r, the bound e of xh, and the relative error dr of r."""
    _, m, r = ref.norm(h, 1.0, None, kind, eps)
    c = h - m
    dm = N * U * np.abs(h).mean(1, keepdims=True) if kind == "layer" else 0.0
    var = (c ** 2).mean(1, keepdims=True) + eps
    dr = 0.5 * (N * U + 2 * dm * np.abs(c).mean(1, keepdims=True) / var + (dm ** 2) / var) + 4 * U
    return c * r, r, r * (dm + U * np.abs(c)) + np.abs(c * r) * dr, dr


def check(got, want, bound, dtype, what):
    got = d(got)
    tol = bound + HALF[dtype] * (np.abs(want) + bound) + 2.0 ** -133
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, np.argwhere(bad)[:3], got[bad][:3], want[bad][:3], tol[bad][:3])


def run(T, H, kind, x_t=BF, y_t=BF, w_t=BF, add=True, bias=True, eps=1e-5, mean=0.0, shift=0, w_shift=0):
    def rows(dtype, seed, std=1.0, m=0.0):
        if not shift:
            return draw((T, H), dtype, seed, std, m)
        flat = draw((T * H + shift,), dtype, seed, std, m)       # rows off every 16-byte boundary
        return flat[shift:].reshape(T, H)

    x, a = rows(x_t, 1, 1.0, mean), rows(x_t, 2, 2.0) if add else None
    w, b = draw((H + w_shift,), w_t, 3, 0.3, 1.0)[w_shift:], draw((H + w_shift,), w_t, 4)[w_shift:] if bias else None
    dY, da = rows(y_t, 5), rows(x_t, 6) if add else None
    n = Norm(w, b, kind=kind, eps=eps)
    y, h, stats = n.forward(x, add=a, out=y_t)
    g = n.backward(dY, h, stats, add=da)
    assert set(g) == ({"dX", "dW", "dB"} if bias else {"dX", "dW"})
    assert y.dtype == y_t and h.dtype == x_t and g["dX"].dtype == x_t and g["dW"].dtype == w_t
    if add:
        assert torch.equal(h, (x.float() + a.float()).to(x_t))
    else:
        assert h is x or h.data_ptr() == x.data_ptr()
    hd, wd, dYd = d(h), d(w), d(dY)
    xh, r, e, dr = errors(hd, kind, eps)
    bd = d(b) if bias else 0.0
    check(y, xh * wd + bd, e * np.abs(wd) + 3 * U * (np.abs(xh * wd) + np.abs(bd)), y_t, "y")
    dX, dW, dB = ref.norm_grad(hd, wd, dYd, kind, eps)
    t = dYd * wd
    s1 = np.abs(t).mean(1, keepdims=True) if kind == "layer" else 0.0
    s2 = np.abs(t * xh).mean(1, keepdims=True)
    ds2 = (N + 2) * U * s2 + (np.abs(t) * e).mean(1, keepdims=True)
    size = np.abs(t) + s1 + np.abs(xh) * s2
    add_d = d(da) if add else 0.0
    bound = r * ((N + 4) * U * s1 + e * s2 + np.abs(xh) * ds2 + (6 * U + dr) * size) + \
        U * np.abs(add_d)
    check(g["dX"], dX + add_d, bound, x_t, "dX")
    rows_u = (T + 12) * U
    check(g["dW"], dW, (np.abs(dYd) * e).sum(0) + rows_u * np.abs(dYd * xh).sum(0), w_t, "dW")
    if bias:
        check(g["dB"], dB, rows_u * np.abs(dYd).sum(0), w_t, "dB")


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", [(1, 1), (1, 8), (3, 7), (5, 64), (2, 256), (70, 264), (33, 1000),
                                 (17, 1024), (9, 1031), (300, 2048), (40, 4096), (6, 4104), (3, 7168),
                                 (2, 8200), (2, 16384), (1, 32767), (2, 32768)])
def test_sizes(kind, T, H):
    run(T, H, kind)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("x_t", [BF, F32])
@pytest.mark.parametrize("y_t", [BF, F32])
@pytest.mark.parametrize("w_t", [BF, F32])
@pytest.mark.parametrize("H", [520, 523])
def test_types(kind, x_t, y_t, w_t, H):
    run(37, H, kind, x_t, y_t, w_t)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", [(3, 8), (400, 136), (20, 260), (700, 1024), (9, 4096), (400, 7168), (3, 8192), (3, 8200),
                                 (2, 16384), (2, 20001)])
def test_sizes_in_fp32(kind, T, H):
    run(T, H, kind, F32, F32, F32)
    run(T, H, kind, F32, BF, F32, bias=False)


@pytest.mark.parametrize("T,H", [(500, 7168), (900, 1536), (3000, 256)])
def test_long_batches(T, H):
    """Several rows a team, and weights of either type beside the ring."""
    run(T, H, "layer", w_t=F32)
    run(T, H, "rms", bias=False)
    run(T, H, "layer", bias=False, add=False)


@pytest.mark.parametrize("add,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("H", [2048, 2047])
def test_without_residual_or_bias(add, bias, H):
    run(50, H, "layer", add=add, bias=bias)
    run(50, H, "rms", add=add, bias=bias)


@pytest.mark.parametrize("T", [1, 15, 16, 31, 151, 152, 153, 608, 1217, 4003])
def test_row_counts(T):
    run(T, 136, "layer", F32, F32, F32)


@pytest.mark.parametrize("H", [64, 1024, 7168])
@pytest.mark.parametrize("shift", [1, 3])
def test_rows_off_16_byte_boundaries(H, shift):
    run(20, H, "rms", shift=shift)
    run(20, H, "layer", F32, F32, F32, shift=shift)


@pytest.mark.parametrize("T,H", [(1, 255), (700, 57), (3, 1025), (2500, 1031), (9, 2041), (700, 2047), (5, 4087),
                                 (5, 4089), (330, 4099), (330, 7167), (3, 8177), (3, 8185), (3, 8193)])
def test_rows_that_begin_between_boundaries(T, H):
    run(T, H, "layer")
    run(T, H, "rms", w_t=F32, bias=False)
    run(T, H, "layer", bias=False, add=False)
    run(T, H, "layer", F32, F32, F32)
    run(T, H, "rms", F32, BF, BF, bias=False)


@pytest.mark.parametrize("x_t", [BF, F32])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("H", [57, 1031, 4100, 7167])
def test_a_row_without_numbers_leaves_its_neighbours_alone(x_t, kind, H):
    """Rows share accesses with the rows beside them; so do the buffers' ends with what follows."""
    from grouped_gemm_built_gb300 import mok
    T = 310
    x, a, dY, da = (draw((T, H), x_t, i) for i in range(4))
    w, b = draw((H,), x_t, 5), draw((H,), x_t, 6)
    bad = torch.arange(T, device="cuda") % 3 == 1
    good = ~bad
    n = Norm(w, b, kind=kind)
    y, h, stats = n.forward(x, add=a)
    g = n.backward(dY, h, stats, add=da)
    for value in (float("nan"), float("inf")):
        x2 = x.clone()
        x2[bad] = value
        flat = torch.full((3, T * H + 16), 7.0, dtype=x_t, device="cuda")
        y2, h2, dX2 = (f[:T * H].view(T, H) for f in flat)
        whole = all(t.data_ptr() % 16 == 0 for t in (y2, h2, dX2))
        st, dW, dB = torch.empty_like(stats), torch.empty_like(w), torch.empty_like(w)
        t = 0 if x_t == BF else 1
        dims = mok.MokNormDims(T=T, H=H, kind=mok.MOK_NORM_RMS if kind == "rms" else mok.MOK_NORM_LAYER, eps=n.eps,
                               x_type=t, y_type=t, w_type=t)
        s = torch.cuda.current_stream().cuda_stream
        mok.mok_norm_fwd(dims, x2.data_ptr(), a.data_ptr(), w.data_ptr(), b.data_ptr(), h2.data_ptr(), y2.data_ptr(),
                         st.data_ptr(), s)
        ws = torch.empty(mok.mok_norm_get_sizes(dims).workspace_bytes, dtype=torch.uint8, device="cuda")
        mok.mok_norm_bwd(dims, dY.data_ptr(), h2.data_ptr(), w.data_ptr(), st.data_ptr(), da.data_ptr(), dX2.data_ptr(),
                         dW.data_ptr(), dB.data_ptr(), ws.data_ptr(), s)
        if whole:                                            # the same form of kernel
            assert torch.equal(h2[good], h[good]) and torch.equal(y2[good], y[good])
            assert torch.equal(st[good], stats[good]) and torch.equal(dX2[good], g["dX"][good])
            assert torch.equal(dB, g["dB"])                  # a sum of dY alone
        assert y2[good].isfinite().all() and dX2[good].isfinite().all() and dB.isfinite().all()
        assert y2[bad].isnan().any(1).all()
        assert (flat[:, T * H:] == 7.0).all()


@pytest.mark.parametrize("H", [64, 1024, 7168])
def test_parameters_off_16_byte_boundaries(H):
    """Aligned rows with parameters that are slices of one tensor."""
    run(40, H, "layer", w_shift=1)
    run(40, H, "rms", w_t=F32, bias=False, w_shift=1)
    run(40, H, "layer", F32, F32, F32, w_shift=1)


@pytest.mark.parametrize("H", [1024, 5000])
def test_a_mean_far_from_zero(H):
    run(11, H, "layer", F32, F32, F32, add=False, mean=1000.0)


def test_without_rows():
    n = Norm(draw((24,), F32, 0), draw((24,), F32, 1), kind="layer")
    x = torch.empty(0, 24, device="cuda")
    y, h, stats = n.forward(x, add=x.clone())
    g = n.backward(y, h, stats)
    assert y.shape == h.shape == g["dX"].shape == (0, 24)
    assert not g["dW"].any() and not g["dB"].any()


def test_rows_that_are_not_finite_stay_alone():
    """Infinities and NaN reach their own row, dW and dB; constant rows have the formula's values."""
    x = draw((6, 512), F32, 1)
    clean = Norm(torch.ones(512, device="cuda"), kind="layer").forward(x)[0]
    x[1, 7], x[3, 9], x[4] = float("nan"), float("inf"), 3.0
    n = Norm(torch.ones(512, device="cuda"), torch.full((512,), 0.5, device="cuda"), kind="layer")
    y, h, stats = n.forward(x)
    assert torch.isnan(y[1]).all() and torch.isnan(y[3]).all()
    assert (y[4] == 0.5).all()
    for t in (0, 2, 5):
        assert torch.equal(y[t], clean[t] + 0.5)
    dX = n.backward(torch.ones_like(y), h, stats)["dX"]
    assert torch.isnan(dX[1]).all() and torch.isfinite(dX[[0, 2, 4, 5]]).all()
    zero = Norm(torch.ones(512, device="cuda"), kind="rms", eps=0.0).forward(torch.zeros(1, 512, device="cuda"))
    assert torch.isnan(zero[0]).all()                        # 0 / 0


def test_results_repeat_bit_for_bit():
    x, dY = draw((1000, 2056), BF, 1), draw((1000, 2056), BF, 2)
    n = Norm(draw((2056,), BF, 3), draw((2056,), BF, 4), kind="layer")

    def once():
        y, h, stats = n.forward(x, add=dY)
        return [y, h, stats, *n.backward(dY, h, stats, add=x).values()]

    first = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, once()))


@pytest.mark.parametrize("H", [1000, 7168])
def test_captured_on_another_stream(H):
    x, a, dY = (draw((130, H), BF, i) for i in range(3))
    n = Norm(draw((H,), BF, 3), kind="rms")

    def once():
        y, h, stats = n.forward(x, add=a)
        return [y, h, *n.backward(dY, h, stats, add=a).values()]

    want = once()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        got = once()
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        with torch.cuda.graph(graph, stream=s):
            got = once()
    x.copy_(draw((130, H), BF, 9))
    want = once()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))


@pytest.mark.parametrize("H", [1024, 1027, 7168])
def test_results_in_place_of_inputs(H):
    """h over x or add, y over the other; dX over add: through the C ABI."""
    from grouped_gemm_built_gb300 import mok
    T = 40
    x, a, dY = (draw((T, H), BF, i) for i in range(3))
    w = draw((H,), BF, 3)
    n = Norm(w, kind="rms", eps=1e-5)
    y, h, stats = n.forward(x, add=a)
    g = n.backward(dY, h, stats, add=a)
    dims = mok.MokNormDims(T=T, H=H, kind=mok.MOK_NORM_RMS, eps=1e-5, x_type=0, y_type=0, w_type=0)
    s = torch.cuda.current_stream().cuda_stream
    for first, second in ((0, 1), (1, 0)):
        io = [x.clone(), a.clone()]
        st = torch.empty_like(stats)
        mok.mok_norm_fwd(dims, io[0].data_ptr(), io[1].data_ptr(), w.data_ptr(), None, io[first].data_ptr(),
                         io[second].data_ptr(), st.data_ptr(), s)
        assert torch.equal(io[first], h) and torch.equal(io[second], y) and torch.equal(st, stats)
    out, dW = a.clone(), torch.empty_like(w)
    ws = torch.empty(mok.mok_norm_get_sizes(dims).workspace_bytes, dtype=torch.uint8, device="cuda")
    mok.mok_norm_bwd(dims, dY.data_ptr(), h.data_ptr(), w.data_ptr(), stats.data_ptr(), out.data_ptr(),
                     out.data_ptr(), dW.data_ptr(), None, ws.data_ptr(), s)
    assert torch.equal(out, g["dX"]) and torch.equal(dW, g["dW"])
    y2 = torch.empty_like(y)                                 # a forward that keeps no statistics
    mok.mok_norm_fwd(dims, h.data_ptr(), None, w.data_ptr(), None, None, y2.data_ptr(), None, s)
    assert torch.equal(y2, y)


def test_offsets_past_32_bits():
    T, H = 300_100, 7168
    x = torch.zeros((T, H), dtype=BF, device="cuda")
    x[-3:] = draw((3, H), BF, 1)
    n = Norm(draw((H,), BF, 2), kind="rms")
    y, h, stats = n.forward(x)
    few = n.forward(x[-3:].contiguous())
    assert torch.equal(y[-3:], few[0]) and torch.equal(stats[-3:], few[2])
    dY = torch.zeros_like(x)
    dY[-3:] = draw((3, H), BF, 3)
    g, want = n.backward(dY, h, stats), n.backward(dY[-3:].contiguous(), x[-3:].contiguous(), few[2])
    assert torch.equal(g["dX"][-3:], want["dX"])
    torch.testing.assert_close(g["dW"], want["dW"], rtol=2 ** -7, atol=0)


def test_replaced_parameters_are_what_the_next_call_reads():
    x = draw((5, 64), F32, 1)
    n = Norm(draw((64,), F32, 2), kind="rms")
    n.forward(x)
    n.weight = draw((64,), F32, 3)
    n.bias = draw((64,), F32, 4)
    assert torch.equal(n.forward(x)[0], Norm(n.weight, n.bias, kind="rms").forward(x)[0])

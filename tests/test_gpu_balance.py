"""The balance loss, the logit penalty and their gradients on the GPU against float64.

Bounds, u = 2^-24: an exponential is off by 3 u plus u for each unit of its argument (the
argument's rounding), a sigmoid by 6 u more; sums of E <= 512 terms over a warp by 22 u (16 in a
lane, 5 shuffles). Scores are therefore off by q = (2 R + 40) u relative, R the largest |logit|
or the row's spread of logits. A row's loss is off by (q + 24 u) of itself, a gradient entry
slope (f - p.f) by slope (q |f - p.f| + (q + 30 u) sum p |f|), f the factor times the counts
relative to their mean."""
import numpy as np
import pytest
import torch

from grouped_gemm_built_gb300.balance import Balance
from grouped_gemm_built_gb300.routing import Routing
from tests import step_reference as ref
from tests.ops_reference import scores

pytestmark = pytest.mark.gpu
U = ref.U
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def make(T, E, k, dtype, seed=0, std=2.0, bad_ids=False):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn(T, E, generator=g) * std + torch.randn(E, generator=g)).to(dtype)
    idx = l.float().argsort(1, descending=True)[:, :k].to(torch.int32).contiguous()
    if bad_ids and T:
        idx[::3, 0] = -1
        idx[1::4, -1] = E + 5
    return l.cuda(), idx.cuda()


def check(l, idx, score, coef=0.5, z=0.25, seqs=None, add=None, dlosses=None, dtype=None):
    T, E = l.shape
    B = Balance(E, idx.shape[1], score=score, coef=coef, z_coef=z)
    sq = None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device="cuda")
    losses, counts, saved = B.forward(l, idx, sq)
    dl = B.backward(l, saved, sq, dlosses=dlosses, add=add, dtype=dtype)
    ld = l.double().cpu().numpy()
    want, cnt, g0, g1 = ref.balance(ld, idx.cpu().numpy(), score, coef, z, seqs)
    np.testing.assert_array_equal(counts.cpu().numpy(), cnt)
    finite = np.where(np.isfinite(ld), ld, 0.0)
    R = (finite.max(1) - finite.min(1) + np.abs(finite).max(1)) if T else np.zeros(0)
    q = (2 * R + 40) * U                                           # per row
    got = losses.double().cpu().numpy()
    worst = q.max() if T else 0.0
    assert abs(got[0] - want[0]) <= (worst + 26 * U) * want[0]
    # lse is off by the rounding of the largest logit, of log z and of the sum
    assert abs(got[1] - want[1]) <= 2 * (worst + 26 * U) * (want[1] + z)
    d0, d1 = (1.0, 1.0) if dlosses is None else dlosses.double().cpu().numpy()
    exact = d0 * g0 + d1 * g1 + (0.0 if add is None else add.double().cpu().numpy())
    tol = np.zeros_like(exact)
    ends = [0, T] if seqs is None else seqs
    total = ends[-1] - ends[0]
    for lo, hi in zip(ends, ends[1:]):
        ids = idx[lo:hi].cpu().numpy().reshape(-1)
        c = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        f = coef * E / (idx.shape[1] * (hi - lo) * total) * (c - c.sum() // E) if hi > lo else None
        for t in range(lo, hi):
            _, live, s = scores(ld[t], score)
            if not live.any():
                continue
            if s.sum() < 1e-30:                 # as in the reference: relative to the largest logit
                top = ld[t][live].max()
                s = np.where(live, np.exp(np.where(live, ld[t], top) - top), 0.0)
            p = s / s.sum()
            dot = p @ np.abs(f)
            # p bounds the slope; lse, whose gradient is 2 z / Tv lse softmax, is off by q
            e = p * (2 * q[t] * (np.abs(f) + dot) + 30 * U * dot)
            tol[t] = abs(d0) * e + abs(d1) * (np.abs(g1[t]) * (q[t] + 6 * U) + 2 * z / total * q[t])
    tol += 4 * U * (np.abs(exact) + (0.0 if add is None else np.abs(add.double().cpu().numpy())))
    out = dl.dtype
    err = np.abs(dl.double().cpu().numpy() - exact)
    tol = tol + HALF[out] * (np.abs(exact) + tol) + 2.0 ** -133
    bad = ~(err <= tol)
    assert not bad.any(), (np.argwhere(bad)[:3], err[bad][:3], tol[bad][:3], exact[bad][:3])
    return losses, counts, dl


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (2, 3, 2), (7, 33, 4), (64, 64, 6), (130, 60, 6),
                                   (300, 256, 8), (257, 384, 8), (100, 511, 9), (90, 512, 32), (9, 130, 1),
                                   (2500, 16, 2)])
def test_sizes(score, T, E, k):
    l, idx = make(T, E, k, F32)
    check(l, idx, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("z", [0.0, 0.3])
def test_types_and_added_gradient(score, dtype, out, z):
    l, idx = make(150, 96, 6, dtype, seed=3)
    add = (torch.randn(150, 96, generator=torch.Generator().manual_seed(1)) * 1e-3).to(out).cuda()
    check(l, idx, score, z=z, add=add, dlosses=torch.tensor([2.0, -0.5], device="cuda"))
    check(l, idx, score, z=z, dtype=out)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("seqs", [[0, 200], [0, 1, 2, 200], [0, 0, 57, 57, 57, 190, 190], [5, 9, 31], [13, 13],
                                  [200, 200], list(range(201)), [0, 199, 200]])
def test_sequences(score, seqs):
    l, idx = make(200, 48, 4, F32, seed=5, bad_ids=True)
    add = torch.full((200, 48), 0.125, device="cuda")
    _, _, dl = check(l, idx, score, seqs=seqs, add=add)
    outside = [t for t in range(200) if not seqs[0] <= t < seqs[-1]]
    assert (dl[outside] == 0.125).all()


def test_one_sequence_is_the_whole_batch():
    l, idx = make(777, 256, 8, BF)
    B = Balance(256, 8, score="sigmoid", z_coef=0.1)
    a, b = B.forward(l, idx), B.forward(l, idx, torch.tensor([0, 777], dtype=torch.int32, device="cuda"))
    # the same positive terms in another order: each sum of them is off by at most 26 u (the bounds above)
    torch.testing.assert_close(a[0], b[0], rtol=2 * 26 * U, atol=0)
    assert torch.equal(a[1], b[1])


def test_without_rows():
    l, idx = make(0, 32, 2, F32)
    for seqs in (None, [0, 0], [0, 0, 0, 0]):
        losses, counts, dl = check(l, idx, "softmax", seqs=seqs)
        assert not losses.any() and not counts.any() and dl.shape == (0, 32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_and_extreme_logits(score):
    l, idx = make(40, 24, 3, F32, seed=2, bad_ids=True)
    l[:, 5] = -float("inf")
    l[3, 7] = float("nan")
    l[4] = -float("inf")                       # nothing left in this row
    l[6] = -200.0                              # sigmoid scores that underflow
    l[7] = -200.0 + l[8] * 0.1
    l[9] = 60.0                                # saturated
    l[10] = torch.where(torch.arange(24, device="cuda") == 2, 80.0, -80.0)
    losses, _, dl = check(l, idx, score, z=0.01)
    masked = [t for t in range(40) if t not in (6, 9, 10)]      # those rows set expert 5 again
    assert (dl[masked, 5] == 0).all() and (dl[4] == 0).all() and dl[3, 7] == 0
    l[11, 0] = float("inf")                    # the largest finite value
    B = Balance(24, 3, score=score, coef=0.5)
    losses, _, saved = B.forward(l, idx)
    assert torch.isfinite(losses).all() and torch.isfinite(B.backward(l, saved)).all()


def test_nearly_even_counts_keep_their_gradient():
    """Counts that differ by a few in thousands: the differences carry the gradient."""
    T, E = 4096, 8
    l, _ = make(T, E, 1, F32, std=0.3)
    idx = (torch.arange(T) % E).to(torch.int32).reshape(T, 1)
    idx[:3] = 0
    check(l, idx.cuda(), "softmax", z=0.0)
    check(l, idx.cuda(), "sigmoid", z=0.0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,seqs", [
    (513, 16, 16, None), (1025, 16, 1, None), (1024, 257, 2, None), (1000, 24, 9, None),   # around one launch
    (9000, 16, 8, None), (9001, 9, 7, None),                            # counted by several clusters
    (9000, 16, 8, [0, 9000]), (9000, 16, 8, [5, 8990]), (9000, 12, 8, [0, 4, 8999])])
def test_forms_of_the_forward(score, T, E, k, seqs):
    """One launch for few rows, two otherwise; a long batch counted in parts, or as sequences with
    padding before and behind."""
    l, idx = make(T, E, k, BF, seed=T, std=1.0)
    check(l, idx, score, seqs=seqs)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_choices_and_logits_off_16_byte_boundaries(shift):
    l, idx = make(3000, 64, 5, F32, seed=4)
    ids = torch.cat([idx.flatten()[:shift], idx.flatten()])[shift:].reshape(3000, 5)
    lg = torch.cat([l.flatten()[:shift], l.flatten()])[shift:].reshape(3000, 64)
    assert ids.data_ptr() % 16 and lg.data_ptr() % 16
    a, _, _ = check(lg, ids, "sigmoid", seqs=[7, 500, 2999])
    b, _, _ = check(l, idx, "sigmoid", seqs=[7, 500, 2999])
    torch.testing.assert_close(a, b, rtol=2 * 26 * U, atol=0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_of_any_size(score):
    """Rows whose scores overflow, vanish or spread over the whole range beside ordinary ones."""
    l, idx = make(600, 40, 3, F32, seed=12)
    for t, (a, b) in enumerate([(90, 1), (-90, 1), (300, 5), (-300, 5), (0, 60), (1e4, 1e3), (-1e4, 1e3), (40, 10)]):
        l[t::17] = l[t::17] * b + a
    check(l, idx, score, z=0.0)
    check(l, idx, score, z=1e-6, seqs=[0, 100, 590])


def test_every_row_count_that_an_int_holds():
    T = 2 ** 31 - 1
    l = torch.zeros((T, 1), dtype=BF, device="cuda")
    idx = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    B = Balance(1, 1, coef=0.5, z_coef=0.1)
    losses, counts, saved = B.forward(l, idx)
    assert int(counts) == T
    # up to 2^31 / (608 CTAs 8 warps) = 441506 rows of one expert after one another, 0.5 / T each: a bit
    # of the sum an addition at worst, 441506 u
    assert abs(float(losses[0]) - 0.5) <= 441506 * U * 0.5 + 60 * U and float(losses[1]) == 0.0
    dl = B.backward(l, saved)
    assert not dl[:1000].any() and not dl[-1000:].any()


def test_repeats_bit_for_bit_and_in_place():
    l, idx = make(5000, 256, 8, BF, seed=9)
    seqs = torch.tensor([0, 100, 101, 3000, 4900], dtype=torch.int32, device="cuda")
    B = Balance(256, 8, score="sigmoid", z_coef=0.1)
    R = Routing(256, 8, score="sigmoid")
    ids, gates = R.forward(l)
    first = None
    for _ in range(3):
        losses, counts, saved = B.forward(l, ids, seqs)
        dl = R.backward(l, ids, torch.ones_like(gates), dtype=F32)
        out = B.backward(l, saved, seqs, add=dl)
        assert out.dtype == F32
        now = [losses, counts, out]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, now))
        first = now
    from grouped_gemm_built_gb300 import mok
    mok.mok_balance_bwd(B.rule, 5000, l.data_ptr(), mok.MOK_OUT_BF16, seqs.data_ptr(), 4, saved.data_ptr(), None,
                        dl.data_ptr(), dl.data_ptr(), mok.MOK_OUT_F32, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(dl, out)


@pytest.mark.parametrize("T", [100, 3000])
def test_captured_on_another_stream(T):
    l, idx = make(T, 64, 4, F32)
    seqs = torch.tensor([0, T // 3, T - 2], dtype=torch.int32, device="cuda")
    B = Balance(64, 4, z_coef=0.01)

    def once():
        losses, counts, saved = B.forward(l, idx, seqs)
        return [losses, counts, B.backward(l, saved, seqs)]

    once()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        once()
        s.synchronize()
        with torch.cuda.graph(graph, stream=s):
            got = once()
    other, ids = make(T, 64, 4, F32, seed=8)
    l.copy_(other)
    idx.copy_(ids)
    seqs.copy_(torch.tensor([1, 50, T], dtype=torch.int32))
    want = once()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("seqs", [[5, 3, 90], [0, 400, 100], [-7, 20, 100], [90, 10, 5, 2], [0, 100, 2**31 - 1]])
def test_bad_offsets_stay_in_bounds(seqs):
    """Unspecified losses, but counts and rows of this batch only."""
    l, idx = make(100, 16, 2, F32)
    B = Balance(16, 2)
    sq = torch.tensor(seqs, dtype=torch.int32, device="cuda")
    _, counts, saved = B.forward(l, idx, sq)
    B.backward(l, saved, sq)
    torch.cuda.synchronize()
    assert 0 <= int(counts.sum()) <= 200


def test_offsets_past_32_bits():
    T, E = 4_300_000, 512
    l = torch.zeros((T, E), dtype=BF, device="cuda")
    l[-50:], idx50 = make(50, E, 4, BF)
    idx = torch.full((T, 4), -1, dtype=torch.int32, device="cuda")
    idx[-50:] = idx50
    seqs = torch.tensor([T - 50, T], dtype=torch.int32, device="cuda")
    B = Balance(E, 4, score="sigmoid", z_coef=0.1)
    losses, counts, saved = B.forward(l, idx, seqs)
    dl = B.backward(l, saved, seqs)
    few = B.forward(l[-50:].contiguous(), idx50)
    torch.testing.assert_close(losses, few[0], rtol=1e-6, atol=0)
    assert torch.equal(counts, few[1])
    assert torch.equal(dl[-50:], B.backward(l[-50:].contiguous(), few[2]))
    assert not dl[:-50].any()

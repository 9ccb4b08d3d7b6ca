"""mok_lora_fwd and mok_lora_bwd on the GPU against the 64-bit form in ops_reference.py.

Bound of an element, from S, the same sums over absolute values: each of the C products of a
sum is exact in fp32 and meets at most C additions, so the sums are within C 2^-23 S (the
tensor cores may truncate, hence 2^-23); the r values of the low-rank path enter the second
product with 16 significant bits and sums of their own, (2^-16 + (K + N) 2^-23) S; bf16 results
add half a step, 2^-8 of the value."""
import numpy as np
import pytest
import torch

from grouped_gemm_built_gb300 import mok
from grouped_gemm_built_gb300.lora import AdaptedLinear
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


def make(rng, T, K, N, n, r, order):
    def bf(*shape, std=1.0):
        return torch.tensor(rng.normal(0, std, shape), dtype=torch.bfloat16)

    c = dict(x=bf(T, K), W=bf(K, N, std=0.1), A=bf(n, r, K, std=0.1), B=bf(n, r, N, std=0.1),
             scale=torch.tensor(rng.uniform(0.5, 2, n), dtype=torch.float32), dY=bf(T, N))
    if order == "rows":
        ids = rng.integers(-1, n, T)
    elif order == "none":
        ids = np.full(T, -1)
    elif order == "one":
        ids = np.full(T, n - 1)
    else:
        ids = np.sort(rng.integers(0, n, T))
        ids[ids == 0] = 2 ** 31 - 1          # outside [0, n): no adapter
    c["ids"] = torch.tensor(ids, dtype=torch.int32)
    return c


def run(c, xa=None, out=torch.bfloat16, grad=True):
    d = {k: v.cuda() for k, v in c.items()}
    xa = None if xa is None else xa.cuda()
    L = AdaptedLinear(d["W"], d["A"], d["B"], d["scale"])
    y, saved = L.forward(d["x"], d["ids"], x_ad=xa, out=out)
    res = {"y": y}
    if grad:
        res.update(L.backward(d["x"], d["ids"], saved, d["dY"], x_ad=xa, out=out))
    assert L.status() == 0
    return res


def check(c, res, out=torch.bfloat16, xa=None):
    f = {k: v.double().numpy() for k, v in c.items() if k != "ids"}
    want, mag = ref.lora(f["x"], f["W"], f["A"], f["B"], f["scale"], c["ids"].numpy(),
                         xa=None if xa is None else xa.double().numpy(), dY=f["dY"])
    if xa is None:
        want["dX"], mag["dX"] = want["base"] + want["ad"], mag["base"] + mag["ad"]
    else:
        want["dX"], mag["dX"], want["dXa"], mag["dXa"] = (want["base"], mag["base"], want["ad"],
                                                          mag["ad"])
    T, (K, N) = len(f["x"]), f["W"].shape
    rel = 2.0 ** -16 + (K + N + T) * 2.0 ** -23
    for name, v in res.items():
        v = v.double().cpu().numpy()
        tol = rel * mag[name] + (2.0 ** -8 * np.abs(want[name]) if out == torch.bfloat16 else 0)
        over = np.abs(v - want[name]) - tol
        assert (over <= 1e-30).all(), (name, over.max())
        assert np.isfinite(v).all()


@pytest.mark.parametrize("T,K,N,n,r,order", [
    (1, 64, 64, 1, 1, "one"),
    (1, 1032, 8, 3, 16, "one"),
    (2, 8, 520, 5, 3, "rows"),
    (31, 136, 200, 4, 17, "rows"),
    (128, 256, 128, 128, 16, "rows"),
    (129, 264, 328, 300, 5, "rows"),
    (257, 128, 256, 2, 33, "packed"),
    (300, 520, 72, 9, 64, "rows"),
    (200, 192, 264, 6, 128, "rows"),
    (384, 128, 576, 3, 100, "packed"),
    (500, 72, 1000, 1, 8, "one"),
    (130, 64, 64, 2, 8, "none"),
    (640, 576, 320, 70, 32, "rows"),
])
def test_forward_and_gradients(T, K, N, n, r, order, rng):
    c = make(rng, T, K, N, n, r, order)
    check(c, run(c))


@pytest.mark.parametrize("T,K,N,n,r", [(33, 136, 72, 4, 5), (260, 264, 200, 20, 40)])
def test_fp32_results(T, K, N, n, r, rng):
    c = make(rng, T, K, N, n, r, "rows")
    check(c, run(c, out=torch.float32), out=torch.float32)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,r,order", [(150, 7, 5, "rows"), (300, 3, 48, "packed"),
                                         (5, 2, 16, "none")])
def test_adapter_input_of_its_own(T, n, r, order, out, rng):
    c = make(rng, T, 136, 200, n, r, order)
    xa = torch.tensor(rng.normal(size=(T, 136)), dtype=torch.bfloat16)
    check(c, run(c, xa=xa, out=out), out=out, xa=xa)


def test_many_row_tiles_and_wide_outputs(rng):
    """More tiles than SMs, so that CTAs take several (the two accumulators alternate)."""
    c = make(rng, 2100, 128, 3008, 12, 8, "packed")
    check(c, run(c))


@pytest.mark.parametrize("T,K,N,n,r,order", [
    (1500, 520, 2000, 40, 40, "rows"), (1409, 2056, 1544, 5, 16, "packed"),
    (2304, 264, 3016, 3, 7, "packed")])
def test_pairs_of_row_tiles(T, K, N, n, r, order, rng):
    """Large enough for the two-CTA form in both directions, odd counts of row tiles among them."""
    c = make(rng, T, K, N, n, r, order)
    check(c, run(c))


@pytest.mark.parametrize("used", [0, 1, 3, 70, 700])
def test_few_rows_with_adapters(used, rng):
    """The weight gradients share the rows that have an adapter, fewer than shares among them."""
    c = make(rng, 3000, 72, 136, 6, 9, "none")
    at = torch.tensor(rng.choice(3000, used, replace=False))
    c["ids"][at] = torch.tensor(rng.choice([0, 2, 5], used), dtype=torch.int32)
    check(c, run(c))


def test_adapters_of_very_unequal_sizes(rng):
    """One adapter's rows cover several shares, others end inside one."""
    c = make(rng, 2000, 136, 200, 9, 20, "none")
    c["ids"][:] = torch.tensor(np.repeat([3, 7, 1, 8], [1700, 90, 10, 200]), dtype=torch.int32)
    c["ids"] = c["ids"][torch.tensor(rng.permutation(2000))].contiguous()
    check(c, run(c))


def test_long_contraction(rng):
    """Contraction shared between the CTAs of a cluster."""
    c = make(rng, 40, 4104, 136, 11, 16, "rows")
    check(c, run(c))


def test_one_request_cannot_reach_another(rng):
    """Adapter 1 full of inf and NaN, and rows of adapter 2 with NaN inputs and gradients: the
    other rows' results and the other adapters' gradients keep their bits."""
    T, n = 300, 5
    c = make(rng, T, 136, 200, n, 12, "rows")
    clean = run(c)
    d = {k: v.clone() for k, v in c.items()}
    ids = c["ids"]
    d["A"][1, :, ::3], d["B"][1, :, 1::2] = float("inf"), float("nan")
    d["x"][ids == 2], d["dY"][ids == 2] = float("nan"), float("inf")
    dirty = run(d)
    rows = ((ids != 1) & (ids != 2)).cuda()
    for name in ("y", "dX"):
        assert torch.equal(clean[name][rows], dirty[name][rows])
        assert not torch.isfinite(dirty[name][(ids == 1).cuda()]).all()
    for name in ("dA", "dB"):
        for a in (0, 3, 4):
            assert torch.equal(clean[name][a], dirty[name][a])


def test_padding_ranks_stay_zero_next_to_infinite_rows(rng):
    """rank 1: an inf in x gives +-inf, not NaN, where every product has one sign."""
    c = make(rng, 3, 64, 64, 1, 1, "one")
    for k in ("W", "A", "B", "x"):
        c[k] = c[k].abs() + 0.125
    c["x"][1, 5] = float("inf")
    y = run(c, grad=False)["y"]
    assert torch.isinf(y[1]).all() and torch.isfinite(y[[0, 2]]).all()


def test_rows_keep_their_bits_in_any_order(rng):
    """A row's result does not depend on its place or its neighbours."""
    c = make(rng, 256, 136, 200, 9, 20, "rows")
    y = run(c, grad=False)["y"]
    perm = torch.tensor(rng.permutation(256))
    d = dict(c, x=c["x"][perm].contiguous(), ids=c["ids"][perm].contiguous())
    assert torch.equal(run(d, grad=False)["y"], y[perm.cuda()])


def test_empty_batch_clears_the_weight_gradients():
    z = dict(dtype=torch.bfloat16, device="cuda")
    L = AdaptedLinear(torch.ones(64, 32, **z), torch.ones(2, 3, 64, **z), torch.ones(2, 3, 32, **z),
                      torch.ones(2, device="cuda"))
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    y, saved = L.forward(torch.empty(0, 64, **z), ids)
    g = L.backward(torch.empty(0, 64, **z), ids, saved, torch.empty(0, 32, **z))
    assert y.shape == (0, 32) and g["dX"].shape == (0, 64)
    assert (g["dA"] == 0).all() and (g["dB"] == 0).all()


def test_repeats_bitwise_on_another_stream(rng):
    c = {k: v.cuda() for k, v in make(rng, 700, 264, 328, 6, 24, "rows").items()}
    L = AdaptedLinear(c["W"], c["A"], c["B"], c["scale"])

    def step():
        y, saved = L.forward(c["x"], c["ids"])
        return dict(L.backward(c["x"], c["ids"], saved, c["dY"]), y=y)

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = [step() for _ in range(3)]
    side.synchronize()
    for g in again:
        for k, v in first.items():
            assert torch.equal(v, g[k]), k


def test_step_is_captured_in_a_graph(rng):
    """A whole step (its launches depend on one another ahead of time) replays from a graph."""
    c = {k: v.cuda() for k, v in make(rng, 520, 264, 328, 6, 24, "rows").items()}
    L = AdaptedLinear(c["W"], c["A"], c["B"], c["scale"])

    def step():
        y, saved = L.forward(c["x"], c["ids"])
        return dict(L.backward(c["x"], c["ids"], saved, c["dY"]), y=y)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    c["x"].copy_(torch.randn_like(c["x"]))
    c["ids"].copy_(c["ids"].flip(0))
    graph.replay()
    graph.replay()
    for k, v in step().items():
        assert torch.equal(v, got[k]), k


def test_status_word_is_read_and_cleared():
    z = dict(dtype=torch.bfloat16, device="cuda")
    L = AdaptedLinear(torch.ones(8, 8, **z), torch.ones(1, 1, 8, **z), torch.ones(1, 1, 8, **z),
                      torch.ones(1, device="cuda"))
    assert L.status() == 0
    L._status.fill_(1)                        # what a kernel does when a wait passes its bound
    assert L.status() == mok.MOK_ERR_TIMEOUT and L.status() == 0


def test_updated_weights_are_read(rng):
    c = {k: v.cuda() for k, v in make(rng, 20, 64, 64, 2, 4, "one").items()}
    L = AdaptedLinear(c["W"], c["A"], c["B"], c["scale"])
    y0, _ = L.forward(c["x"], c["ids"])
    c["B"].zero_()
    y1, _ = L.forward(c["x"], c["ids"])
    c["W"].zero_()
    y2, _ = L.forward(c["x"], c["ids"])
    assert not torch.equal(y0, y1) and not torch.equal(y1, y2) and (y2 == 0).all()


def test_row_offsets_past_32_bits():
    """More than 2^31 elements of x and dX: the last rows match the same rows alone."""
    T, K, N, r = 300_032, 7168, 64, 8
    z = dict(dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(5)

    def rnd(*shape):
        return torch.empty(shape, **z).normal_(0, 0.5, generator=g)

    W, A, B, scale = rnd(K, N), rnd(3, r, K), rnd(3, r, N), torch.ones(3, device="cuda")
    x = torch.zeros(T, K, **z)
    x[-128:] = rnd(128, K)
    dY = torch.zeros(T, N, **z)
    dY[-128:] = rnd(128, N)
    ids = (torch.arange(T, device="cuda") % 4 - 1).to(torch.int32)
    L = AdaptedLinear(W, A, B, scale)
    y, saved = L.forward(x, ids)
    got = L.backward(x, ids, saved, dY)
    tail = slice(T - 128, T)
    xs, ds, ts = x[tail].clone(), dY[tail].clone(), ids[tail].clone()
    f = [v.double().cpu().numpy() for v in (xs, W, A, B, scale)]
    want, mag = ref.lora(*f, ts.cpu().numpy(), dY=ds.double().cpu().numpy())
    want["dX"], mag["dX"] = want["base"] + want["ad"], mag["base"] + mag["ad"]
    res = {"y": y[tail], "dX": got["dX"][tail], "dA": got["dA"], "dB": got["dB"]}
    for name, v in res.items():
        tol = (2.0 ** -16 + (K + N + 128) * 2.0 ** -23) * mag[name] + 2.0 ** -8 * np.abs(want[name])
        assert (np.abs(v.double().cpu().numpy() - want[name]) <= tol).all(), name
    assert (y[:1000] == 0).all() and (got["dX"][:1000] == 0).all() and L.status() == 0

"""Every form of the adapters' kernels on the GPU, at a shape that takes it: mok_lora_get_forms says
which one a call runs, and a test fails where no shape near the given one takes its form any more.

Inputs are whole numbers small enough that every sum is exact in fp32, also of the r values, which
take up to 16 bits; the oracle is the formulas in 64 bits. What is left to differ: a high part whose
rest is 0 has a low part of 2^-24 of it, after which an accumulation may cut a last bit, 2^-23 of the
sum, off. y and dX meet at most 32 such accumulations (two parts of 8 x 16 ranks, the row's own
adapter only, joined over at most 8 CTAs), a weight gradient 2 T / 16 and the join; a sum on the way
is taken to be at most twice the largest result. Products that a kernel leaves out or adds are whole
numbers."""
import pytest
import torch

from grouped_gemm_built_gb300 import mok
from grouped_gemm_built_gb300.lora import AdaptedLinear

pytestmark = pytest.mark.gpu


def whole(g, shape, most, live=0.5):
    """Whole numbers up to `most` in size, a share `live` of them not zero."""
    v = torch.randint(1, most + 1, shape, generator=g, device="cuda").float()
    v *= torch.randint(0, 2, shape, generator=g, device="cuda") * 2 - 1
    v *= torch.rand(shape, generator=g, device="cuda") < live
    return v.to(torch.bfloat16)


def case(T, K, N, n, r, order, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dict(x=whole(g, (T, K), 1), W=whole(g, (K, N), 1), dY=whole(g, (T, N), 1),
             A=whole(g, (n, r, K), 127, min(0.5, 32 / K)), B=whole(g, (n, r, N), 127, min(0.5, 32 / N)),
             scale=torch.randint(1, 3, (n,), generator=g, device="cuda").float(),
             ids=torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32))
    if order == "packed":
        c["ids"] = c["ids"].sort().values
    return c


def formulas(c, xa=None):
    f = {k: v.double() for k, v in c.items()}
    x, xa, dY = f["x"], f["x"] if xa is None else xa.double(), f["dY"]
    out = {"y": x @ f["W"], "dX": dY @ f["W"].t(), "dXa": torch.zeros_like(x),
           "dA": torch.zeros_like(f["A"]), "dB": torch.zeros_like(f["B"])}
    for a in range(len(f["A"])):
        t = (c["ids"] == a).nonzero().flatten()
        A, B = f["A"][a], f["B"][a]
        u, v = f["scale"][a] * (xa[t] @ A.t()), f["scale"][a] * (dY[t] @ B.t())
        assert max(float(w.abs().amax()) if w.numel() else 0 for w in (u, v)) < 2 ** 16
        out["y"][t] += u @ B
        out["dXa"][t] = v @ A
        out["dA"][a], out["dB"][a] = v.t() @ xa[t], u.t() @ dY[t]
    return out


def near(T, K, N, n, r):
    """The shape, then shapes of a few row tiles more or fewer."""
    for d in (0, 1, -1, 2, -2, 4, -4, 8, -8, 12, -12, 16, -16):
        if T + 128 * d > 0:
            yield T + 128 * d, K, N, n, r


def shape_of(form, shape, backward, own):
    for T, K, N, n, r in near(*shape):
        f = mok.mok_lora_get_forms(mok.MokLoraDims(T=T, K=K, N=N, n=n, r=r), backward, own)
        if form(f):
            return T, K, N, n, r
    pytest.fail(f"no shape near {shape} takes this form")


def check(shape, order, out, own=False, backward=True):
    c = case(*shape, order)
    T = shape[0]
    g = torch.Generator(device="cuda").manual_seed(7)
    xa = whole(g, c["x"].shape, 1) if own else None
    L = AdaptedLinear(c["W"], c["A"], c["B"], c["scale"])
    y, saved = L.forward(c["x"], c["ids"], x_ad=xa, out=out)
    got = {"y": y}
    if backward:
        got.update(L.backward(c["x"], c["ids"], saved, c["dY"], x_ad=xa, out=out))
    want = formulas(c, xa)
    if not own:
        want["dX"] = want["dX"] + want["dXa"]
    for k, v in got.items():
        w = want[k]
        most = float(w.abs().amax())
        assert most < 2 ** 24
        steps = T / 8 + 32 if k in ("dA", "dB") else 32
        tol = 0.25 + steps * 2.0 ** -22 * most + (2.0 ** -8 * w.abs() if out == torch.bfloat16 else 0)
        off = ((v.double() - w).abs() - tol).amax()
        assert off <= 0, (k, float(off), most)
    assert L.status() == 0


def proj(columns, split, pair=0, halved=None, part="proj"):
    def form(f):
        p = getattr(f, part)
        return (p.columns, p.split, p.pair) == (columns, split, pair) and halved in (None, p.halved > 0)

    return form


FORWARD = [
    ((1, 64, 64, 2, 8), proj(64, 1)), ((1, 264, 64, 6, 100), proj(64, 2)),
    ((1, 520, 64, 2, 8), proj(64, 4)), ((1, 1032, 64, 2, 8), proj(64, 8)),
    ((1, 64, 7168, 2, 8), proj(128, 1)), ((1, 1032, 7168, 2, 8), proj(128, 2)),
    ((1, 520, 2056, 2, 8), proj(128, 4)), ((1, 1032, 1032, 2, 8), proj(128, 8)),
    ((257, 64, 7168, 2, 8), proj(192, 1)), ((520, 64, 7168, 2, 8), proj(256, 1)),
    ((6000, 64, 1032, 6, 100), proj(256, 1, 1, False)), ((8192, 64, 520, 6, 100), proj(256, 1, 1, True)),
    ((8192, 7168, 2048, 12, 32), proj(256, 1, 1, True)),
]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape,form", FORWARD, ids=lambda v: "x".join(map(str, v)) if type(v) is tuple else "")
def test_forms_of_the_forward_projection(shape, form, out):
    check(shape_of(form, shape, False, False), "rows" if shape[0] < 8192 else "packed", out, backward=False)


BACKWARD = [
    ((1, 64, 64, 2, 8), proj(64, 1)), ((1, 64, 264, 6, 100), proj(64, 2)),
    ((1, 64, 520, 2, 8), proj(64, 4)), ((1, 64, 1032, 2, 8), proj(64, 8)),
    ((1, 7168, 64, 2, 8), proj(128, 1)), ((1, 7168, 1032, 2, 8), proj(128, 2)),
    ((1, 2056, 520, 2, 8), proj(128, 4)), ((1, 1032, 1032, 2, 8), proj(128, 8)),
    ((257, 7168, 64, 2, 8), proj(192, 1)), ((129, 16400, 64, 2, 8), proj(256, 1)),
    ((129, 16400, 64, 6, 100), proj(256, 1, 1)), ((6000, 1032, 64, 6, 100), proj(256, 1, 1, False)),
    ((8192, 520, 64, 6, 100), proj(256, 1, 1, True)), ((8192, 7168, 2048, 4, 16), proj(256, 1, 1)),
]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape,form", BACKWARD, ids=lambda v: "x".join(map(str, v)) if type(v) is tuple else "")
def test_forms_of_the_backward_projection(shape, form, out):
    check(shape_of(form, shape, True, False), "rows" if shape[0] < 8192 else "packed", out)


APART = [
    ((1, 64, 64, 2, 8), proj(64, 1, part="adapters")), ((1, 7168, 64, 2, 8), proj(128, 1, part="adapters")),
    ((257, 7168, 64, 2, 8), proj(192, 1, part="adapters")),
    ((129, 16400, 64, 2, 8), proj(256, 1, part="adapters")),
    ((129, 16400, 64, 6, 100), proj(256, 1, 1, part="adapters")),
    ((8192, 520, 64, 6, 100), proj(256, 1, 1, True, part="adapters")),
    ((8192, 7168, 2048, 4, 16), proj(256, 1, part="adapters")),
    ((1, 7168, 2056, 2, 8), proj(128, 2)), ((257, 1032, 4104, 2, 8), proj(64, 2)),
    ((129, 16400, 264, 2, 8), proj(256, 1, 1)), ((8192, 520, 520, 2, 8), proj(256, 1, 1, True)),
]


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape,form", APART, ids=lambda v: "x".join(map(str, v)) if type(v) is tuple else "")
def test_forms_with_an_adapter_input_of_its_own(shape, form, out):
    check(shape_of(form, shape, True, True), "rows", out, own=True)


def u_rows(ranks):
    return lambda f: f.u_ranks == ranks


def u_tiles(split, several):
    return lambda f: (f.u_ranks, f.u_split, f.u_chunks > 1) == (0, split, several)


@pytest.mark.parametrize("shape,form", [
    ((1, 64, 64, 2, 8), u_rows(2)), ((5, 64, 64, 48, 40), u_rows(4)), ((40, 64, 64, 2, 8), u_rows(8)),
    ((40, 64, 64, 12, 24), u_rows(16)), ((129, 64, 64, 2, 8), u_rows(16)),
    ((257, 64, 64, 2, 8), u_tiles(1, False)), ((257, 64, 64, 130, 16), u_tiles(1, True)),
    ((257, 264, 64, 6, 100), u_tiles(2, True)), ((257, 520, 64, 12, 24), u_tiles(4, True)),
    ((520, 4104, 64, 130, 16), u_tiles(8, True)), ((8192, 1032, 64, 6, 100), u_tiles(2, False)),
    ((4100, 2056, 64, 6, 100), u_tiles(4, False)),
    # fewer rows than a tile, in tiles: the stages are short, the MMA reads past them
    ((1, 16400, 64, 2, 8), u_tiles(8, False)), ((1, 16400, 64, 48, 40), u_tiles(8, False)),
    ((40, 16400, 64, 130, 16), u_tiles(8, True)), ((100, 2056, 64, 6, 100), u_tiles(8, True)),
    ((100, 4104, 64, 48, 40), u_tiles(8, True)), ((13, 16400, 64, 12, 24), u_tiles(8, True)),
], ids=lambda v: "x".join(map(str, v)) if type(v) is tuple else "")
def test_forms_of_u(shape, form):
    check(shape_of(form, shape, False, False), "rows", torch.float32, backward=False)


@pytest.mark.parametrize("order", ["rows", "packed"])
@pytest.mark.parametrize("T,K,N,columns,split", [
    (1, 64, 64, 128, 1), (129, 64, 64, 128, 2), (257, 64, 64, 128, 4), (520, 64, 64, 128, 8),
    (2050, 16400, 4104, 256, 1), (2050, 16400, 64, 256, 2), (2050, 64, 4104, 256, 4), (2050, 64, 64, 256, 8)])
@pytest.mark.parametrize("n,r", [(2, 8), (12, 24), (48, 40), (6, 100)])
def test_forms_of_the_weight_gradients(T, K, N, columns, split, n, r, order):
    wide = 128 if r > 64 else columns

    def form(f):
        return f.grad_columns == wide and (f.grad_split == split or wide != columns)

    check(shape_of(form, (T, K, N, n, r), True, False), order, torch.float32)


def test_forms_of_an_empty_batch_and_refusals():
    f = mok.mok_lora_get_forms(mok.MokLoraDims(T=0, K=64, N=64, n=1, r=1), True, True)
    assert f.proj.columns == f.adapters.columns == f.grad_columns == 0
    with pytest.raises(mok.MokError):
        mok.mok_lora_get_forms(mok.MokLoraDims(T=1, K=12, N=64, n=1, r=1))

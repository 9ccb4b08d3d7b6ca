"""The operators together: the block of examples/adapted_moe.py against the same block written
in plain fp32 torch, differentiated by autograd."""
import pytest
import torch

from examples import adapted_moe as ex
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


def plain(s, w, x, ids, idx, mask):
    """y of the block in fp32 at the given choice; adapters, x are leaves."""
    T = x.shape[0]
    xa = x if mask is None else x * mask

    def proj(name, v, va):
        y = v @ w[name]
        for a in range(s.tenants):
            rows = ids == a
            low = (va[rows] @ w[name + ".A"][a].t()) @ w[name + ".B"][a]
            y = y.index_put((rows.nonzero().flatten(),), w["scale"][a] * low, accumulate=True)
        return y

    sc = torch.sigmoid(proj("router", x, xa)).gather(1, idx.long())
    gates = 1.5 * sc / sc.sum(1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(s.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        h = torch.nn.functional.silu(x[t] @ w["W_gate"][e]) * (x[t] @ w["W_up"][e])
        y = y.index_put((t,), gates[t, j, None] * (h @ w["W_down"][e]), accumulate=True)
    h = torch.nn.functional.silu(proj("gate", x, xa)) * proj("up", x, xa)
    return y + proj("down", h, h)


@pytest.mark.parametrize("seed", [None, 77])
def test_block_matches_autograd(seed):
    """bf16 operands and results through a chain of at most four products against fp32 ones:
    each rounding is 2^-8 of a value, so 4 x 2^-8 of the largest magnitude, 2%, holds with room
    for sums whose terms cancel (largest against largest, not element against element)."""
    s, T = ex.Sizes(), 200
    w = ex.make_weights(s, seed=3)
    for n in ex.AdaptedMoEBlock.PROJECTIONS:            # adapters that matter
        w[n + ".B"].copy_(torch.randn(w[n + ".B"].shape, device="cuda") * 0.05)
    x = torch.randn(T, s.H, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, s.tenants, (T,), device="cuda", dtype=torch.int32)
    dY = torch.randn(T, s.H, device="cuda").to(torch.bfloat16)
    block = ex.AdaptedMoEBlock(s, T, w)
    y = block.forward(x, ids, seed=seed)
    idx = block.kept[5]
    dX, grads = block.backward(dY)
    assert block.status() == 0

    mask = None
    if seed is not None:
        t = round(65536 * s.p)
        keep = torch.tensor(ref.dropout_words(x.numel(), seed, 0) >= t, device="cuda").reshape(x.shape)
        mask = keep.float() * 65536 / (65536 - t)
    v = {k: t.float().requires_grad_(k.endswith((".A", ".B"))) for k, t in w.items()}
    xf = x.float().requires_grad_()
    out = plain(s, v, xf, ids, idx, mask)
    out.backward(dY.float())

    def close(got, want, what):
        err = (got.float() - want).abs().max() / want.abs().max()
        assert err <= 0.02, (what, float(err))

    close(y, out.detach(), "y")
    close(dX, xf.grad, "dX")
    for n, (dA, dB) in grads.items():
        close(dA, v[n + ".A"].grad, n + ".A")
        close(dB, v[n + ".B"].grad, n + ".B")


def test_adapters_learn_and_serve():
    s, T = ex.Sizes(p=0.05), 256
    w = ex.make_weights(s, seed=5)
    x = torch.randn(T, s.H, device="cuda").to(torch.bfloat16)
    ids = (torch.arange(T, device="cuda") % s.tenants).to(torch.int32)
    block = ex.AdaptedMoEBlock(s, T, w)
    frozen = w["down"].clone()
    target = block.forward(x, ids).float() + 0.2 * torch.tanh(x.float())
    losses = ex.train(block, x, ids, target, steps=25, lr=30.0)
    assert losses[-1] < 0.97 * losses[0] and torch.equal(frozen, w["down"])
    y = block.forward(x, ids)
    one = ex.AdaptedMoEBlock(s, 1, w)                   # a single token on its own
    got = one.forward(x[5:6].contiguous(), ids[5:6].contiguous())
    assert (got.float() - y[5:6].float()).abs().max() <= 0.02 * y.float().abs().max()
    assert block.status() == 0 and one.status() == 0

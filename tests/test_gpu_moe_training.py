"""The norm, the routing, the balance loss, the experts, the gradient norm and the AdamW step
together: the block of examples/moe_training.py against the same block in plain fp32 torch,
differentiated by autograd, and its training loop eager and captured."""
import pytest
import torch

from examples import moe_training as ex

pytestmark = pytest.mark.gpu


def plain(s, w, x, residual, idx, seqs):
    """(out, losses) of the block in fp32 at the given choice; the weights and x are leaves."""
    h = x + residual
    z = h * torch.rsqrt((h * h).mean(1, keepdim=True) + 1e-5) * w["norm"]
    logits = z @ w["Wr"]
    idx = idx.long()
    gates = torch.softmax(logits.gather(1, idx), 1)          # renormalised softmax scores
    y = torch.zeros_like(x)
    for e in range(s.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        a = torch.nn.functional.silu(z[t] @ w["W_gate"][e]) * (z[t] @ w["W_up"][e])
        y = y.index_put((t,), gates[t, j, None] * (a @ w["W_down"][e]), accumulate=True)
    balance = zloss = 0.0
    p, total = torch.softmax(logits, 1), seqs[-1] - seqs[0]
    for lo, hi in zip(seqs, seqs[1:]):
        share = torch.bincount(idx[lo:hi].reshape(-1), minlength=s.E) / (s.k * (hi - lo))
        balance = balance + s.coef * s.E * (share * p[lo:hi].mean(0)).sum() * (hi - lo) / total
        zloss = zloss + s.z_coef * (torch.logsumexp(logits[lo:hi], 1) ** 2).sum() / total
    return h + y, balance, zloss


def data(s, T, seed):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(T, s.H, generator=g).to(torch.bfloat16).cuda() for _ in range(3)]


@pytest.mark.parametrize("seqs", [[0, 200], [0, 60, 61, 180]])
def test_block_matches_autograd(seqs):
    """bf16 operands and results through a chain of at most four products and the norm: 4 x 2^-8 of
    the largest magnitude, and as much again for the norm's input and output, 4 %. The losses come
    from fp32 logits of a bf16 z: 2^-8 |logit| on each, which moves a softmax share by that and the
    losses by less than 2 %."""
    s, T = ex.Sizes(coef=0.5, z_coef=0.02), 200
    w = ex.make_weights(s, seed=3)
    w["norm"].copy_(1 + 0.2 * torch.randn(s.H, device="cuda"))
    x, residual, dout = data(s, T, 4)
    block = ex.MoEBlock(s, T, w)
    out, losses, counts = block.forward(x, residual,
                                        torch.tensor(seqs, dtype=torch.int32, device="cuda"))
    idx = block.kept[4]
    got = block.backward(dout)
    assert block.status() == 0
    assert torch.equal(counts.long(), torch.bincount(idx[:seqs[-1]].reshape(-1).long(), minlength=s.E))

    v = {k: t.float().requires_grad_() for k, t in w.items()}
    xf = x.float().requires_grad_()
    want, balance, zloss = plain(s, v, xf, residual.float(), idx, seqs)
    ((want * dout.float()).sum() + balance + zloss).backward()

    def close(a, b, what, tol=0.04):
        err = (a.float() - b).abs().max() / b.abs().max()
        assert err <= tol, (what, float(err))

    close(out, want.detach(), "out")
    close(losses, torch.stack([balance, zloss]).detach(), "losses", 0.02)
    close(got["dX"], xf.grad, "dX")
    for n in ex.NAMES:
        close(got[ex.GRADS[n]], v[n].grad, n)


@pytest.mark.parametrize("bits", [8, 32])
def test_a_captured_training_step_equals_the_eager_one(bits):
    s, T = ex.Sizes(), 256
    x, residual, other = data(s, T, 9)
    target = residual.float() + 0.3 * torch.tanh(other.float())
    seqs = torch.tensor([0, 100, 250], dtype=torch.int32, device="cuda")

    def make():
        w = ex.make_weights(s, seed=5)
        return w, ex.MoEBlock(s, T, w), ex.make_optimizer(w, bits), torch.zeros(1, dtype=torch.int32, device="cuda")

    lr = torch.full((1,), 1e-3, device="cuda")
    w, block, opt, t = make()
    v, twin, eager, n = make()

    def one(block, opt, t):
        t.add_(1)
        return ex.train_step(block, opt, x, residual, target, lr, step=t, seqs=seqs)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        one(block, opt, t)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = one(block, opt, t)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for _ in range(4):
        want = one(twin, eager, n)
    assert int(t) == int(n) == 4
    for a, b in zip([*got, *w.values(), opt.m, opt.v, opt.master], [*want, *v.values(), eager.m, eager.v, eager.master]):
        assert torch.equal(a, b)
    assert block.status() == 0 and twin.status() == 0


def test_the_example_runs(capsys):
    ex.main()
    assert "steps 41 status 0" in capsys.readouterr().out

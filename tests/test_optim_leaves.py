"""AdamW over leaves of autograd, a module's parameters: its state is no part of a graph."""
import copy

import pytest
import torch

from grouped_gemm_built_gb300.optim import AdamW


def test_masters_of_leaves_are_plain_tensors():
    leaf = torch.nn.Parameter(torch.randn(300).to(torch.bfloat16))
    opt = AdamW.__new__(AdamW)                       # without a device: only what read_params needs
    opt.params, opt.master = (leaf, torch.zeros(5)), torch.zeros(768)
    for _ in range(2):
        opt.read_params()
        assert not opt.master.requires_grad and opt.master.grad_fn is None
    assert torch.equal(opt.master[:300], leaf.detach().float()) and not opt.master[300:].any()
    copy.deepcopy(opt.master)                        # which a tensor inside a graph refuses


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_steps_on_a_modules_parameters(bits):
    """The same steps with leaves and with plain tensors, gradients from autograd."""
    torch.manual_seed(0)
    lin = torch.nn.Linear(40, 30, dtype=torch.bfloat16, device="cuda")
    plain = [p.detach().clone() for p in lin.parameters()]
    a, b = (AdamW(list(ps), weight_decay=0.1, bits=bits, seed=4) for ps in (lin.parameters(), plain))
    for k in range(3):
        lin.zero_grad()
        lin(torch.randn(7, 40, device="cuda", dtype=torch.bfloat16)).square().sum().backward()
        grads = [p.grad for p in lin.parameters()]
        a.step(grads, lr=0.01)
        b.step(grads, lr=0.01)
    for t in (a.master, a.m, a.v, a.scales):
        assert t is None or (not t.requires_grad and t.grad_fn is None)
    assert all(torch.equal(p, q) for p, q in zip(lin.parameters(), plain))
    assert torch.equal(a.master, b.master) and torch.equal(a.m, b.m) and torch.equal(a.v, b.v)
    a.read_params()
    assert a.master.grad_fn is None
    again = copy.deepcopy((a.master, a.m, a.v, a.scales))
    assert torch.equal(again[0], a.master)

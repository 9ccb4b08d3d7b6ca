"""The objects that programs keep between calls, on the GPU: copies of a rule, replaced weights."""
import copy
import gc
import pickle

import pytest
import torch

from grouped_gemm_built_gb300.lora import AdaptedLinear
from grouped_gemm_built_gb300.routing import Routing

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("again", [copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
def test_copied_rules_outlive_the_original(again):
    """The copy gives the original's results when the original is gone and its memory reused."""
    l = torch.randn(33, 64, device="cuda")
    R = Routing(64, 4, score="sigmoid", groups=8, top_groups=3, scale=2.5)
    idx, gates = R.forward(l)
    dl = R.backward(l, idx, torch.ones_like(gates))
    C = again(R)
    del R
    gc.collect()
    others = [Routing(7, 1) for _ in range(64)]
    got = C.forward(l)
    assert torch.equal(got[0], idx) and torch.equal(got[1], gates)
    assert torch.equal(C.backward(l, idx, torch.ones_like(gates)), dl)
    assert len(others) == 64


def bf(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def step(L, x, ids, dY):
    y, saved = L.forward(x, ids)
    return dict(L.backward(x, ids, saved, dY), y=y)


@pytest.mark.parametrize("name", ["W", "A", "B", "scale"])
@pytest.mark.parametrize("how", ["attribute", "data", "set_"])
def test_replaced_weights_are_what_the_next_call_reads(name, how):
    """Another tensor in the weight's place, or other storage under the same tensor."""
    x, dY = bf(50, 64), bf(50, 40)
    ids = (torch.arange(50, device="cuda") % 4 - 1).to(torch.int32)
    w = {"W": bf(64, 40), "A": bf(3, 5, 64), "B": bf(3, 5, 40), "scale": torch.rand(3, device="cuda")}
    L = AdaptedLinear(**w)
    step(L, x, ids, dY)
    new = dict(w, **{name: torch.randn_like(w[name].float()).to(w[name].dtype)})
    want = step(AdaptedLinear(**{k: v.clone() for k, v in new.items()}), x, ids, dY)
    if how == "attribute":
        setattr(L, name, new[name])
    elif how == "data":
        w[name].data = new[name].clone()
    else:
        w[name].set_(new[name].clone())
    got = step(L, x, ids, dY)
    for k, v in want.items():
        assert torch.equal(got[k], v), k


def test_copied_projections_have_weights_of_their_own():
    x, dY = bf(50, 64), bf(50, 40)
    ids = (torch.arange(50, device="cuda") % 4 - 1).to(torch.int32)
    L = AdaptedLinear(bf(64, 40), bf(3, 5, 64), bf(3, 5, 40), torch.rand(3, device="cuda"))
    want = step(L, x, ids, dY)
    C = copy.deepcopy(L)
    for t in (L.W, L.A, L.B, L.scale):
        t.zero_()
    for k, v in step(C, x, ids, dY).items():
        assert torch.equal(v, want[k]), k

"""The objects that programs keep between calls, on the GPU: copies of a rule, replaced weights."""
import copy
import gc
import pickle

import pytest
import torch

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

"""The objects that programs keep between calls, without a GPU: copies and pickles stand on
their own, and tensors that do not belong together are refused."""
import copy
import ctypes
import pickle

import pytest
import torch

from grouped_gemm_built_gb300 import build, mok
from grouped_gemm_built_gb300.lora import AdaptedLinear
from grouped_gemm_built_gb300.routing import Routing


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    mok.lib()


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
def test_a_copied_rule_holds_no_address_of_the_original(again):
    R = Routing(64, 4, score="sigmoid", groups=8, top_groups=3, scale=2.5)
    at = ctypes.addressof(R.rule)
    C = again(R)
    assert at not in [v for v in vars(C).values() if isinstance(v, int)]
    assert [getattr(C.rule, n) for n, _ in C.rule._fields_] == [64, 4, 1, 8, 3, 0, 1, 2.5]


def test_a_call_reads_the_rule_object_itself():
    """Anything else in its place is an error, not an address to read from."""
    calls = mok.torch_calls()
    for wrong in (12345, mok.MokLoraDims()):
        with pytest.raises(TypeError):
            calls.route(wrong, torch.zeros(3, 64), None)
        with pytest.raises(TypeError):
            calls.route_bwd(wrong, torch.zeros(3, 64), None, None, mok.MOK_OUT_F32)


class _On(torch.Tensor):
    """A host tensor that claims to be on a CUDA device of its own, for the checks only."""

    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.index_)


def on(index, *shape, dtype=torch.bfloat16):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(_On)
    t.index_ = index
    return t


@pytest.mark.parametrize("name", ["A", "B", "scale"])
def test_weights_share_a_device(name):
    w = dict(W=on(0, 64, 32), A=on(0, 2, 4, 64), B=on(0, 2, 4, 32),
             scale=on(0, 2, dtype=torch.float32))
    w[name].index_ = 1
    with pytest.raises(ValueError, match=f"{name} must be on W's device cuda:0, got cuda:1"):
        AdaptedLinear(**w)


def test_rows_are_on_the_device_of_the_weights():
    L = AdaptedLinear.__new__(AdaptedLinear)
    L.K, L.N, L.n, L.r, L.device = 64, 32, 2, 4, torch.device("cuda", 0)
    x, ids = on(1, 3, 64), on(1, 3, dtype=torch.int32)
    saved = on(1, mok.mok_lora_get_sizes(mok.MokLoraDims(T=3, K=64, N=32, n=2, r=4)).saved_bytes,
               dtype=torch.uint8)
    with pytest.raises(ValueError, match="x must be on the weights' device cuda:0, got cuda:1"):
        L.forward(x, ids)
    with pytest.raises(ValueError, match="x must be on the weights' device cuda:0, got cuda:1"):
        L.backward(x, ids, saved, on(1, 3, 32))


def test_replaced_weights_are_checked_at_the_call(monkeypatch):
    """Weights that another tensor has replaced: the call looks at that one."""
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, _z=torch.zeros, **k: _z(*a, **k))
    W, A = on(0, 64, 32), on(0, 2, 4, 64)
    L = AdaptedLinear(W, A, on(0, 2, 4, 32), on(0, 2, dtype=torch.float32))
    x, ids = on(0, 3, 64), on(0, 3, dtype=torch.int32)
    for name, wrong, what in (("A", on(1, 2, 4, 64), "A must be on"), ("A", on(0, 2, 64, 4), r"A must be \["),
                              ("W", on(0, 64, 40), "W must have"), ("scale", on(0, 2), "scale must be"),
                              ("B", torch.zeros(2, 4, 32, dtype=torch.bfloat16), "B must be on a CUDA")):
        right = getattr(L, name)
        setattr(L, name, wrong)
        with pytest.raises(ValueError, match=what):
            L.forward(x, ids)
        setattr(L, name, right)
    A.set_(on(0, 2, 3, 64))
    with pytest.raises(ValueError, match="A must have"):
        L.forward(x, ids)

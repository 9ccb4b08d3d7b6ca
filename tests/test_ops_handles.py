"""The objects that programs keep between calls, without a GPU: copies and pickles stand on
their own, and tensors that do not belong together are refused."""
import copy
import ctypes
import pickle

import pytest
import torch

from grouped_gemm_built_gb300 import build, mok
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

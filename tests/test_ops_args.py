"""Refusals of the operators in include/mok_ops.h, without a GPU: the library checks its
arguments before it touches the device, and the torch-facing classes check their tensors
before they hand out an address."""
import pytest
import torch

from grouped_gemm_built_gb300 import build, mok
from grouped_gemm_built_gb300.dropout import dropout
from grouped_gemm_built_gb300.lora import AdaptedLinear
from grouped_gemm_built_gb300.routing import Routing
from tests.test_layer_args import dev

INVALID, WORKSPACE = mok.MOK_ERR_INVALID_ARG, mok.MOK_ERR_WORKSPACE
F32, BF = mok.MOK_OUT_F32, mok.MOK_OUT_BF16


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    mok.lib()


def refused(status, fn, *args):
    with pytest.raises(mok.MokError) as ei:
        fn(*args)
    assert ei.value.status == status


def rule(**over):
    base = dict(E=64, k=4, score=0, groups=1, top_groups=1, group_score=0, renormalize=1, scale=1.0)
    base.update(over)
    return mok.MokRouting(**base)


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=513), dict(k=0), dict(k=33), dict(E=3, k=4), dict(score=2), dict(score=-1),
    dict(group_score=2), dict(groups=0), dict(groups=5), dict(groups=33, E=66), dict(top_groups=0),
    dict(groups=4, top_groups=5), dict(groups=32, top_groups=1, k=4), dict(scale=float("nan")),
    dict(scale=float("inf"))])
def test_route_refuses_bad_rules(bad):
    refused(INVALID, mok.mok_route, rule(**bad), 4, 16, F32, None, 16, 16, None)
    refused(INVALID, mok.mok_route_bwd, rule(**bad), 4, 16, F32, 16, 16, 16, F32, None)


@pytest.mark.parametrize("T,logits,kind,bias,idx,gates", [
    (-1, 16, F32, None, 16, 16), (4, None, F32, None, 16, 16), (4, 16, 2, None, 16, 16),
    (4, 16, F32, None, None, 16), (4, 16, F32, None, 16, None), (4, 18, F32, None, 16, 16),
    (4, 17, BF, None, 16, 16), (4, 16, F32, 6, 16, 16), (4, 16, F32, None, 18, 16)])
def test_route_refuses_bad_buffers(T, logits, kind, bias, idx, gates):
    refused(INVALID, mok.mok_route, rule(), T, logits, kind, bias, idx, gates, None)


def test_zero_rows_are_a_valid_call():
    mok.mok_route(rule(), 0, None, F32, None, None, None, None)
    mok.mok_route_bwd(rule(), 0, None, F32, None, None, None, F32, None)
    mok.mok_dropout(None, None, None, 0, 0.5, 0, 0, BF, None)
    mok.mok_lora_fwd(lora_dims(T=0), lora_weights(), None, None, None, None, BF, None, None, None)


def test_route_bwd_refuses_bad_buffers():
    for args in ((None, F32, 16, 16, 16, F32), (16, F32, None, 16, 16, F32),
                 (16, F32, 16, None, 16, F32), (16, F32, 16, 16, None, F32),
                 (16, F32, 16, 16, 16, 5), (16, F32, 16, 16, 18, F32)):
        refused(INVALID, mok.mok_route_bwd, rule(), 4, *args, None)


@pytest.mark.parametrize("x,add,y,p,kind", [
    (None, None, 16, 0.1, BF), (16, None, None, 0.1, BF), (16, None, 16, -0.1, BF),
    (16, None, 16, 1.0, BF), (16, None, 16, float("nan"), BF), (16, None, 16, 0.999999, BF),
    (16, None, 16, 0.1, 2), (17, None, 16, 0.1, BF), (16, 18, 16, 0.1, F32)])
def test_dropout_refuses(x, add, y, p, kind):
    refused(INVALID, mok.mok_dropout, x, add, y, 8, p, 0, 0, kind, None)


def lora_dims(**over):
    base = dict(T=4, K=64, N=64, n=2, r=4)
    base.update(over)
    return mok.MokLoraDims(**base)


def lora_weights(**over):
    base = dict(W=256, A=256, B=256, scale=256)
    base.update(over)
    return mok.MokLoraWeights(**base)


@pytest.mark.parametrize("bad", [dict(T=-1), dict(K=0), dict(K=12), dict(N=0), dict(N=65),
                                 dict(n=0), dict(r=0), dict(r=129)])
def test_lora_refuses_bad_dims(bad):
    refused(INVALID, mok.mok_lora_get_sizes, lora_dims(**bad))
    refused(INVALID, mok.mok_lora_fwd, lora_dims(**bad), lora_weights(), 256, None, 256, 256, BF,
            256, None, None)


def test_lora_refuses_bad_buffers():
    d = lora_dims()
    fwd = dict(x=256, x_ad=None, ids=256, y=256, out=BF, saved=256, status=None)
    for bad in (dict(x=None), dict(x=264), dict(x_ad=258), dict(ids=None), dict(ids=258),
                dict(y=None), dict(y=264), dict(out=7), dict(status=258)):
        refused(INVALID, mok.mok_lora_fwd, d, lora_weights(), *{**fwd, **bad}.values(), None)
    for bad in (dict(saved=None), dict(saved=128)):
        refused(WORKSPACE, mok.mok_lora_fwd, d, lora_weights(), *{**fwd, **bad}.values(), None)
    for bad in (dict(W=None), dict(W=264), dict(A=None), dict(B=264), dict(scale=None)):
        refused(INVALID, mok.mok_lora_fwd, d, lora_weights(**bad), *fwd.values(), None)
    bwd = dict(x=256, x_ad=None, ids=256, saved=256, dY=256, dX=256, dXa=None, dA=256, dB=256,
               out=BF, workspace=256, status=None)
    for bad in (dict(x=None), dict(dY=None), dict(dX=264), dict(dA=None), dict(dB=None),
                dict(out=-1), dict(dXa=256), dict(x_ad=256), dict(ids=None)):
        refused(INVALID, mok.mok_lora_bwd, d, lora_weights(), *{**bwd, **bad}.values(), None)
    for bad in (dict(saved=None), dict(workspace=None), dict(workspace=64)):
        refused(WORKSPACE, mok.mok_lora_bwd, d, lora_weights(), *{**bwd, **bad}.values(), None)
    refused(INVALID, lambda: mok._check(mok.mok_lora_get_status(None, None), "status"))


def test_lora_sizes_grow_with_rows_and_rank():
    def sizes(**over):
        s = mok.mok_lora_get_sizes(lora_dims(**over))
        return s.saved_bytes, s.workspace_bytes

    base, rows, rank = sizes(T=1000), sizes(T=2000), sizes(T=1000, r=100)
    assert base[0] >= 1000 * 128 and rows[0] > base[0] and rank[0] >= 1000 * 4 * 128
    assert base[1] > base[0]


def test_torch_classes_check_their_tensors():
    with pytest.raises(ValueError, match="score"):
        Routing(64, 4, score="tanh")
    with pytest.raises(ValueError, match="group_score"):
        Routing(64, 4, group_score="mean")
    with pytest.raises(mok.MokError):
        Routing(64, 65)
    R = Routing(64, 4)
    with pytest.raises(ValueError, match="CUDA"):
        R.forward(torch.zeros(3, 64))
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        R.forward(dev(3, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match=r"\[T, 64\]"):
        R.forward(dev(3, 63))
    with pytest.raises(ValueError, match="contiguous"):
        R.forward(dev(64, 64).t())
    with pytest.raises(ValueError, match="bias"):
        R.forward(dev(3, 64), dev(63, dtype=torch.float32))
    with pytest.raises(ValueError, match="dgates"):
        R.backward(dev(3, 64), dev(3, 4, dtype=torch.int32), dev(3, 4))
    with pytest.raises(ValueError, match="CUDA"):
        dropout(torch.zeros(8), 0.5, 0)
    with pytest.raises(ValueError, match="float16"):
        dropout(dev(8, dtype=torch.float16), 0.5, 0)
    with pytest.raises(ValueError, match="add"):
        dropout(dev(8), 0.5, 0, add=dev(9))
    W, A, B, s = dev(64, 32), dev(2, 4, 64), dev(2, 4, 32), dev(2, dtype=torch.float32)
    with pytest.raises(ValueError, match="must be"):
        AdaptedLinear(W, A, dev(2, 3, 32), s)
    with pytest.raises(ValueError, match="scale"):
        AdaptedLinear(W, A, B, dev(3, dtype=torch.float32))
    with pytest.raises(ValueError, match="CUDA"):
        AdaptedLinear(W, torch.zeros(2, 4, 64, dtype=torch.bfloat16), B, s)
    with pytest.raises(TypeError, match="torch.Tensor"):
        AdaptedLinear([1], A, B, s)
    L = AdaptedLinear.__new__(AdaptedLinear)
    L.K, L.N, L.n, L.r = 64, 32, 2, 4
    with pytest.raises(ValueError, match="x must be"):
        L.forward(dev(3, 60), dev(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="ids"):
        L.forward(dev(3, 64), dev(3, dtype=torch.int64))
    with pytest.raises(ValueError, match="x_ad"):
        L.forward(dev(3, 64), dev(3, dtype=torch.int32), x_ad=dev(4, 64))
    with pytest.raises(ValueError, match="dY"):
        sizes = mok.mok_lora_get_sizes(lora_dims(T=3, N=32))
        L.backward(dev(3, 64), dev(3, dtype=torch.int32), dev(sizes.saved_bytes, dtype=torch.uint8),
                   dev(3, 31))

"""Refusals of the norm, the balance loss, the gradient norm and the AdamW step, without a GPU:
the library checks its arguments before it touches the device, the torch-facing classes check
their tensors before they hand out an address."""
import copy
import pickle

import pytest
import torch

from grouped_gemm_built_gb300 import build, mok
from grouped_gemm_built_gb300.balance import Balance
from grouped_gemm_built_gb300.norm import Norm
from grouped_gemm_built_gb300.optim import AdamW, grad_norm
from tests.test_layer_args import dev

INVALID, WORKSPACE = mok.MOK_ERR_INVALID_ARG, mok.MOK_ERR_WORKSPACE
F32, BF = mok.MOK_OUT_F32, mok.MOK_OUT_BF16
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    mok.lib()


def refused(status, fn, *args):
    with pytest.raises(mok.MokError) as ei:
        fn(*args)
    assert ei.value.status == status


# -------------------------------------------------------------------------------- norm
def norm_dims(**over):
    base = dict(T=4, H=64, kind=0, eps=1e-6, x_type=BF, y_type=BF, w_type=BF)
    base.update(over)
    return mok.MokNormDims(**base)


FWD = dict(x=256, add=None, w=256, b=None, h=None, y=256, stats=256)
BWD = dict(dY=256, h=256, w=256, stats=256, add=None, dX=256, dW=256, dB=None, workspace=256)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(H=32769), dict(kind=2), dict(kind=-1), dict(eps=-1e-9), dict(eps=NAN),
    dict(eps=INF), dict(x_type=2), dict(y_type=-1), dict(w_type=5)])
def test_norm_refuses_bad_dims(bad):
    d = norm_dims(**bad)
    refused(INVALID, mok.mok_norm_get_sizes, d)
    refused(INVALID, mok.mok_norm_fwd, d, *FWD.values(), None)
    refused(INVALID, mok.mok_norm_bwd, d, *BWD.values(), None)


def test_norm_refuses_bad_buffers():
    for bad in (dict(x=None), dict(w=None), dict(y=None), dict(add=256), dict(h=256), dict(x=257),
                dict(y=255), dict(w=129), dict(b=257), dict(stats=252), dict(add=257, h=256),
                dict(add=256, h=257)):
        refused(INVALID, mok.mok_norm_fwd, norm_dims(), *{**FWD, **bad}.values(), None)
    for bad in (dict(dY=None), dict(h=None), dict(w=None), dict(stats=None), dict(dX=None),
                dict(dW=None), dict(dY=257), dict(h=255), dict(add=3), dict(dX=257), dict(dW=1),
                dict(dB=1), dict(stats=260)):
        refused(INVALID, mok.mok_norm_bwd, norm_dims(), *{**BWD, **bad}.values(), None)
    for bad in (dict(workspace=None), dict(workspace=128)):
        refused(WORKSPACE, mok.mok_norm_bwd, norm_dims(), *{**BWD, **bad}.values(), None)
    wide = norm_dims(x_type=F32, y_type=F32, w_type=F32)
    for bad in (dict(x=258), dict(y=254), dict(w=258), dict(b=2)):
        refused(INVALID, mok.mok_norm_fwd, wide, *{**FWD, **bad}.values(), None)


def test_norm_without_rows_is_a_valid_forward():
    mok.mok_norm_fwd(norm_dims(T=0), None, None, None, None, None, None, None, None)
    assert mok.mok_norm_get_sizes(norm_dims(T=0)).stats_bytes == 0


def test_norm_class_checks_its_tensors():
    w = dev(64)
    with pytest.raises(ValueError, match="kind"):
        Norm(w, kind="batch")
    with pytest.raises(mok.MokError):
        Norm(w, eps=-1.0)
    with pytest.raises(ValueError, match="CUDA"):
        Norm(torch.zeros(64))
    with pytest.raises(ValueError, match="1 dimension"):
        Norm(dev(8, 8))
    with pytest.raises(ValueError, match="bias"):
        Norm(w, dev(63))
    with pytest.raises(ValueError, match="bias"):
        Norm(w, dev(64, dtype=torch.float32))
    with pytest.raises(TypeError, match="weight"):
        Norm([1.0])
    N = Norm(w)
    with pytest.raises(ValueError, match=r"\[T, 64\]"):
        N.forward(dev(3, 65))
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        N.forward(dev(3, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="contiguous"):
        N.forward(dev(64, 64).t())
    with pytest.raises(ValueError, match="add"):
        N.forward(dev(3, 64), add=dev(2, 64))
    with pytest.raises(ValueError, match="add"):
        N.forward(dev(3, 64), add=dev(3, 64, dtype=torch.float32))
    stats = dev(3, 2, dtype=torch.float32)
    with pytest.raises(ValueError, match="dY"):
        N.backward(dev(2, 64), dev(3, 64), stats)
    with pytest.raises(ValueError, match="stats"):
        N.backward(dev(3, 64), dev(3, 64), dev(3, dtype=torch.float32))
    with pytest.raises(ValueError, match="add"):
        N.backward(dev(3, 64), dev(3, 64), stats, add=dev(3, 65))
    N.weight = dev(63)
    with pytest.raises(ValueError, match="weight must have 64"):
        N.forward(dev(3, 64))


# ----------------------------------------------------------------------------- balance
def bal(**over):
    base = dict(E=64, k=4, score=0, coef=0.01, z_coef=0.0)
    base.update(over)
    return mok.MokBalance(**base)


@pytest.mark.parametrize("bad", [
    dict(E=0), dict(E=513), dict(k=0), dict(k=33), dict(score=2), dict(score=-1), dict(coef=-0.1),
    dict(coef=NAN), dict(coef=INF), dict(z_coef=-1.0), dict(z_coef=INF)])
def test_balance_refuses_bad_rules(bad):
    refused(INVALID, mok.mok_balance_get_sizes, bal(**bad), 4)
    refused(INVALID, mok.mok_balance_fwd, bal(**bad), 4, 256, F32, 256, None, 1, 256, 256, 256, None)
    refused(INVALID, mok.mok_balance_bwd, bal(**bad), 4, 256, F32, None, 1, 256, None, None, 256, F32,
            None)


def test_balance_refuses_bad_buffers():
    fwd = dict(T=4, logits=256, lt=F32, idx=256, seqs=None, S=1, losses=256, counts=256, saved=256)
    for bad in (dict(T=-1), dict(logits=None), dict(lt=2), dict(idx=None), dict(S=2), dict(S=0),
                dict(seqs=256, S=2**20 + 1), dict(seqs=258), dict(losses=None), dict(counts=None),
                dict(losses=254), dict(counts=258), dict(logits=254), dict(idx=1)):
        refused(INVALID, mok.mok_balance_fwd, bal(), *{**fwd, **bad}.values(), None)
    bwd = dict(T=4, logits=256, lt=F32, seqs=None, S=1, saved=256, dlosses=None, add=None, dl=256, dt=F32)
    for bad in (dict(T=-1), dict(logits=None), dict(lt=7), dict(S=3), dict(dlosses=2), dict(add=2),
                dict(dl=None), dict(dl=6), dict(dt=2)):
        refused(INVALID, mok.mok_balance_bwd, bal(), *{**bwd, **bad}.values(), None)
    for bad in (dict(saved=None), dict(saved=64)):
        refused(WORKSPACE, mok.mok_balance_fwd, bal(), *{**fwd, **bad}.values(), None)
        refused(WORKSPACE, mok.mok_balance_bwd, bal(), *{**bwd, **bad}.values(), None)
    mok.mok_balance_bwd(bal(), 0, None, F32, None, 1, None, None, None, None, F32, None)


def test_balance_class_checks_its_tensors():
    with pytest.raises(ValueError, match="score"):
        Balance(64, 4, score="tanh")
    with pytest.raises(mok.MokError):
        Balance(64, 4, coef=-1.0)
    B = Balance(64, 4)
    l, idx = dev(3, 64), dev(3, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        B.forward(torch.zeros(3, 64), idx)
    with pytest.raises(ValueError, match=r"\[T, 64\]"):
        B.forward(dev(3, 63), idx)
    with pytest.raises(ValueError, match="topk_idx"):
        B.forward(l, dev(3, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="topk_idx"):
        B.forward(l, dev(3, 4, dtype=torch.int64))
    with pytest.raises(ValueError, match="seqs"):
        B.forward(l, idx, dev(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="seqs"):
        B.forward(l, idx, dev(3, dtype=torch.int64))
    n = mok.mok_balance_get_sizes(B.rule, 3)
    saved = dev(n, dtype=torch.uint8)
    with pytest.raises(ValueError, match="saved"):
        B.backward(l, dev(n - 1, dtype=torch.uint8))
    with pytest.raises(ValueError, match="dlosses"):
        B.backward(l, saved, dlosses=dev(3, dtype=torch.float32))
    with pytest.raises(ValueError, match="add"):
        B.backward(l, saved, add=dev(3, 65))
    with pytest.raises(ValueError, match="add"):
        B.backward(l, saved, add=dev(3, 64), dtype=torch.float32)
    C = pickle.loads(pickle.dumps(copy.deepcopy(B)))
    assert [getattr(C.rule, f) for f, _ in C.rule._fields_] == [64, 4, 0, B.rule.coef, 0.0]


# ---------------------------------------------------------------------- gradient norm
def grad(**over):
    base = dict(g=256, n=8, type=BF)
    base.update(over)
    return mok.MokGrad(**base)


def test_grad_norm_refuses():
    ok = dict(max_norm=1.0, scale=1.0, norm=256, coef=256, ws=256)
    for bad in (dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=NAN), dict(scale=0.0),
                dict(scale=INF), dict(scale=NAN), dict(norm=None), dict(coef=None), dict(norm=2),
                dict(coef=258)):
        refused(INVALID, mok.mok_grad_norm, [grad()], *{**ok, **bad}.values(), None)
    for bad in (dict(type=2), dict(g=257), dict(g=258, type=F32), dict(n=2**63)):
        refused(INVALID, mok.mok_grad_norm, [grad(), grad(**bad)], *ok.values(), None)
    for bad in (dict(ws=None), dict(ws=8)):
        refused(WORKSPACE, mok.mok_grad_norm, [grad()], *{**ok, **bad}.values(), None)
    with pytest.raises(TypeError, match="list or tuple"):
        grad_norm(dev(8))
    with pytest.raises(ValueError, match="at least one"):
        grad_norm([None])
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        grad_norm([dev(8), torch.zeros(8)])
    with pytest.raises(ValueError, match=r"grads\[0\]"):
        grad_norm([dev(8, dtype=torch.float16)])


# ------------------------------------------------------------------------------- AdamW
def rule(**over):
    base = dict(beta1=0.9, beta2=0.95, eps=1e-8, bits=32)
    base.update(over)
    return mok.MokAdamwRule(**base)


def tensor(**over):
    base = dict(p=1 << 12, g=1 << 13, n=8, decay=0.0, p_type=F32, g_type=F32)
    base.update(over)
    return mok.MokAdamwTensor(**base)


def state(**over):
    base = dict(master=1 << 20, m=1 << 21, v=1 << 22, scales=1 << 23)
    base.update(over)
    return mok.MokAdamwState(**base)


def adamw_call(r=None, tensors=None, s=None, lr=1e-3, lr_dev=None, t=1, t_dev=None, coef=None):
    mok.mok_adamw(r or rule(), tensors or [tensor()], s or state(), lr, lr_dev, t, t_dev, coef, 0, None)


def test_adamw_refuses():
    for bad in (dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=NAN), dict(eps=0.0),
                dict(eps=1e-39), dict(eps=INF), dict(bits=16)):
        refused(INVALID, adamw_call, rule(**bad))
    for bad in (dict(p=None), dict(p=(1 << 12) + 2), dict(g=(1 << 13) + 1), dict(p_type=2),
                dict(g_type=-1), dict(decay=NAN), dict(decay=INF), dict(n=2**60)):
        refused(INVALID, adamw_call, None, [tensor(**bad)])
    for bad in (dict(m=None), dict(v=None), dict(m=(1 << 21) + 4), dict(v=(1 << 22) + 8)):
        refused(INVALID, adamw_call, None, None, state(**bad))
    refused(INVALID, adamw_call, rule(bits=8), None, state(scales=None))
    refused(INVALID, adamw_call, None, [tensor(p_type=BF)], state(master=None))
    for bad in (dict(lr=NAN), dict(lr=INF), dict(t=0), dict(t=-3), dict(lr_dev=2), dict(t_dev=6),
                dict(coef=1)):
        refused(INVALID, lambda kw=bad: adamw_call(**kw))


def test_adamw_refuses_tensors_that_overlap():
    a = tensor()
    refused(INVALID, adamw_call, None, [a, tensor()])                       # the same one twice
    refused(INVALID, adamw_call, None, [a, tensor(p=(1 << 12) + 28)])       # its last element
    refused(INVALID, adamw_call, None, [tensor(g=1 << 12)])                 # its own gradient
    refused(INVALID, adamw_call, None, [tensor(p=1 << 21)])                 # the state
    refused(INVALID, adamw_call, None, None, state(v=(1 << 21) + 1008))     # m and v
    refused(INVALID, adamw_call, None, [a, tensor(p=1 << 14, g=(1 << 12) + 4)])


def test_adamw_without_elements_is_a_valid_call():
    mok.mok_adamw(rule(), [], mok.MokAdamwState(), 0.1, None, 1, None, None, 0, None)
    mok.mok_adamw(rule(), [tensor(p=None, g=None, n=0)], mok.MokAdamwState(), 0.1, None, 1, None, None,
                  0, None)
    mok.mok_adamw_moments(0, mok.MokAdamwState(), None, None, None)
    assert mok.mok_adamw_get_sizes([]) == 0
    assert mok.mok_adamw_get_sizes([1, 256, 257, 0]) == 256 + 256 + 512
    refused(INVALID, mok.mok_adamw_get_sizes, [2**63, 2**63])
    ok = dict(m=256, v=512)
    refused(INVALID, mok.mok_adamw_moments, 255, state(), *ok.values(), None)
    for bad in (dict(m=None), dict(v=8)):
        refused(INVALID, mok.mok_adamw_moments, 256, state(), *{**ok, **bad}.values(), None)
    refused(INVALID, mok.mok_adamw_moments, 256, state(scales=None), *ok.values(), None)


def test_adamw_class_checks_its_tensors():
    with pytest.raises(ValueError, match="at least one"):
        AdamW([])
    with pytest.raises(ValueError, match=r"params\[1\]"):
        AdamW([dev(8), torch.zeros(8)])
    with pytest.raises(ValueError, match=r"params\[0\]"):
        AdamW([dev(8, dtype=torch.float16)])
    with pytest.raises(ValueError, match="weight_decay"):
        AdamW([dev(8), dev(9)], weight_decay=[0.1])
    with pytest.raises(ValueError, match="bits"):
        AdamW([dev(8)], bits=16)
    with pytest.raises(mok.MokError):
        AdamW([dev(8)], betas=(1.0, 0.9))
    opt = AdamW([dev(8, dtype=torch.float32), dev(3, 3)], weight_decay=0.1)
    assert opt.elements == 512 and opt.master.numel() == 512
    g = [dev(8), dev(3, 3)]
    for grads, what in (([dev(8)], "hold 2"), ([dev(7), dev(9)], r"grads\[0\]"), ((dev(8), [1]), r"grads\[1\]"),
                        ([torch.zeros(8), dev(9)], r"grads")):
        with pytest.raises((ValueError, TypeError), match=what):
            opt.step(grads, lr=0.1)
    with pytest.raises(ValueError, match="coef"):
        opt.step(g, lr=0.1, coef=dev(2, dtype=torch.float32))
    with pytest.raises(ValueError, match="lr"):
        opt.step(g, lr=dev(1))
    with pytest.raises(ValueError, match="step"):
        opt.step(g, lr=0.1, step=dev(1, dtype=torch.int64))
    opt.m = dev(511, dtype=torch.float32)
    with pytest.raises(ValueError, match="m must have 512"):
        opt.step(g, lr=0.1)
    assert opt.steps == 0

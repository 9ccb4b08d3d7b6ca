"""Tensors of the right number of elements and another shape: refused, on the CPU by the classes'
checks, on the GPU by the compiled calls (which alone look when all is well)."""
import pytest
import torch

from grouped_gemm_built_gb300 import build, mok
from grouped_gemm_built_gb300.balance import Balance
from grouped_gemm_built_gb300.norm import Norm
from grouped_gemm_built_gb300.optim import AdamW
from tests.test_layer_args import dev

I32, F32 = torch.int32, torch.float32


def on_gpu(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    mok.lib()


@pytest.fixture(params=[pytest.param(dev, id="cpu"), pytest.param(on_gpu, id="gpu", marks=pytest.mark.gpu)])
def make(request):
    return request.param


@pytest.mark.parametrize("shape", [(64, 3), (192,), (3, 8, 8), (1, 192), (6, 32)])
def test_norm(make, shape):
    N = Norm(make(64), kind="layer")
    x, stats = make(3, 64), make(3, 2, dtype=F32)
    with pytest.raises(ValueError, match="add"):
        N.forward(x, add=make(*shape))
    with pytest.raises(ValueError, match="dY"):
        N.backward(make(*shape), x, stats)
    with pytest.raises(ValueError, match="dY"):
        N.backward(make(*shape, dtype=F32), x, stats)
    with pytest.raises(ValueError, match="add"):
        N.backward(x, x, stats, add=make(*shape))


def test_norm_of_square_rows_transposed(make):
    """[H, T] with T = H has the shape, but not contiguous."""
    N = Norm(make(64))
    with pytest.raises(ValueError, match="contiguous"):
        N.backward(make(64, 64).t(), make(64, 64), make(64, 2, dtype=F32))


@pytest.mark.parametrize("shape", [(4, 3), (12,), (1, 12), (3, 4, 1), (6, 2)])
def test_balance_choices(make, shape):
    with pytest.raises(ValueError, match="topk_idx"):
        Balance(64, 4).forward(make(3, 64), make(*shape, dtype=I32))


@pytest.mark.parametrize("shape", [(64, 3), (192,), (1, 192), (3, 8, 8)])
def test_balance_gradient(make, shape):
    B = Balance(64, 4)
    saved = make(mok.mok_balance_get_sizes(B.rule, 3), dtype=torch.uint8)
    with pytest.raises(ValueError, match="add"):
        B.backward(make(3, 64), saved, add=make(*shape))
    with pytest.raises(ValueError, match="add"):
        B.backward(make(3, 64), saved, add=make(*shape, dtype=F32), dtype=F32)


def test_adamw_gradients(make):
    """A gradient has its tensor's shape, or is a flat view in its order."""
    opt = AdamW([make(8, 32), make(64), make(2, 3, 4)])
    good = [make(8, 32), make(64), make(2, 3, 4)]
    for i, shape in ((0, (32, 8)), (0, (1, 256)), (2, (4, 3, 2)), (2, (6, 4)), (2, (2, 12))):
        with pytest.raises(ValueError, match=rf"grads\[{i}\]"):
            opt.step(good[:i] + [make(*shape)] + good[i + 1:], lr=0.1)
    assert opt.steps == 0


@pytest.mark.gpu
def test_adamw_takes_flat_gradients():
    g = torch.randn(8, 32, generator=torch.Generator().manual_seed(1)).cuda()
    p, q, flat = (torch.ones(8, 32, device="cuda") for _ in range(3))
    for t, d in ((p, g), (q, g.view(-1))):
        AdamW([t]).step([d], lr=0.1)
    flat = flat.view(-1)
    AdamW([flat]).step([g], lr=0.1)
    assert torch.equal(p, q) and torch.equal(p.view(-1), flat) and not torch.equal(p, torch.ones_like(p))

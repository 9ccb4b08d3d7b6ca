"""mok_dropout on the GPU against the 64-bit form in ops_reference.py. fp32: x * up is one
rounding and the sum another, 2^-23 of the values' size; bf16: half a step of the result,
2^-8, on top. The mask itself must be equal."""
import numpy as np
import pytest
import torch

from grouped_gemm_built_gb300.dropout import dropout
from tests import ops_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 7, 8, 9, 2048, 4099])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("p,add", [(0.1, False), (0.5, True), (0.0, True), (0.9999, False)])
def test_values(n, dtype, p, add, rng):
    x = torch.tensor(rng.normal(size=n) + 4, dtype=dtype)       # no zeros: the mask shows
    a = torch.tensor(rng.normal(size=n), dtype=dtype) if add else None
    seed, offset = 0x123456789ABCDEF, 2 ** 40 + 5
    y = dropout(x.cuda(), p, seed, offset, add=None if a is None else a.cuda()).double().cpu().numpy()
    xd, ad = x.double().numpy(), None if a is None else a.double().numpy()
    want = ref.dropout(xd, p, seed, offset, ad)
    up = 65536 / (65536 - round(65536 * p))
    tol = 2.0 ** -22 * (np.abs(xd) * up + (0 if a is None else np.abs(ad)))
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    assert (np.abs(y - want) <= tol).all()
    if not add:
        assert np.array_equal(y != 0, ref.dropout_words(n, seed, offset) >= round(65536 * p))


def test_dropped_infinities_give_zero_and_kept_ones_stay():
    x = torch.full((4096,), float("nan"), device="cuda")
    x[::2] = float("inf")
    y = dropout(x, 0.5, 3)
    keep = torch.tensor(ref.dropout_words(4096, 3, 0) >= 32768, device="cuda")
    assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unaligned_tensors_and_offsets_continue_one_stream(dtype):
    x = torch.randn(8 * 100 + 3, device="cuda").to(dtype)
    whole = dropout(x, 0.3, 11)
    parts = [dropout(x[:400], 0.3, 11), dropout(x[400:], 0.3, 11, offset=50)]
    assert torch.equal(whole, torch.cat(parts))
    base = torch.randn(810, device="cuda").to(dtype)            # one element off 16 bytes
    base[1:804] = x
    assert torch.equal(dropout(base[1:804], 0.3, 11), whole)
    assert not torch.equal(dropout(x, 0.3, 12), whole)


def test_in_place_and_backward_is_the_same_call():
    x = torch.randn(1000, 33, device="cuda", dtype=torch.bfloat16)
    a = torch.randn_like(x)
    want = dropout(x, 0.2, 5, add=a)
    y = x.clone()
    assert dropout(y, 0.2, 5, add=a, y=y) is y and torch.equal(y, want)
    y = a.clone()
    assert torch.equal(dropout(x, 0.2, 5, add=y, y=y), want)
    # y = D x with D diagonal: the gradient of <dy, D x> is D dy
    dy = torch.randn_like(x)
    lhs = (dropout(x, 0.2, 5).double() * dy.double()).sum()
    rhs = (x.double() * dropout(dy, 0.2, 5).double()).sum()
    assert abs(lhs - rhs) <= 2.0 ** -8 * (x.double() * dy.double()).abs().sum()


def test_share_of_dropped_elements():
    """Binomial: 2^22 draws, six standard deviations."""
    n, p = 1 << 22, 0.1
    y = dropout(torch.ones(n, device="cuda"), p, 77)
    t = round(65536 * p) / 65536
    assert abs((y == 0).double().mean().item() - t) <= 6 * (t * (1 - t) / n) ** 0.5
    assert abs(y.double().mean().item() - 1) <= 6 * (t / (1 - t) / n) ** 0.5


def test_elements_past_32_bits():
    n = (1 << 32) + 24
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = dropout(x, 0.5, 9, y=x)
    tail = ref.dropout_words(24, 9, (1 << 32) // 8) >= 32768
    assert np.array_equal((y[-24:] != 0).cpu().numpy(), tail)
    head = ref.dropout_words(64, 9, 0) >= 32768
    assert np.array_equal((y[:64] != 0).cpu().numpy(), head)

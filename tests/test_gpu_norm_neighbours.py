"""Rows that share 16-byte accesses with the rows beside them, of which some hold no numbers, in every
form that shifted rows take: several teams a CTA (57, 511), two accesses of a thread (1031, 2047,
4089 and wider in bf16), four and eight (4099, 7167 in fp32). The buffers begin at 16-byte boundaries,
so that no call falls back to single elements; what follows them stays as it was."""
import pytest
import torch

from grouped_gemm_built_gb300 import mok
from grouped_gemm_built_gb300.norm import Norm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def buffers(count, T, H, dtype):
    """`count` row tensors [T, H], each at a 16-byte boundary with a guard of 7.0 behind it."""
    n = -(-T * H // 16) * 16 + 16
    flat = torch.full((count, n), 7.0, dtype=dtype, device="cuda")
    rows = [f[:T * H].view(T, H) for f in flat]
    assert all(t.data_ptr() % 16 == 0 for t in rows)
    return rows, flat[:, T * H:]


@pytest.mark.parametrize("x_t,y_t", [(BF, BF), (F32, F32), (F32, BF)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("T,H", [(310, 57), (700, 511), (310, 1031), (1300, 1031), (310, 2047), (310, 4089), (310, 4099),
                                 (310, 7167), (9, 8177)])
@pytest.mark.parametrize("bias", [True, False])
def test_a_row_without_numbers_leaves_its_neighbours_alone(x_t, y_t, kind, T, H, bias):
    g = torch.Generator().manual_seed(H)

    def draw(shape, dtype):
        return torch.randn(shape, generator=g).to(dtype).cuda()

    (x, a, da), _ = buffers(3, T, H, x_t)
    (dY,), _ = buffers(1, T, H, y_t)
    for t in (x, a, da, dY):
        t.copy_(draw((T, H), t.dtype))
    w, b = draw((H,), x_t), draw((H,), x_t) if bias else None
    bad = torch.arange(T, device="cuda") % 3 == 1
    good = ~bad
    n = Norm(w, b, kind=kind)
    y, h, stats = n.forward(x, add=a, out=y_t)
    want = n.backward(dY, h, stats, add=da)
    assert all(t.data_ptr() % 16 == 0 for t in (y, h, want["dX"]))
    code = {BF: mok.MOK_OUT_BF16, F32: mok.MOK_OUT_F32}
    dims = mok.MokNormDims(T=T, H=H, kind=Norm.KINDS[kind], eps=n.eps, x_type=code[x_t], y_type=code[y_t],
                           w_type=code[x_t])
    ws = torch.empty(mok.mok_norm_get_sizes(dims).workspace_bytes, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    bp = b.data_ptr() if bias else None
    for value in (float("nan"), float("inf")):
        (x2, h2, dX2), guard = buffers(3, T, H, x_t)
        (y2,), guard_y = buffers(1, T, H, y_t)
        x2.copy_(x)
        x2[bad] = value
        st, dW, dB = torch.empty_like(stats), torch.empty_like(w), torch.empty_like(w)
        mok.mok_norm_fwd(dims, x2.data_ptr(), a.data_ptr(), w.data_ptr(), bp, h2.data_ptr(), y2.data_ptr(),
                         st.data_ptr(), s)
        mok.mok_norm_bwd(dims, dY.data_ptr(), h2.data_ptr(), w.data_ptr(), st.data_ptr(), da.data_ptr(), dX2.data_ptr(),
                         dW.data_ptr(), dB.data_ptr() if bias else None, ws.data_ptr(), s)
        assert torch.equal(h2[good], h[good]) and torch.equal(y2[good], y[good])
        assert torch.equal(st[good], stats[good]) and torch.equal(dX2[good], want["dX"][good])
        if bias:
            assert torch.equal(dB, want["dB"])               # a sum of dY alone
        assert y2[bad].isnan().any(1).all() and dX2[bad].isnan().any(1).all() and dW.isnan().any()
        assert (guard == 7.0).all() and (guard_y == 7.0).all()

"""The backward pass of a linear layer in exactly the workspace that its outputs need."""
import pytest
import torch

from mixed_precision_vit_b200 import _lib as L
from mixed_precision_vit_b200 import sc
from test_gpu_layers import BF16, F16, F32, gen, rnd, strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,ot", [(BF16, BF16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_backward_workspace_is_enough(t, ot, pad, act):
    """Every set of wanted outputs through the C entry, the unread operands NULL with strides that
    mean nothing, in a workspace of the queried size whose end is watched.  The products keep
    their bits; dbias alone adds the same partial sums, 256 at most, in another order, so both are
    within 255 u sum|dz| of the exact sum of those."""
    g = gen(71)
    M, N, K = 300, 136, 88
    x, w = strided(rnd(g, M, K, dtype=t), pad)[0], strided(rnd(g, N, K, dtype=t), pad)[0]
    dout, pre = strided(rnd(g, M, N, dtype=ot), pad)[0], strided(rnd(g, M, N, dtype=t), pad)[0]
    full = sc.linear_backward(dout, x, w, pre, act, grad_dtype=F32)
    stream = torch.cuda.current_stream().cuda_stream
    for want in range(1, 8):
        dx, dw, db = (torch.full_like(f, 7) if want >> i & 1 else None for i, f in enumerate(full))
        xx, ww = x if dw is not None else None, w if dx is not None else None
        d = L.ScLinearDesc(M, N, K, 3 if xx is None else x.stride(0), 5 if ww is None else w.stride(0), dout.stride(0), 0,
                           pre.stride(0), K, K, sc._TYPES[t], sc._TYPES[ot], 0, L.SC_F32, sc.ACTIVATIONS[act])
        need = L.sc_linear_backward_workspace_bytes(d, dout, xx, ww)
        ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
        d.workspace, d.workspace_bytes = ws.data_ptr(), need
        L.check(L.lib().sc_linear_backward(d, *(L._ptr(p) for p in (dout, xx, ww, pre, dx, dw, db)), None, stream))
        assert (ws[need:] == 77).all()
        for got, ref in zip((dx, dw), full):
            assert got is None or torch.equal(got, ref)
        if db is not None:
            dz = dout.double() if act == "none" else dout.double() * (pre > 0)
            assert ((db.double() - full[2].double()).abs() <= 2 * 255 * 2.0 ** -24 * dz.abs().sum(0)).all()


def test_a_part_of_the_gradients_takes_less_memory():
    x, w = torch.randn(4096, 1024, device="cuda"), torch.randn(2048, 1024, device="cuda")
    dout = torch.randn(4096, 2048, device="cuda")

    def peak(**kw):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        sc.linear_backward(dout, x, w, **{**dict(want_dx=False, want_dw=False, want_db=False), **kw})
        return torch.cuda.max_memory_allocated() - before

    dz, xs, ws, small = 6 * dout.numel(), 6 * x.numel(), 6 * w.numel(), 1 << 22  # column sums, rounding up
    assert peak(want_db=True) < small
    assert peak(want_dx=True) < dz + ws + 4 * x.numel() + small
    assert peak(want_dw=True) < dz + xs + 4 * w.numel() + small


@pytest.mark.parametrize("t", [BF16, F32])
def test_a_single_row_has_any_stride(t):
    """A stride of 2^45 elements between rows that do not exist."""
    g = gen(72)
    N, K, far = 64, 128, 1 << 45
    x, dout, w = rnd(g, 1, K, dtype=t), rnd(g, 1, N, dtype=t), rnd(g, N, K, dtype=t)
    stream = torch.cuda.current_stream().cuda_stream
    out, dx, dw = torch.empty_like(dout), torch.empty_like(x), torch.empty_like(w)
    k = sc._TYPES[t]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    d = L.ScLinearDesc(1, N, K, far, K, far, 0, 0, far, K, k, k, 0, k, 0, ws.data_ptr(), ws.numel())
    L.check(L.lib().sc_linear(d, *(L._ptr(p) for p in (x, w, None, None, out, None)), None, stream))
    assert torch.equal(out, sc.linear(x, w)[0])
    L.check(L.lib().sc_linear_backward(d, *(L._ptr(p) for p in (dout, x, w, None, dx, dw, None)), None, stream))
    ref = sc.linear_backward(dout, x, w, want_db=False)
    assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])
    # w of one row, and its gradient's
    one, col = w[:1].contiguous(), torch.empty(1, 1, dtype=t, device="cuda")
    d = L.ScLinearDesc(1, 1, K, far, far, far, 0, 0, far, far, k, k, 0, k, 0, ws.data_ptr(), ws.numel())
    L.check(L.lib().sc_linear(d, *(L._ptr(p) for p in (x, one, None, None, col, None)), None, stream))
    assert torch.equal(col, sc.linear(x, one)[0])

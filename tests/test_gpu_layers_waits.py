"""What the linear layer does when one of its bounded waits gives up: the self-test's kernels wait
for copies that never bring what their barriers expect, return after about a millisecond, leave NaN
in their results and report it; the calls after them are right."""
import pytest
import torch

from mixed_precision_vit_b200 import _lib as L
from mixed_precision_vit_b200 import sc
from test_gpu_layers import BF16, F16, F32, gen, rnd, strided

pytestmark = pytest.mark.gpu
LIMIT = 1 << 21


def expired(x, w, out, pre, status):
    """The self-test on these operands, as sc.linear lays them out."""
    (M, K), N = x.shape, w.shape[0]
    d = L.ScLinearDesc(M, N, K, x.stride(0), w.stride(0), out.stride(0), 0, N, 0, 0, sc._TYPES[x.dtype],
                       sc._TYPES[out.dtype], 0, 0, L.SC_ACT_GELU)
    ws = sc._scratch(d, L.sc_linear_workspace_bytes(d, x, w), None, x)
    L.sc_selftest_linear_wait_limit(d, x, w, out, pre, LIMIT, status, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    del ws


# tiles of CTA pairs, of single CTAs, and contractions shared by a cluster
@pytest.mark.parametrize("M,N,K", [(257, 384, 1024), (3, 130, 4100), (1300, 1290, 90), (8448, 2048, 512),
                                   (8400, 2001, 512)])
@pytest.mark.parametrize("t,ot", [(BF16, BF16), (F16, F32), (F32, F32)])
def test_expired_waits_leave_nan_and_a_status(M, N, K, t, ot):
    g = gen(61)
    x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t, scale=K ** -0.5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    right, right_pre = sc.linear(x, w, act="gelu", out_dtype=ot, want_pre=True, dev_status=status)
    assert status.item() == 0 and right.isfinite().all()
    for pad in (0, 5):
        out, big = strided(torch.zeros(M, N, dtype=ot, device="cuda"), pad)
        big.fill_(7)
        pre = torch.zeros(M, N, dtype=t, device="cuda")
        status.zero_()
        expired(x, w, out, pre, status)
        assert status.item() == L.SC_DEV_WAIT_LIMIT
        assert out.isnan().all() and pre.isnan().all()
        assert (big[:, N:] == 7).all()
        status.zero_()
        again, again_pre = sc.linear(x, w, act="gelu", out_dtype=ot, want_pre=True, dev_status=status)
        assert status.item() == 0 and torch.equal(again, right) and torch.equal(again_pre, right_pre)


def test_ordinary_calls_report_nothing():
    g = gen(62)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for t in (BF16, F16, F32):
        for M, N, K in ((1, 10, 64), (700, 520, 333), (4112, 1024, 2048)):
            x, w = rnd(g, M, K, dtype=t), rnd(g, N, K, dtype=t)
            out, pre = sc.linear(x, w, act="silu", want_pre=True, dev_status=status)
            sc.linear_backward(out, x, w, pre, "silu", dev_status=status)
    assert status.item() == 0

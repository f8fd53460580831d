"""More host-side checks of the floating-point layers that need no GPU."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from mixed_precision_vit_b200 import _lib as L
from mixed_precision_vit_b200 import sc

P = 4096  # an aligned address that no accepted call here ever reaches


@pytest.fixture(scope="module")
def lib():
    from mixed_precision_vit_b200 import build
    build.build()
    return L.load()


def _linear(**kw):
    d = L.ScLinearDesc(4, 16, 64, 64, 64, 16, 16, 16, 64, 64, L.SC_BF16, L.SC_BF16, L.SC_F32,
                       L.SC_BF16, L.SC_ACT_NONE)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def test_wait_limit_selftest_refuses(lib):
    d = _linear()
    for bad in ((P, 0), (P, (1 << 34) + 1), (P, -1), (None, 1000)):
        status, limit = bad
        assert lib.sc_selftest_linear_wait_limit(ctypes.byref(d), P, P, P, P, limit, status, None) == L.SC_ERR_ARG
        assert L.sc_last_error().startswith("sc_selftest_linear_wait_limit:")
    d = _linear(ld_out=15)
    assert lib.sc_selftest_linear_wait_limit(ctypes.byref(d), P, P, P, P, 1000, P, None) == L.SC_ERR_ARG


@pytest.mark.parametrize("t", [L.SC_BF16, L.SC_F32])
def test_backward_workspace_counts_what_the_call_reads(lib, t):
    """dz, x and w take room (6 bytes an element here: three planes, or one copy of rows off their
    boundaries and their padding) only where a wanted output needs them."""
    M, N, K, size = 40, 24, 56, 6 if t == L.SC_F32 else 2
    kw = dict(M=M, N=N, K=K, type=t, out_type=t, ld_x=K + 1, ld_w=K + 1, ld_out=N + 1)
    q = lambda x, w: L.sc_linear_backward_workspace_bytes(_linear(**kw), P, x, w)
    up = lambda n: (n + 255) // 256 * 256
    sums, dz = q(None, None), up(M * N * size)
    assert 0 < sums <= up(256 * N * 4)
    assert q(None, P) == sums + dz + up(N * K * size)
    assert q(P, None) == sums + dz + up(M * K * size)
    assert q(P, P) == sums + dz + up(N * K * size) + up(M * K * size)


def test_backward_asks_for_no_more_than_the_outputs_need(lib):
    """Calls refused for a workspace of 64 bytes name the bytes that they need: nothing for operands
    that they do not read, whatever stands in those operands' strides."""
    dz, x, w = 256, 512, 2048  # 4 x 16, 4 x 64 and 16 x 64 bf16
    part = L.sc_linear_backward_workspace_bytes(_linear(), P, None, None)
    kw = dict(ld_out=17, workspace=P, workspace_bytes=64)
    for ops, outs, strides, need in (((None, P), (P, None, None), dict(ld_x=3), dz),
                                     ((P, None), (None, P, None), dict(ld_w=3), dz),
                                     ((P, P), (None, P, P), dict(ld_x=65, ld_w=3), dz + x + part),
                                     ((P, P), (P, None, None), dict(ld_x=3, ld_w=65), dz + w),
                                     ((None, None), (None, None, P), dict(ld_x=3, ld_w=5), part)):
        d = _linear(**{**kw, **strides})
        rc = lib.sc_linear_backward(ctypes.byref(d), P, *ops, None, *outs, None, None)
        assert rc == L.SC_ERR_ARG and f"{need} needed" in L.sc_last_error(), (L.sc_last_error(), need)


@pytest.mark.parametrize("M,N,K", [(2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 1, 2 ** 31 - 1),
                                   (1, 2 ** 31 - 1, 2 ** 26), (2 ** 30, 2 ** 27, 1)])
def test_sizes_that_no_byte_count_holds_are_refused(lib, M, N, K):
    """The workspace's bytes passed 2^63 there, and their sum could come out small."""
    for t in (L.SC_F32, L.SC_BF16):
        kw = dict(M=M, N=N, K=K, type=t, out_type=t, ld_x=K + 1, ld_w=K + 1, ld_out=N, ld_dx=K, ld_dw=K, workspace=P,
                  workspace_bytes=1 << 62)
        for query in (lambda: L.sc_linear_workspace_bytes(_linear(**kw), P, P),
                      lambda: L.sc_linear_backward_workspace_bytes(_linear(**kw), P, P, P)):
            with pytest.raises(L.ScError) as e:
                query()
            assert e.value.code == L.SC_ERR_ARG and "2^56" in str(e.value)
        assert lib.sc_linear(ctypes.byref(_linear(**kw)), P, P, P, P, P, P, None, None) == L.SC_ERR_ARG
        assert lib.sc_linear_backward(ctypes.byref(_linear(**kw)), P, P, P, P, P, P, P, None, None) == L.SC_ERR_ARG


def test_a_stream_of_another_device_is_refused():
    """It would become current, and its device with it, and the work would go elsewhere."""
    with pytest.raises(ValueError, match="cuda:1"):
        sc._On(torch.device("cuda", 0), SimpleNamespace(device=torch.device("cuda", 1)))

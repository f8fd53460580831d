"""Host-side checks of the floating-point layers that need no GPU: every
refusal happens before any CUDA call, and workspace queries are host only."""
import ctypes

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


def _norm(**kw):
    d = L.ScNormDesc(4, 64, 64, 64, 64, 64, 1e-6, L.SC_F32, L.SC_F32, L.SC_F32)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def _linear(**kw):
    d = L.ScLinearDesc(4, 16, 64, 64, 64, 16, 16, 16, 64, 64, L.SC_BF16, L.SC_BF16, L.SC_F32,
                       L.SC_BF16, L.SC_ACT_NONE)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


BAD_NORM = [dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=1 << 31), dict(x_type=3),
            dict(y_type=-1), dict(w_type=7), dict(ld_x=63), dict(ld_y=63)]


@pytest.mark.parametrize("bad", BAD_NORM + [dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))])
def test_layer_norm_refuses(lib, bad):
    d = _norm(**bad)
    assert lib.sc_layer_norm(ctypes.byref(d), P, P, P, P, P, P, None) == L.SC_ERR_ARG
    assert L.sc_last_error().startswith("sc_layer_norm:")


def test_layer_norm_refuses_null_and_mixed_types(lib):
    d = _norm()
    assert lib.sc_layer_norm(None, P, P, P, P, P, P, None) == L.SC_ERR_ARG
    assert lib.sc_layer_norm(ctypes.byref(d), None, P, P, P, P, P, None) == L.SC_ERR_ARG
    assert lib.sc_layer_norm(ctypes.byref(d), P, P, P, None, P, P, None) == L.SC_ERR_ARG
    d = _norm(x_type=L.SC_BF16, y_type=L.SC_F16)
    assert lib.sc_layer_norm(ctypes.byref(d), P, P, P, P, P, P, None) == L.SC_ERR_UNSUPPORTED
    assert lib.sc_layer_norm_backward(ctypes.byref(d), P, P, P, P, P, P, P, P, P, None) == L.SC_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", BAD_NORM + [dict(ld_dx=63), dict(ld_add=63), dict(workspace=None),
                                            dict(workspace_bytes=16), dict(workspace=P + 16)])
def test_layer_norm_backward_refuses(lib, bad):
    d = _norm(**{**dict(workspace=P, workspace_bytes=1 << 30), **bad})
    assert lib.sc_layer_norm_backward(ctypes.byref(d), P, P, P, P, P, P, P, P, P, None) == L.SC_ERR_ARG
    for null in (0, 1, 3, 4):  # dy, x, mean, rstd
        a = [P] * 9
        a[null] = None
        d = _norm(workspace=P, workspace_bytes=1 << 30)
        assert lib.sc_layer_norm_backward(ctypes.byref(d), *a, None) == L.SC_ERR_ARG


def test_empty_calls_launch_nothing(lib):
    d = _norm(rows=0)
    assert lib.sc_layer_norm(ctypes.byref(d), None, None, None, None, None, None, None) == L.SC_OK
    d = _norm()
    assert lib.sc_layer_norm_backward(ctypes.byref(d), P, P, P, P, P, None, None, None, None, None) == L.SC_OK
    for kw in (dict(M=0), dict(N=0, ld_out=0)):
        d = _linear(**kw)
        assert lib.sc_linear(ctypes.byref(d), None, None, None, None, None, None, None, None) == L.SC_OK
    d = _linear()
    assert lib.sc_linear_backward(ctypes.byref(d), P, P, P, P, None, None, None, None, None) == L.SC_OK


BAD_LINEAR = [dict(M=-1), dict(N=-1), dict(K=0), dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31),
              dict(type=3), dict(out_type=L.SC_F16), dict(type=L.SC_F32), dict(act=5), dict(act=-1),
              dict(workspace_bytes=-1), dict(workspace=P + 8), dict(ld_x=63), dict(ld_w=63), dict(ld_out=15)]


@pytest.mark.parametrize("bad", BAD_LINEAR + [dict(bias_type=9), dict(ld_res=15), dict(ld_pre=15)])
def test_linear_refuses(lib, bad):
    d = _linear(**{**dict(workspace=P, workspace_bytes=1 << 30), **bad})
    assert lib.sc_linear(ctypes.byref(d), P, P, P, P, P, P, None, None) == L.SC_ERR_ARG
    assert L.sc_last_error().startswith("sc_linear:")


def test_linear_refuses_null(lib):
    d = _linear(workspace=P, workspace_bytes=1 << 30)
    for null in (0, 1, 4):
        a = [P] * 7
        a[null] = None
        assert lib.sc_linear(ctypes.byref(d), *a, None) == L.SC_ERR_ARG
    assert lib.sc_linear(None, P, P, P, P, P, P, None, None) == L.SC_ERR_ARG


@pytest.mark.parametrize("bad", BAD_LINEAR + [dict(grad_type=4), dict(ld_dx=63), dict(ld_dw=63),
                                              dict(act=L.SC_ACT_GELU, ld_pre=15), dict(workspace=None),
                                              dict(workspace_bytes=64)])
def test_linear_backward_refuses(lib, bad):
    d = _linear(**{**dict(workspace=P, workspace_bytes=1 << 30), **bad})
    assert lib.sc_linear_backward(ctypes.byref(d), P, P, P, P, P, P, P, None, None) == L.SC_ERR_ARG
    d = _linear(workspace=P, workspace_bytes=1 << 30, act=L.SC_ACT_RELU)
    for null in (0, 1, 2, 3):  # dout, x, w, pre
        a = [P] * 7
        a[null] = None
        assert lib.sc_linear_backward(ctypes.byref(d), *a, None, None) == L.SC_ERR_ARG


def test_workspace_queries(lib):
    assert L.sc_layer_norm_workspace_bytes(_norm()) >= 2 * 4 * 64 * 4
    assert L.sc_linear_workspace_bytes(_linear(), P, P) == 0  # aligned 16-bit operands run in place
    assert L.sc_linear_backward_workspace_bytes(_linear(), P, P, P) > 0
    for q, d in ((L.sc_layer_norm_workspace_bytes, (_norm(cols=0),)),
                 (L.sc_linear_workspace_bytes, (_linear(K=0), P, P)),
                 (L.sc_linear_backward_workspace_bytes, (_linear(act=77), P, P, P))):
        with pytest.raises(L.ScError) as e:
            q(*d)
        assert e.value.code == L.SC_ERR_ARG


def test_python_entry_points_refuse_cpu_tensors():
    x, w = torch.zeros(3, 8), torch.zeros(5, 8)
    with pytest.raises(ValueError, match="CUDA"):
        sc.layer_norm(x)
    with pytest.raises(ValueError, match="CUDA"):
        sc.layer_norm_backward(x, x, x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        sc.linear(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        sc.linear_backward(torch.zeros(3, 5), x, w)

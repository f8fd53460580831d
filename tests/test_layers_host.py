"""More host-side checks of the floating-point layers that need no GPU."""
import ctypes

import pytest

from mixed_precision_vit_b200 import _lib as L

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

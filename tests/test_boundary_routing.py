"""Host-side refusals of the routing's row movers where a size is zero: a call
that reaches a kernel has every pointer the kernel reads (no GPU: each call
here is refused or has nothing to do)."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_scale_calibration_amd", "liblh.so")
OK, NULL, SHAPE, DTYPE, LAYOUT, WORKSPACE, ARG, HIP = range(8)
FAKE = 0x10000  # aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import nvfp4_scale_calibration_amd._build as b
        b.build()
    import nvfp4_scale_calibration_amd as m
    return m.lib


P = ctypes.c_void_p


def _grad(lib, dy=P(FAKE), n=4, c=8, ys=P(FAKE), rows=8, pos=P(FAKE), k=2, w=P(FAKE), dys=P(FAKE), dw=P(FAKE)):
    return lib.lh_moe_combine_grad(dy, 1, n, c, 8, ys, rows, 8, pos, k, w, dys, 8, dw, None)


def test_combine_grad_without_columns_needs_its_positions(lib):
    """The routing weights' gradient is written (zeros) for rows of no columns too, by position."""
    for dys in (None, P(FAKE)):
        assert _grad(lib, c=0, pos=None, dys=dys) == NULL
        assert "position" in lib.lh_last_error_message().decode()
        assert _grad(lib, c=0, pos=None, dys=dys, dy=None, ys=None) == NULL
    assert _grad(lib, pos=None) == NULL and _grad(lib, pos=None, dw=None) == NULL and _grad(lib, pos=None, dys=None) == NULL


def test_row_movers_with_nothing_to_do(lib):
    assert _grad(lib, c=0, pos=None, dy=None, ys=None, dw=None) == OK   # no columns, no weights' gradient
    assert _grad(lib, n=0, pos=None, dy=None, ys=None) == OK
    assert _grad(lib, k=0, pos=None, ys=None) == OK
    assert lib.lh_moe_dispatch(None, 1, 4, 0, 8, None, 2, None, 8, 8, None) == OK
    assert lib.lh_moe_combine(None, 1, 8, 0, 8, None, None, 4, 2, None, 8, None) == OK

"""Calls without tokens: their outputs have no elements, so their pointers may
be NULL (torch gives 0 for an empty tensor), and nothing is launched (no GPU
needed).  With tokens a call that asks for nothing is still refused."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_scale_calibration_amd", "liblh.so")
OK, NULL, SHAPE, DTYPE, LAYOUT, WORKSPACE, ARG, HIP = range(8)
P = ctypes.c_void_p
FAKE = P(0x10000)  # aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import nvfp4_scale_calibration_amd._build as b
        b.build()
    import nvfp4_scale_calibration_amd as m
    return m.lib


@pytest.mark.parametrize("g,rows,c_in", [(1, 0, 64), (3, 0, 64), (1, 5, 0), (0, 5, 64)])
def test_quantize_of_nothing(lib, g, rows, c_in):
    def call(dt=1, c=c_in, amax=FAKE, v=None, s=None):
        return lib.lh_quantize_nvfp4(None, dt, rows, c, c, g, 0, amax, v, 1, None, None, s, None)

    assert call() == OK and call(v=FAKE) == OK
    assert call(dt=5) == DTYPE and call(c=24) == SHAPE
    if g:
        assert call(amax=None) == NULL


def test_combine_grad_of_nothing(lib):
    def call(dt=1, n=4, c=8, k=2, rows=8, dys=None, dw=None, ld=8):
        return lib.lh_moe_combine_grad(FAKE, dt, n, c, ld, FAKE, rows, ld, FAKE, k, None, dys, ld, dw, None)

    assert call(n=0, rows=0) == OK and call(n=0, rows=6) == OK and call(k=0, rows=0) == OK and call(c=0) == OK
    assert call() == ARG and "no output" in lib.lh_last_error_message().decode()
    assert call(n=0, dt=5) == DTYPE and call(n=-1) == SHAPE and call(n=0, ld=7) == SHAPE

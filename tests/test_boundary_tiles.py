"""Products of more tiles than one launch takes (2^32 threads along a grid
dimension wrap around without an error) are refused on the host, in every
kernel's path.  No GPU: every call here is refused."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_scale_calibration_amd", "liblh.so")
SHAPE = 2
P = ctypes.c_void_p
FAKE = P(0x10000)  # aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import nvfp4_scale_calibration_amd._build as b
        b.build()
    import nvfp4_scale_calibration_amd as m
    return m.lib


@pytest.mark.parametrize("dt", [0, 1])                # fp32 without a workspace: the general kernel
@pytest.mark.parametrize("rows", [1, 2, 3, 20, 300])  # the dot-product kernel, and tiles
def test_dense_groups(lib, rows, dt):
    g, c_out, c_in = 1 << 24, 512, 512
    st = lib.lh_linear_nvfp4(FAKE, dt, rows, c_in, c_in, rows * c_in, FAKE, FAKE, FAKE, c_out, g, None, FAKE, 1, c_out,
                             rows * c_out, None, 0, None)
    assert st == SHAPE and "one launch" in lib.lh_last_error_message().decode()
    st = lib.lh_linear_nvfp4_grad(FAKE, dt, rows, c_out, c_out, rows * c_out, FAKE, FAKE, FAKE, c_in, g, FAKE, 1, c_in,
                                  rows * c_in, None, 0, None)
    assert st == SHAPE and "one launch" in lib.lh_last_error_message().decode()


@pytest.mark.parametrize("dt", [0, 1])
def test_ragged_rows(lib, dt):
    n, c_out, c_in = 1 << 24, 512, 512
    st = lib.lh_linear_nvfp4_ragged(FAKE, dt, n, c_in, c_in, FAKE, n, 0, FAKE, FAKE, FAKE, c_out, None, FAKE, 1, c_out, None,
                                    0, None)
    assert st == SHAPE and "one launch" in lib.lh_last_error_message().decode()
    st = lib.lh_linear_nvfp4_ragged_grad(FAKE, dt, n, c_out, c_out, FAKE, n, 0, FAKE, FAKE, FAKE, c_in, FAKE, 1, c_in, None,
                                         0, None)
    assert st == SHAPE and "one launch" in lib.lh_last_error_message().decode()

"""Sizes and strides up to the largest 64-bit numbers: the checks' own
arithmetic must not overflow (an overflow could let a call pass that overlaps
or reads outside its buffers).  No GPU: every call is refused."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_scale_calibration_amd", "liblh.so")
SHAPE = 2
P = ctypes.c_void_p
FAKE = P(0x10000)  # aligned non-null address; never dereferenced
BIG = (1 << 63) - 16   # a multiple of 16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import nvfp4_scale_calibration_amd._build as b
        b.build()
    import nvfp4_scale_calibration_amd as m
    return m.lib


@pytest.mark.parametrize("rows,c_in,c_out,g,ld_y,gs_y", [
    (BIG, 64, 64, 2, 64, 64 * 64), (4, 64, 64, 2, BIG, 1 << 20), (4, 64, 64, BIG, 64, 128), (1 << 32, 64, 64, 1 << 31, 64, BIG),
    (1 << 40, 64, 64, 1 << 40, 64, BIG), (4, BIG, 64, 1, 64, 0), (4, 64, BIG, 1, BIG, 0), (BIG, 64, 64, 1, 64, 0),
    (BIG, BIG, BIG, BIG, BIG, BIG)])
@pytest.mark.parametrize("dt", [0, 1])
def test_products(lib, rows, c_in, c_out, g, ld_y, gs_y, dt):
    st = lib.lh_linear_nvfp4(FAKE, dt, rows, c_in, c_in, 0, FAKE, FAKE, FAKE, c_out, g, None, FAKE, 1, max(ld_y, c_out), gs_y,
                             None, 0, None)
    assert st == SHAPE, lib.lh_last_error_message()
    st = lib.lh_linear_nvfp4_grad(FAKE, dt, rows, c_out, c_out, 0, FAKE, FAKE, FAKE, c_in, g, FAKE, 1, max(ld_y, c_in), gs_y,
                                  None, 0, None)
    assert st == SHAPE, lib.lh_last_error_message()
    if max(rows, g, c_in, c_out) > 4096:              # not the stride alone
        assert lib.lh_linear_nvfp4_workspace_bytes(0, 0, dt, rows, c_in, c_out, g, 0) == 0
        assert lib.lh_linear_nvfp4_workspace_bytes(1, 0, dt, rows, c_in, c_out, g, 0) == 0


def test_routing(lib):
    for n, k in ((BIG, 1), (1 << 32, 1 << 32), (1, BIG), (3, BIG // 2)):
        assert lib.lh_moe_sort(FAKE, 1, n, k, 4, FAKE, FAKE, None, None, 0, None) == SHAPE
        assert lib.lh_moe_sort_workspace_bytes(n, k, 4) == 0
        assert lib.lh_moe_dispatch(FAKE, 1, n, 8, 8, FAKE, k, FAKE, BIG, 8, None) == SHAPE
        assert lib.lh_moe_combine(FAKE, 1, BIG, 8, 8, FAKE, None, n, k, FAKE, 8, None) == SHAPE
        assert lib.lh_moe_combine_grad(FAKE, 1, n, 8, 8, FAKE, BIG, 8, FAKE, k, None, FAKE, 8, FAKE, None) == SHAPE
    assert lib.lh_moe_dispatch(FAKE, 1, 4, BIG, BIG, FAKE, 2, FAKE, 8, BIG, None) == SHAPE
    assert lib.lh_moe_combine(FAKE, 1, 8, BIG, BIG, FAKE, None, 4, 2, FAKE, BIG, None) == SHAPE
    assert lib.lh_moe_combine_grad(FAKE, 1, 4, BIG, BIG, FAKE, 8, BIG, FAKE, 2, None, FAKE, BIG, None, None) == SHAPE


def test_quantize(lib):
    def call(rows, c, ld, g, gs):
        return lib.lh_quantize_nvfp4(FAKE, 1, rows, c, ld, g, gs, FAKE, FAKE, 1, None, None, None, None)

    for a in ((BIG, 64, 64, 1, 0), (4, BIG, BIG, 1, 0), (4, 64, 64, BIG, 0), (1 << 40, 64, 64, 1 << 40, 0)):
        assert call(*a) == SHAPE, lib.lh_last_error_message()

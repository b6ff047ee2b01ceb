"""Host-side refusals of the product, quantisation and routing entry points
(no GPU: every call here fails validation or is an empty problem, so none
reaches a launch), and the workspace queries, which are host logic."""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_scale_calibration_amd", "liblh.so")
OK, NULL, SHAPE, DTYPE, LAYOUT, WORKSPACE, ARG, HIP = range(8)
FAKE = 0x10000  # aligned non-null address; never dereferenced (validation fails first)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import nvfp4_scale_calibration_amd._build as b
        b.build()
    import nvfp4_scale_calibration_amd as m
    return m.lib


def _msg(lib):
    return lib.lh_last_error_message().decode()


def test_quantize(lib):
    P = ctypes.c_void_p
    ok = dict(x=P(FAKE), dt=1, rows=4, c=32, ld=32, g=1, gs=0, amax=P(FAKE), v=P(FAKE), vdt=1, pk=None, sc=None,
              s=None, st=None)

    def call(**kw):
        a = dict(ok, **kw)
        return lib.lh_quantize_nvfp4(a["x"], a["dt"], a["rows"], a["c"], a["ld"], a["g"], a["gs"], a["amax"], a["v"],
                                     a["vdt"], a["pk"], a["sc"], a["s"], a["st"])

    assert call(dt=5) == DTYPE and call(vdt=5) == DTYPE
    assert call(c=24) == SHAPE and "multiple of 16" in _msg(lib)
    assert call(ld=16) == SHAPE and call(rows=-1) == SHAPE and call(gs=-1) == SHAPE
    assert call(x=None) == NULL and call(amax=None) == NULL
    assert call(v=None) == ARG and "no output" in _msg(lib)
    assert call(v=P(FAKE + 8)) == ARG and call(pk=P(FAKE + 4)) == ARG and call(x=P(FAKE + 1)) == ARG
    assert call(g=0) == OK


def _linear(lib, grad, ragged, **kw):
    P = ctypes.c_void_p
    a = dict(x=P(FAKE), dt=1, rows=8, c_in=64, c_out=48, ld_x=None, gs_x=0, off=P(FAKE), g=1, most=0, pk=P(FAKE),
             sc=P(FAKE), gsc=P(FAKE), xs=None, y=P(FAKE), ydt=1, ld_y=None, gs_y=0, ws=None, wsb=0, st=None)
    a.update(kw)
    k, m = (a["c_out"], a["c_in"]) if grad else (a["c_in"], a["c_out"])
    ld_x, ld_y = k if a["ld_x"] is None else a["ld_x"], m if a["ld_y"] is None else a["ld_y"]
    end = (a["ws"], a["wsb"], a["st"])
    xs = () if grad else (a["xs"],)
    if ragged:
        f = lib.lh_linear_nvfp4_ragged_grad if grad else lib.lh_linear_nvfp4_ragged
        return f(a["x"], a["dt"], a["rows"], k, ld_x, a["off"], a["g"], a["most"], a["pk"], a["sc"], a["gsc"], m, *xs,
                 a["y"], a["ydt"], ld_y, *end)
    f = lib.lh_linear_nvfp4_grad if grad else lib.lh_linear_nvfp4
    return f(a["x"], a["dt"], a["rows"], k, ld_x, a["gs_x"], a["pk"], a["sc"], a["gsc"], m, a["g"], *xs, a["y"],
             a["ydt"], ld_y, a["gs_y"], *end)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("ragged", [False, True])
def test_products(lib, grad, ragged):
    P = ctypes.c_void_p

    def call(**kw):
        return _linear(lib, grad, ragged, **kw)

    assert call(dt=3) == DTYPE and call(ydt=3) == DTYPE
    assert call(c_in=40) == SHAPE and "multiple of 16" in _msg(lib)
    assert call(ld_x=15) == SHAPE and call(ld_y=15) == SHAPE
    assert call(rows=-1) == SHAPE and call(g=-1) == SHAPE and call(c_out=-1) == SHAPE
    assert call(x=None) == NULL and call(y=None) == NULL and call(pk=None) == NULL and call(sc=None) == NULL
    assert call(gsc=None) == NULL
    if ragged:
        assert call(off=None) == NULL and call(most=-1) == SHAPE and call(off=P(FAKE + 4)) == ARG
    else:
        assert call(g=2, gs_y=7) == SHAPE and "overlap" in _msg(lib)
        assert call(gs_x=-1) == SHAPE
    assert call(x=P(FAKE + 1)) == ARG and call(pk=P(FAKE + 4)) == ARG and call(y=P(FAKE + 1)) == ARG
    assert call(ws=None, wsb=64) == NULL
    assert call(ws=P(FAKE + 16), wsb=1 << 30) == ARG
    # empty problems are valid and launch nothing
    assert call(rows=0, x=None, y=None) == OK
    assert call(g=0) == OK
    if grad:
        assert call(c_in=0, pk=None, sc=None, y=None) == OK
    else:
        assert call(c_out=0, pk=None, sc=None, y=None) == OK


def test_product_workspace(lib):
    q = lib.lh_linear_nvfp4_workspace_bytes
    assert q(0, 0, 1, 0, 64, 64, 1, 0) == 0 and q(0, 0, 1, 8, 63, 64, 1, 0) == 0 and q(0, 0, 7, 8, 64, 64, 1, 0) == 0
    assert q(0, 0, 1, 1, 4096, 4096, 1, 0) == 0                       # one token: straight from the packed rows
    assert q(0, 0, 1, 8192, 4096, 12288, 1, 0) == 0                   # whole tiles of bf16 rows: nothing to stage
    assert q(0, 0, 0, 8192, 4096, 12288, 1, 0) == 8192 * 3 * 4096 * 2  # fp32: three bf16 planes
    assert q(0, 0, 1, 8192, 4112, 12288, 1, 0) == 8192 * 4224 * 2     # rows padded to whole chunks
    assert q(1, 0, 1, 8192, 12288, 4100, 1, 0) == 8192 * 4160 * 2     # the gradient pads c_out
    few = q(0, 0, 1, 128, 4096, 4096, 1, 0)                           # few tiles: partial sums of 2..16 parts
    assert few % (128 * 4096 * 4) == 0 and 2 <= few // (128 * 4096 * 4) <= 16
    assert q(0, 1, 1, 128, 4096, 4096, 4, 0) == 0                     # ragged rows are never split
    need = few
    assert _linear(lib, False, False, rows=128, c_in=4096, c_out=4096, ws=ctypes.c_void_p(FAKE),
                   wsb=need - 1) == WORKSPACE


def test_routing(lib):
    P = ctypes.c_void_p
    ws = lib.lh_moe_sort_workspace_bytes
    assert ws(16, 8, 64) == 0 and ws(0, 8, 64) == 0 and ws(16, 8, 2000) == 0
    assert ws(4096, 8, 64) == 16 * 65 * 4
    ok = dict(ids=P(FAKE), t=1, n=4096, k=8, g=64, off=P(FAKE), pos=P(FAKE), order=None, ws=P(FAKE), wsb=16 * 65 * 4,
              st=None)

    def sort(**kw):
        a = dict(ok, **kw)
        return lib.lh_moe_sort(a["ids"], a["t"], a["n"], a["k"], a["g"], a["off"], a["pos"], a["order"], a["ws"],
                               a["wsb"], a["st"])

    assert sort(t=2) == DTYPE
    assert sort(n=-1) == SHAPE and sort(g=1025) == SHAPE and sort(n=1 << 30) == SHAPE
    assert sort(ids=None) == NULL and sort(off=None) == NULL and sort(pos=None) == NULL
    assert sort(ws=None, wsb=4) == NULL
    assert sort(wsb=16 * 65 * 4 - 4) == WORKSPACE and sort(ws=None, wsb=0) == WORKSPACE
    assert sort(ids=P(FAKE + 4)) == ARG and sort(off=P(FAKE + 4)) == ARG and sort(pos=P(FAKE + 2)) == ARG

    def dispatch(x=P(FAKE), dt=1, n=4, c=8, ld=8, pos=P(FAKE), k=2, xs=P(FAKE), rows=8, ldo=8):
        return lib.lh_moe_dispatch(x, dt, n, c, ld, pos, k, xs, rows, ldo, None)

    assert dispatch(dt=9) == DTYPE and dispatch(n=-1) == SHAPE and dispatch(rows=7) == SHAPE
    assert dispatch(ld=7) == SHAPE and dispatch(ldo=7) == SHAPE and dispatch(n=1 << 30, rows=1 << 40) == SHAPE
    assert dispatch(x=None) == NULL and dispatch(pos=None) == NULL and dispatch(xs=None) == NULL
    assert dispatch(x=P(FAKE + 1)) == ARG and dispatch(pos=P(FAKE + 2)) == ARG
    assert dispatch(n=0, x=None, pos=None, xs=None, rows=0) == OK and dispatch(c=0) == OK

    def combine(ys=P(FAKE), dt=1, rows=8, c=8, ld=8, pos=P(FAKE), w=P(FAKE), n=4, k=2, y=P(FAKE), ldy=8):
        return lib.lh_moe_combine(ys, dt, rows, c, ld, pos, w, n, k, y, ldy, None)

    assert combine(dt=9) == DTYPE and combine(rows=7) == SHAPE and combine(ldy=7) == SHAPE
    assert combine(ys=None) == NULL and combine(y=None) == NULL and combine(w=P(FAKE + 2)) == ARG
    assert combine(n=0, ys=None, pos=None, y=None, rows=0) == OK

    def grad(dy=P(FAKE), dt=1, n=4, c=8, ld=8, ys=P(FAKE), rows=8, ldy=8, pos=P(FAKE), k=2, w=P(FAKE), dys=P(FAKE),
             ldd=8, dw=P(FAKE)):
        return lib.lh_moe_combine_grad(dy, dt, n, c, ld, ys, rows, ldy, pos, k, w, dys, ldd, dw, None)

    assert grad(dys=None, dw=None) == ARG and grad(dt=9) == DTYPE
    assert grad(ys=None) == NULL and grad(dy=None) == NULL and grad(dy=None, dw=None) == NULL
    assert grad(ldd=7) == SHAPE and grad(ldy=7) == SHAPE and grad(rows=7) == SHAPE
    assert grad(dw=P(FAKE + 2)) == ARG
    assert grad(n=0, dy=None, ys=None, pos=None, dys=None, rows=0) == OK

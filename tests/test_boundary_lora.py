"""Host-side refusals of the adapters' and checkpoints' entry points (no GPU:
every call here fails validation or is an empty problem, so none reaches a
launch), sizes up to the largest 64-bit numbers, and the binding's checks."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_scale_calibration_amd", "liblh.so")
OK, NULL, SHAPE, DTYPE, LAYOUT, WORKSPACE, ARG, HIP = range(8)
P = ctypes.c_void_p
FAKE = 0x10000  # aligned non-null address; never dereferenced (validation fails first)
BIG = (1 << 63) - 16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(LIB):
        import nvfp4_scale_calibration_amd._build as b
        b.build()
    import nvfp4_scale_calibration_amd as m
    return m.lib


def _msg(lib):
    return lib.lh_last_error_message().decode()


def _lora(lib, grad, **kw):
    a = dict(x=P(FAKE), xdt=1, rows=8, c_in=64, c_out=48, ld_x=None, off=P(FAKE), ids=P(FAKE), it=0, n=3, a=P(FAKE),
             b=P(FAKE), wdt=1, ad=4, rank=8, scale=P(FAKE), base=P(FAKE), ld_b=None, y=P(FAKE), ydt=1, ld_y=None, s=None,
             ws=P(FAKE), wsb=1 << 20, st=None)
    a.update(kw)
    k, m = (a["c_out"], a["c_in"]) if grad else (a["c_in"], a["c_out"])
    for key, v in (("ld_x", k), ("ld_b", m), ("ld_y", m)):
        a[key] = v if a[key] is None else a[key]
    f = lib.lh_lora_grad if grad else lib.lh_lora
    return f(a["x"], a["xdt"], a["rows"], k, a["ld_x"], a["off"], a["ids"], a["it"], a["n"], a["a"], a["b"], a["wdt"],
             a["ad"], a["rank"], a["scale"], a["base"], a["ld_b"], m, a["y"], a["ydt"], a["ld_y"], a["s"], a["ws"],
             a["wsb"], a["st"])


@pytest.mark.parametrize("grad", [False, True])
def test_lora(lib, grad):
    def call(**kw):
        return _lora(lib, grad, **kw)

    assert call(xdt=2) == DTYPE and call(wdt=2) == DTYPE and call(ydt=2) == DTYPE and call(it=2) == DTYPE
    assert call(rows=-1) == SHAPE and call(c_in=-1) == SHAPE and call(c_out=-1) == SHAPE and call(n=-1) == SHAPE
    assert call(ad=-1) == SHAPE and call(rank=-1) == SHAPE and call(rank=257) == SHAPE and "256" in _msg(lib)
    assert call(ld_x=40) == SHAPE and call(ld_y=40) == SHAPE and call(ld_b=40) == SHAPE
    assert call(off=None) == SHAPE and "n_rows or 1" in _msg(lib)
    assert call(ids=None, ad=2) == SHAPE and "every segment" in _msg(lib)
    assert call(base=P(FAKE), y=P(FAKE), ld_b=80) == SHAPE
    assert call(x=None) == NULL and call(a=None) == NULL and call(b=None) == NULL and call(y=None) == NULL
    assert call(ws=None, wsb=8) == NULL
    assert call(x=P(FAKE + 1)) == ARG and call(a=P(FAKE + 1)) == ARG and call(b=P(FAKE + 1)) == ARG
    assert call(y=P(FAKE + 1)) == ARG and call(base=P(FAKE + 1)) == ARG and call(scale=P(FAKE + 2)) == ARG
    assert call(s=P(FAKE + 2)) == ARG and call(ws=P(FAKE + 128)) == ARG and call(off=P(FAKE + 4)) == ARG
    assert call(ids=P(FAKE + 2)) == ARG and call(ids=P(FAKE + 4), it=1) == ARG
    need = lib.lh_lora_workspace_bytes(int(grad), 8, 3, 64, 48, 8)
    assert need > 0
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None, wsb=0) == WORKSPACE
    # empty problems are valid and launch nothing
    assert call(rows=0, x=None, y=None, base=None) == OK and call(n=0) == OK
    assert call(rows=0, off=None, n=0) == OK
    assert (call(c_in=0, y=None, a=None) if grad else call(c_out=0, y=None, b=None)) == OK


def test_lora_workspace(lib):
    q = lib.lh_lora_workspace_bytes
    assert q(0, 0, 1, 64, 64, 8) == 0 and q(0, 8, 0, 64, 64, 8) == 0 and q(0, 8, 1, 64, 64, 0) == 0
    assert q(0, 8, 1, 64, 64, 257) == 0 and q(0, 8, 1, -1, 64, 8) == 0
    assert q(0, 333, 5, 4096, 1024, 8) == q(1, 333, 5, 1024, 4096, 8) >= 333 * 8 * 4
    w = lib.lh_lora_weight_grad_workspace_bytes
    assert w(0, 1, 1, 8, 64, 64) == 0 and w(8, 1, 1025, 8, 64, 64) == 0 and w(8, 1, 1, 300, 64, 64) == 0


def _weight(lib, **kw):
    a = dict(x=P(FAKE), xdt=1, xs=None, c_in=64, ld_x=None, dy=P(FAKE), ydt=1, c_out=48, ld_y=None, s=P(FAKE),
             ds=P(FAKE), rows=8, off=P(FAKE), ids=P(FAKE), it=0, n=3, ad=4, rank=8, scale=P(FAKE), beta=0.0, da=P(FAKE),
             db=P(FAKE), odt=0, ws=P(FAKE), wsb=1 << 30, st=None)
    a.update(kw)
    a["ld_x"] = a["c_in"] if a["ld_x"] is None else a["ld_x"]
    a["ld_y"] = a["c_out"] if a["ld_y"] is None else a["ld_y"]
    return lib.lh_lora_weight_grad(a["x"], a["xdt"], a["xs"], a["c_in"], a["ld_x"], a["dy"], a["ydt"], a["c_out"],
                                   a["ld_y"], a["s"], a["ds"], a["rows"], a["off"], a["ids"], a["it"], a["n"], a["ad"],
                                   a["rank"], a["scale"], a["beta"], a["da"], a["db"], a["odt"], a["ws"], a["wsb"],
                                   a["st"])


def test_weight_grad(lib):
    def call(**kw):
        return _weight(lib, **kw)

    assert call(xdt=3) == DTYPE and call(ydt=2) == DTYPE and call(odt=2) == DTYPE and call(it=5) == DTYPE
    assert call(rows=-1) == SHAPE and call(c_in=-1) == SHAPE and call(c_out=-1) == SHAPE and call(n=-1) == SHAPE
    assert call(ad=-1) == SHAPE and call(ad=1025) == SHAPE and "1024" in _msg(lib) and call(rank=257) == SHAPE
    assert call(ld_x=63) == SHAPE and call(ld_y=47) == SHAPE and call(off=None) == SHAPE and call(ids=None, n=5) == SHAPE
    assert call(xdt=2, xs=P(FAKE), ld_x=80) == SHAPE and "dense" in _msg(lib)
    assert call(da=None, db=None) == ARG and "no output" in _msg(lib)
    assert call(x=None) == NULL and call(ds=None) == NULL and call(dy=None) == NULL and call(s=None) == NULL
    assert call(xdt=2) == NULL and call(ws=None, wsb=4) == NULL
    assert call(x=P(FAKE + 1)) == ARG and call(dy=P(FAKE + 1)) == ARG and call(s=P(FAKE + 2)) == ARG
    assert call(ds=P(FAKE + 2)) == ARG and call(da=P(FAKE + 2)) == ARG and call(db=P(FAKE + 2)) == ARG
    assert call(scale=P(FAKE + 1)) == ARG and call(ws=P(FAKE + 16)) == ARG
    assert call(ad=0, n=0) == OK and call(rank=0) == OK and call(c_in=0, c_out=0) == OK
    need = lib.lh_lora_weight_grad_workspace_bytes(8, 3, 4, 8, 64, 48)
    if need:
        assert call(wsb=need - 1) == WORKSPACE and call(ws=None, wsb=0) == WORKSPACE


def test_checkpoint(lib):
    def pack(x=P(FAKE), dt=1, rows=4, cols=40, ld=40, v=P(FAKE), s=P(FAKE)):
        got = (lib.lh_checkpoint_pack(x, dt, rows, cols, ld, v, s, None),
               lib.lh_checkpoint_unpack(v, s, rows, cols, x, dt, ld, None))
        assert got[0] == got[1]
        return got[0]

    assert pack(dt=2) == DTYPE and pack(rows=-1) == SHAPE and pack(cols=-1) == SHAPE and pack(ld=39) == SHAPE
    assert pack(x=None) == NULL and pack(v=None) == NULL and pack(s=None) == NULL and pack(x=P(FAKE + 1)) == ARG
    assert pack(rows=0, x=None, v=None, s=None) == OK and pack(cols=0, ld=0, x=None, v=None, s=None) == OK


def test_extreme_sizes(lib):
    for grad in (False, True):
        for kw in (dict(rows=BIG), dict(c_in=BIG), dict(c_out=BIG), dict(ad=BIG), dict(rows=1 << 40, ld_y=1 << 40),
                   dict(rows=1 << 40, ld_x=1 << 40), dict(rows=1 << 40, ld_b=1 << 40), dict(n=BIG), dict(rank=BIG),
                   dict(rows=BIG, c_in=BIG, c_out=BIG, ad=BIG, n=BIG)):
            assert _lora(lib, grad, **kw) == SHAPE, (kw, _msg(lib))
    for kw in (dict(rows=BIG), dict(c_in=BIG), dict(c_out=BIG), dict(ad=BIG), dict(n=BIG), dict(rank=BIG),
               dict(rows=1 << 40, ld_y=1 << 40), dict(rows=1 << 40, ld_x=1 << 40)):
        assert _weight(lib, **kw) == SHAPE, (kw, _msg(lib))
    for rows, cols, ld in ((BIG, 64, 64), (4, BIG, BIG), (1 << 40, 64, 1 << 40)):
        assert lib.lh_checkpoint_pack(P(FAKE), 1, rows, cols, ld, P(FAKE), P(FAKE), None) == SHAPE
        assert lib.lh_checkpoint_unpack(P(FAKE), P(FAKE), rows, cols, P(FAKE), 1, ld, None) == SHAPE
    for sizes in ((BIG, 1, 64, 64, 8), (8, 1, BIG, 64, 8), (8, 1, 64, BIG, 8), (1 << 40, 1, 1 << 40, 8, 8)):
        assert lib.lh_lora_workspace_bytes(0, *sizes) == 0
        assert lib.lh_lora_weight_grad_workspace_bytes(sizes[0], sizes[1], 1, sizes[4], *sizes[2:4]) == 0


def test_binding_refuses_host_tensors(lib):
    import nvfp4_scale_calibration_amd as m
    x, a, b = torch.zeros(4, 8), torch.zeros(2, 4, 8), torch.zeros(2, 4, 6)
    for call in (lambda: m.lh_lora(x, a, b), lambda: m.lh_lora_grad(torch.zeros(4, 6), a, b),
                 lambda: m.lh_lora_weight_grad(x, torch.zeros(4, 6), torch.zeros(4, 4), torch.zeros(4, 4), 2),
                 lambda: m.lh_checkpoint_pack(x),
                 lambda: m.lh_checkpoint_unpack(torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="device tensors"):
            call()


def test_calls_run_with_their_tensors_device_current(lib, monkeypatch):
    """On another device than the current one the call is made with the tensors' as current."""
    import nvfp4_scale_calibration_amd as m

    class On:
        def get_device(self):
            return 3

    state = dict(current=0)

    class Guard:
        def __init__(self, d):
            self.d = d

        def __enter__(self):
            self.old, state["current"] = state["current"], self.d

        def __exit__(self, *_):
            state["current"] = self.old

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", Guard)
    monkeypatch.setattr(m, "_stream", lambda t: 17)
    seen = []

    def call(*args):
        seen.append((state["current"], args))
        return 0

    m._launch(On(), call, 1, 2)
    state["current"] = 3
    m._launch(On(), call, 4)
    assert seen == [(3, (1, 2, 17)), (3, (4, 17))]

"""Low-rank adapters, their gradients to the input and to the adapters, against
the formulas in 64 bits.

Tolerances, from the arithmetic alone.  A sum of n exact or once-rounded fp32
products added in fp32 is off by at most lambda sqrt(n) 2^-24 sum |terms| (the
probabilistic bound with lambda = 8, failing with probability 2 exp(-32)), plus
2^-24 of each product's own rounding.  s carries its sum's error into y through
|out|; where bf16 factors meet s for a bf16 y, s is cut to 16 bits, 2^-16 of it.
Then one product with the scale, one sum with base (2^-24 each) and the rounding
to the output's type (2^-8 for bf16, 2^-24 for fp32)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def rand(rng, shape, dtype, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def rows_of(offsets, ids, n_rows, n_adapters):
    """Each row's adapter: -1 none, -2 in no segment."""
    g = np.full(n_rows, -2)
    for i in range(len(offsets) - 1):
        lo, hi = max(int(offsets[i]), 0), min(int(offsets[i + 1]), n_rows)
        k = int(ids[i])
        g[lo:max(lo, hi)] = k if 0 <= k < n_adapters else -1
    return g


def spread(n):
    return (8 * np.sqrt(max(n, 1)) + 3) * U


def expected(x, inner, outer, scale, base, g, ydt, planes_cut):
    """(s, tolerance of s, y, tolerance of y) in 64 bits; rows of no segment NaN."""
    x, inner, outer = f64(x), f64(inner), f64(outer)
    rows, rank = x.shape[0], inner.shape[1]
    s, st = np.zeros((rows, rank)), np.zeros((rows, rank))
    y, yt = np.zeros((rows, outer.shape[2])), np.zeros((rows, outer.shape[2]))
    if base is not None:
        y += f64(base)
    for t in range(rows):
        if g[t] < 0:
            continue
        a, b, c = inner[g[t]], outer[g[t]], scale[g[t]]
        s[t] = a @ x[t]
        st[t] = spread(x.shape[1]) * (np.abs(a) @ np.abs(x[t]))
        part = np.abs(s[t]) @ np.abs(b)
        yt[t] = abs(c) * ((st[t] + (2.0 ** -16 if planes_cut else 0) * (np.abs(s[t]) + st[t])) @ np.abs(b) + spread(rank) * part)
        y[t] += c * (s[t] @ b)
        yt[t] += 3 * U * (np.abs(y[t]) + abs(c) * part)
    u = 2.0 ** -8 if ydt == BF16 else U
    return s, st + 1e-37, y, yt + u * (np.abs(y) + yt) + 1e-37


def near(got, want, tol, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its tolerance" % (
        what, bad.sum(), bad.size, np.max(np.abs(got - want) / tol))


def segments(rng, rows, n, adapters, bare=0.2):
    """Skewed segments, empty ones among them, with adapters in any order; rows before the first and behind the last."""
    cut = np.sort(rng.integers(0, rows + 1, n + 1)).astype(np.int64)
    if rng.random() < 0.5:
        cut[0], cut[-1] = 0, rows
    ids = rng.integers(0, adapters, n)
    ids[rng.random(n) < bare] = rng.choice([-1, adapters, -(1 << 31)])
    return cut, ids.astype(np.int32)


def check(lh, rng, rows, c_in, c_out, rank, adapters, offsets, ids, xdt, wdt, ydt, base=True, give_offsets=True, scaled=True):
    print("case rows=%d %d->%d rank=%d adapters=%d segments=%d %s %s %s base=%s" % (
        rows, c_in, c_out, rank, adapters, len(ids), xdt, wdt, ydt, base), flush=True)
    a, b = rand(rng, (adapters, rank, c_in), wdt, c_in ** -0.5), rand(rng, (adapters, rank, c_out), wdt, 0.3)
    scale = torch.from_numpy(rng.uniform(0.25, 2, adapters).astype(np.float32)) if scaled else None
    sc = f64(scale) if scaled else np.ones(adapters)
    g = rows_of(offsets, ids, rows, adapters)
    dev = dict(scale=scale.to(DEV) if scaled else None, offsets=torch.from_numpy(offsets).to(DEV) if give_offsets else None,
               adapter_ids=torch.from_numpy(ids).to(DEV))
    for grad in (False, True):
        k, m = (c_out, c_in) if grad else (c_in, c_out)
        x = rand(rng, (rows, k), xdt)
        bs = rand(rng, (rows, m), ydt) if base else None
        s, st, y, yt = expected(x, b if grad else a, a if grad else b, sc, bs, g, ydt, wdt == BF16 and ydt == BF16)
        out = torch.full((rows, m), 77.0, dtype=ydt, device=DEV)
        keep = torch.full((rows, rank), 55.0, device=DEV)
        f = lh.lh_lora_grad if grad else lh.lh_lora
        kw = dict(dev, base=None if bs is None else bs.to(DEV))
        kw["dx" if grad else "y"], kw["ds" if grad else "s"] = out, keep
        got, got_s = f(x.to(DEV), a.to(DEV), b.to(DEV), **kw)
        assert got is out and got_s is keep
        live = g > -2
        near(got_s[live], s[live], st[live], "s")
        near(got[live], y[live], yt[live], "y")
        assert (got[~live] == 77.0).all() and (got_s[~live] == 55.0).all(), "rows of no segment were written"
        if base:                                     # in place, without s: the same bits
            own = bs.to(DEV)
            kw2 = dict(dev, base=own)
            kw2["dx" if grad else "y"] = own
            f(x.to(DEV), a.to(DEV), b.to(DEV), **kw2)
            assert torch.equal(own[live], got[live]) and torch.equal(own[~live], bs.to(DEV)[~live])


TYPES = [(BF16, BF16, BF16), (F32, F32, F32), (BF16, BF16, F32), (BF16, F32, BF16), (F32, BF16, F32), (F32, BF16, BF16)]
SIZES = [(1, 16, 16, 1), (1, 4096, 512, 16), (2, 17, 33, 3), (3, 128, 1, 5), (5, 1, 128, 16), (16, 64, 64, 16),
         (17, 272, 100, 8), (33, 520, 264, 32), (64, 256, 512, 64), (65, 1040, 130, 33), (100, 96, 1111, 17),
         (130, 513, 144, 100), (257, 200, 1000, 128), (300, 768, 256, 250), (40, 64, 96, 256)]


@pytest.mark.parametrize("rows,c_in,c_out,rank", SIZES)
@pytest.mark.parametrize("types", TYPES)
def test_segments(lh, rows, c_in, c_out, rank, types):
    rng = np.random.default_rng([rows, c_in, c_out, rank])
    n = int(rng.integers(1, 7))
    offsets, ids = segments(rng, rows, n, 3)
    check(lh, rng, rows, c_in, c_out, rank, 3, offsets, ids, *types, base=bool(rng.integers(0, 2)))


@pytest.mark.parametrize("rows,c_in,c_out,rank", [(1, 4096, 520, 16), (7, 100, 300, 5), (48, 512, 256, 16), (70, 144, 1100, 64),
                                                  (200, 64, 64, 8)])
@pytest.mark.parametrize("types", TYPES)
def test_a_row_each(lh, rows, c_in, c_out, rank, types):
    rng = np.random.default_rng([1, rows, c_in, c_out, rank])
    ids = rng.integers(-1, 6, rows).astype(np.int64)
    check(lh, rng, rows, c_in, c_out, rank, 5, np.arange(rows + 1), ids, *types, give_offsets=False, scaled=False)


@pytest.mark.parametrize("segs", [64, 200, 1500])
def test_many_segments(lh, segs):
    """More segments than a wave has lanes, most of them empty or of a row or two."""
    rng = np.random.default_rng(segs)
    offsets, ids = segments(rng, 600, segs, 9)
    check(lh, rng, 600, 72, 80, 12, 9, offsets, ids, BF16, BF16, BF16)
    offsets[:] = np.minimum(offsets, 40)             # all but a few rows behind the last segment
    check(lh, rng, 600, 72, 80, 12, 9, offsets, ids, F32, F32, F32)


def test_runs_inside_a_tile(lh):
    """Segments of 1 to 40 rows that begin and end inside any tile of rows."""
    rng = np.random.default_rng(3)
    lengths = [1, 1, 2, 13, 40, 0, 3, 16, 15, 17, 0, 0, 31, 1, 33, 32, 7]
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    ids = np.array([0, 1, 0, 0, 2, 1, -1, 1, 1, 2, 0, 0, 2, 9, 0, 1, 2], dtype=np.int32)
    for types in TYPES:
        check(lh, rng, int(offsets[-1]), 264, 200, 16, 3, offsets, ids, *types)


@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, F32, F32)])
def test_long_rows(lh, types):
    rng = np.random.default_rng(9)
    for rows, c_in, c_out, rank in ((3, 17408, 64, 16), (130, 8200, 96, 16), (40, 72, 12288, 64)):
        offsets = np.array([0, rows // 2, rows], dtype=np.int64)
        check(lh, rng, rows, c_in, c_out, rank, 2, offsets, np.array([1, 0], dtype=np.int32), *types)


def test_one_adapter_and_defaults(lh):
    """2-D factors, no offsets, no ids, no scale: all rows take the one adapter; y in x's type."""
    rng = np.random.default_rng(4)
    x, a, b = rand(rng, (50, 96), BF16), rand(rng, (8, 96), BF16), rand(rng, (8, 40), BF16)
    y, s = lh.lh_lora(x.to(DEV), a.to(DEV), b.to(DEV), s=True)
    assert y.dtype == BF16 and s.dtype == F32 and s.shape == (50, 8)
    ws, st, wy, yt = expected(x, a[None], b[None], [1.0], None, np.zeros(50, dtype=int), BF16, True)
    near(s, ws, st, "s")
    near(y, wy, yt, "y")
    one = lh.lh_lora(x.to(DEV), a.to(DEV), b.to(DEV), adapter_ids=torch.zeros(1, dtype=torch.int64, device=DEV))
    assert torch.equal(one, y)
    none = lh.lh_lora(x.to(DEV), a.to(DEV), b.to(DEV), adapter_ids=torch.full((1,), -1, device=DEV))
    assert (none == 0).all()


@pytest.mark.parametrize("types", [(BF16, BF16, BF16), (F32, F32, F32)])
def test_strides_and_alignment(lh, types):
    """Rows inside wider buffers, from odd elements on, and factors at odd addresses."""
    rng = np.random.default_rng(11)
    xdt, wdt, ydt = types
    for rows, c_in, c_out, rank in ((37, 160, 96, 16), (5, 160, 96, 16), (80, 101, 77, 7)):
        x, base = rand(rng, (rows, c_in), xdt), rand(rng, (rows, c_out), ydt)
        a, b = rand(rng, (2, rank, c_in), wdt, 0.1), rand(rng, (2, rank, c_out), wdt)
        offsets = np.array([0, rows // 3, rows], dtype=np.int64)
        ids = np.array([1, 0], dtype=np.int32)
        g = rows_of(offsets, ids, rows, 2)
        s, st, y, yt = expected(x, a, b, [1.0, 1.0], base, g, ydt, wdt == BF16)

        def shifted(t, by, pad):
            wide = torch.full((t.numel() + by + 64,), 3.0, dtype=t.dtype, device=DEV)
            if t.dim() == 3:
                v = wide[by:by + t.numel()].view(t.shape)
            else:
                wide = torch.full((t.shape[0] * (t.shape[1] + pad) + by,), 3.0, dtype=t.dtype, device=DEV)
                v = wide[by:].view(t.shape[0], t.shape[1] + pad)[:, :t.shape[1]]
            v.copy_(t)
            return wide, v

        for by, pad in ((0, 5), (1, 8), (3, 3)):
            out, got = shifted(torch.zeros(rows, c_out, dtype=ydt), by, pad + 2)
            lh.lh_lora(shifted(x, by, pad)[1], shifted(a, by, 0)[1], shifted(b, by, 0)[1], base=shifted(base, by, pad)[1], y=got,
                       offsets=torch.from_numpy(offsets).to(DEV), adapter_ids=torch.from_numpy(ids).to(DEV))
            near(got, y, yt, "y at %d" % by)
            assert (out == 3.0).sum() >= out.numel() - rows * c_out, "written outside the rows"


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("rows", [3, 40])
def test_infinities_and_nan_stay_in_their_row(lh, rows, types):
    xdt, wdt, ydt = types
    rng = np.random.default_rng(13)
    x, a, b = rand(rng, (rows, 80), xdt), rand(rng, (2, 20, 80), wdt), rand(rng, (2, 20, 70), wdt)
    clean = lh.lh_lora(x.to(DEV), a.to(DEV), b.to(DEV), adapter_ids=torch.ones(1, dtype=torch.int32, device=DEV), out_dtype=ydt)
    x[1, 7], x[2, 79] = float("inf"), float("nan")
    a[0] = float("nan")                              # an adapter that no row takes
    y, s = lh.lh_lora(x.to(DEV), a.to(DEV), b.to(DEV), adapter_ids=torch.ones(1, dtype=torch.int32, device=DEV), out_dtype=ydt, s=True)
    assert torch.isinf(s[1]).all() and torch.isnan(s[2]).all()
    assert torch.equal(torch.sign(s[1]).cpu(), torch.sign(a[1, :, 7].float()))
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[2]).all()
    others = [t for t in range(rows) if t not in (1, 2)]
    assert torch.equal(y[others], clean[others])
    # two infinities of one sign: the formula's infinity
    b1 = b.abs()
    x1, a1 = torch.ones(rows, 80, dtype=xdt), a.abs()
    x1[1, 7] = float("inf")
    y = lh.lh_lora(x1.to(DEV), a1[1].to(DEV), b1[1].to(DEV), out_dtype=ydt)
    assert (y[1] == float("inf")).all() and torch.isfinite(y[2]).all()


def test_bad_offsets_stay_inside(lh):
    """Offsets outside the rows or decreasing never lead outside a buffer."""
    rng = np.random.default_rng(17)
    x, a, b = rand(rng, (20, 64), BF16).to(DEV), rand(rng, (3, 8, 64), BF16).to(DEV), rand(rng, (3, 8, 48), BF16).to(DEV)
    wide = torch.full((40, 48), 9.0, dtype=BF16, device=DEV)
    for offsets in ([-5, 3, 30, 50], [4, 2, 10, 10], [-(1 << 40), 1 << 40, 5, -3], [30, 40, 50, 60]):
        off = torch.tensor(offsets, device=DEV)
        lh.lh_lora(x, a, b, offsets=off, y=wide[10:30])
        lh.lh_lora_weight_grad(x, wide[10:30], torch.ones(20, 8, device=DEV), torch.ones(20, 8, device=DEV), 3, offsets=off)
        assert (wide[:10] == 9).all() and (wide[30:] == 9).all()
    # every segment claims all rows: more rows than there are, in more slots than there is room for
    rows = 1500
    off = torch.tensor([0, rows] * 20 + [0], device=DEV)
    x, p = rand(rng, (rows, 64), BF16).to(DEV), torch.ones(rows, 8, device=DEV)
    nbytes = lh.lh_lora_weight_grad_workspace_bytes(rows, 40, 40, 8, 64, 64)
    ws = torch.full((nbytes + 4096,), 3, dtype=torch.uint8, device=DEV)
    da, db = lh.lh_lora_weight_grad(x, x, p, p, 40, offsets=off, workspace=ws[:nbytes])
    torch.cuda.synchronize()
    assert (ws[nbytes:] == 3).all() and da.shape == (40, 8, 64)


def test_far_adapters(lh):
    """Adapters whose elements lie past 2^31, and rows past 2^32 bytes."""
    rng = np.random.default_rng(19)
    n, rank, c_in, c_out = 1200, 128, 16384, 64
    a = torch.empty((n, rank, c_in), dtype=BF16, device=DEV)
    last = rand(rng, (1, rank, c_in), BF16, c_in ** -0.5)
    a[-1:] = last.to(DEV)
    b = rand(rng, (n, rank, c_out), BF16, 0.2)
    x = rand(rng, (40, c_in), BF16)
    far = torch.empty((140000, c_in), dtype=BF16, device=DEV)
    far[-40:] = x.to(DEV)
    s, st, y, yt = expected(x, last, b[-1:], [1.0], None, np.zeros(40, dtype=int), BF16, True)
    for ids, off in ((torch.full((140000,), -1, dtype=torch.int32), None), (torch.tensor([-1, n - 1]), torch.tensor([0, 139960, 140000]))):
        if off is None:
            ids[-40:] = n - 1
        got = lh.lh_lora(far, a, b.to(DEV), adapter_ids=ids.to(DEV), offsets=None if off is None else off.to(DEV))
        near(got[-40:], y, yt, "y")
        assert (got[:-40] == 0).all()
    dx = lh.lh_lora_grad(rand(rng, (40, c_out), BF16).to(DEV), a, b.to(DEV), adapter_ids=torch.full((40,), n - 1, device=DEV))
    assert torch.isfinite(dx).all() and (dx != 0).any()


# ---------------------------------------------------------------------------
# gradients to the adapters
# ---------------------------------------------------------------------------
def wanted(p, x, scale, g, adapters, old=None, beta=0.0):
    p, x = f64(p), f64(x)
    out = np.zeros((adapters, p.shape[1], x.shape[1]))
    tol = np.zeros_like(out)
    for k in range(adapters):
        at = np.nonzero(g == k)[0]
        out[k] = scale[k] * (p[at].T @ x[at])
        mass = abs(scale[k]) * (np.abs(p[at]).T @ np.abs(x[at]))
        tol[k] = spread(len(at)) * mass
    if old is not None:
        out += beta * old
        tol += 3 * U * np.abs(beta * old)
    return out, tol + 3 * U * np.abs(out)


def weights_case(lh, rng, rows, c_in, c_out, rank, adapters, offsets, ids, xdt, odt, kept=False, beta=0.0, give_offsets=True,
                 scaled=True):
    print("case rows=%d %d %d rank=%d adapters=%d segments=%d %s %s kept=%s beta=%s" % (
        rows, c_in, c_out, rank, adapters, len(ids), xdt, odt, kept, beta), flush=True)
    x, dy = rand(rng, (rows, c_in), xdt).to(DEV), rand(rng, (rows, c_out), xdt).to(DEV)
    s, ds = rand(rng, (rows, rank), F32).to(DEV), rand(rng, (rows, rank), F32).to(DEV)
    scale = torch.from_numpy(rng.uniform(0.25, 2, adapters).astype(np.float32)).to(DEV) if scaled else None
    sc = f64(scale) if scaled else np.ones(adapters)
    g = rows_of(offsets, ids, rows, adapters)
    for v in (x, dy, s, ds):                         # what no adapter's rows hold is not read
        v[torch.from_numpy(g < 0).to(DEV)] = float("nan")
    values, scales = lh.lh_checkpoint_pack(x) if kept else (x, None)
    meant = lh.lh_checkpoint_unpack(values, scales, out_dtype=F32) if kept else x
    old = [rand(rng, (adapters, rank, c), odt).to(DEV) for c in (c_in, c_out)]
    kw = dict(scale=scale, offsets=torch.from_numpy(offsets).to(DEV) if give_offsets else None,
              adapter_ids=torch.from_numpy(ids).to(DEV), x_scale=scales)
    if beta == 0.0:
        kw.update(da=torch.full_like(old[0], float("nan")), db=torch.full_like(old[1], float("nan")))
    else:
        kw.update(da=old[0].clone(), db=old[1].clone(), beta=beta)
    da, db = lh.lh_lora_weight_grad(values, dy, s, ds, adapters, **kw)
    assert da is kw["da"] and db is kw["db"]
    u = 2.0 ** -8 if odt == BF16 else U
    for got, p, v, o, what in ((da, ds, meant, old[0], "da"), (db, s, dy, old[1], "db")):
        want, tol = wanted(p, v, sc, g, adapters, f64(o) if beta else None, beta)
        near(got, want, tol + u * (np.abs(want) + tol) + 1e-37, what)
    again = {k: v for k, v in kw.items() if k not in ("da", "db", "beta")}
    if beta == 0.0 and odt == F32:                   # one of the two, new tensors, the same bits
        only, none = lh.lh_lora_weight_grad(values, dy, None, ds, adapters, **again, db=False)
        assert none is None and torch.equal(only, da)
        none, only = lh.lh_lora_weight_grad(values, dy, s, None, adapters, **again, da=False)
        assert none is None and torch.equal(only, db)


WSIZES = [(1, 16, 16, 1), (2, 17, 33, 3), (5, 1, 128, 16), (16, 64, 1, 16), (33, 272, 100, 8), (64, 256, 512, 64),
          (100, 96, 1111, 17), (257, 200, 1000, 128), (300, 768, 256, 250), (700, 130, 64, 33), (2500, 64, 520, 16)]


@pytest.mark.parametrize("rows,c_in,c_out,rank", WSIZES)
@pytest.mark.parametrize("xdt,odt,kept", [(BF16, F32, False), (F32, F32, False), (BF16, BF16, True), (F32, F32, True)])
def test_weight_gradients(lh, rows, c_in, c_out, rank, xdt, odt, kept):
    rng = np.random.default_rng([2, rows, c_in, c_out, rank])
    offsets, ids = segments(rng, rows, int(rng.integers(1, 9)), 3)
    weights_case(lh, rng, rows, c_in, c_out, rank, 3, offsets, ids, xdt, odt, kept, beta=float(rng.choice([0.0, 1.0, 0.5])))


@pytest.mark.parametrize("xdt", [BF16, F32])
def test_weight_gradients_of_many_segments(lh, xdt):
    rng = np.random.default_rng(23)
    for rows, n, adapters in ((900, 300, 5), (1200, 40, 70), (64, 64, 900)):
        offsets, ids = segments(rng, rows, n, adapters, 0.1)
        weights_case(lh, rng, rows, 72, 40, 12, adapters, offsets, ids, xdt, F32)
    ids = rng.integers(-1, 4, 130).astype(np.int64)      # a row each
    weights_case(lh, rng, 130, 72, 40, 12, 4, np.arange(131), ids, xdt, F32, give_offsets=False, scaled=False)


def test_weight_gradients_of_long_segments(lh):
    rng = np.random.default_rng(29)
    for kept in (False, True):
        weights_case(lh, rng, 9000, 160, 96, 16, 2, np.array([0, 8500, 9000]), np.array([0, 1], dtype=np.int32), BF16, F32, kept)
    weights_case(lh, rng, 5000, 96, 160, 64, 3, np.array([0, 5000, 5000]), np.array([2, 0], dtype=np.int32), F32, F32)


def test_adapters_without_rows(lh):
    """Their gradient is zero, or beta times what was there."""
    s = torch.ones(4, 8, device=DEV)
    x, dy = torch.ones(4, 40, device=DEV), torch.ones(4, 24, device=DEV)
    off = torch.tensor([0, 4], device=DEV)
    kw = dict(offsets=off, adapter_ids=torch.tensor([2], device=DEV))
    da, db = lh.lh_lora_weight_grad(x, dy, s, s, 5, **kw)
    assert (da[2] == 4).all() and (db[2] == 4).all() and (da[[0, 1, 3, 4]] == 0).all() and (db[[0, 1, 3, 4]] == 0).all()
    lh.lh_lora_weight_grad(x, dy, s, s, 5, **kw, da=da, db=db, beta=0.5)
    assert (da[2] == 6).all() and (db[[0, 1, 3, 4]] == 0).all()
    none = dict(offsets=torch.tensor([0], device=DEV), adapter_ids=torch.empty(0, dtype=torch.int32, device=DEV))
    lh.lh_lora_weight_grad(x, dy, s, s, 5, **none, da=da, db=db, beta=0.5)
    assert (da[2] == 3).all()
    da, db = lh.lh_lora_weight_grad(x[:0], dy[:0], s[:0], s[:0], 5, **none)
    assert (da == 0).all() and (db == 0).all() and da.shape == (5, 8, 40)


def test_gradients_are_differences(lh):
    """The gradients against central differences of a scalar of lh_lora's own
    outputs.  The product is linear in x and in each factor, so a difference of
    any step h is exact but for rounding: with |L| terms summed in 64 bits from
    fp32 outputs y, each off by 2^-20 of its mass at most, 2h below."""
    rng = np.random.default_rng(31)
    rows, c_in, c_out, rank, n = 12, 24, 20, 4, 2
    off, ids = torch.tensor([0, 5, 12], device=DEV), torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    x, a, b = (rand(rng, shape, F32).to(DEV) for shape in ((rows, c_in), (n, rank, c_in), (n, rank, c_out)))
    scale = torch.tensor([0.5, 2.0], device=DEV)
    dy = rand(rng, (rows, c_out), F32).to(DEV)
    kw = dict(scale=scale, offsets=off, adapter_ids=ids)
    y, s = lh.lh_lora(x, a, b, s=True, **kw)
    dx, ds = lh.lh_lora_grad(dy, a, b, ds=True, **kw)
    da, db = lh.lh_lora_weight_grad(x, dy, s, ds, n, **kw)
    mass = f64(lh.lh_lora(x.abs(), a.abs(), b.abs(), **kw))

    def loss():
        return float((lh.lh_lora(x, a, b, **kw).double() * dy.double()).sum())

    tol = 2.0 ** -18 * float((mass * np.abs(f64(dy))).sum())
    for leaf, grad in ((x, dx), (a, da), (b, db)):
        flat, gf = leaf.view(-1), grad.view(-1)
        for i in rng.choice(flat.numel(), 12, replace=False).tolist():
            keep = float(flat[i])
            flat[i] = keep + 1
            up = loss()
            flat[i] = keep - 1
            down = loss()
            flat[i] = keep
            assert abs((up - down) / 2 - float(gf[i])) <= 4 * tol, (i, up, down, float(gf[i]))


# ---------------------------------------------------------------------------
# refusals of the binding
# ---------------------------------------------------------------------------
def test_refusals(lh):
    x, dy = torch.zeros(4, 32, device=DEV), torch.zeros(4, 16, device=DEV)
    a, b = torch.zeros(2, 8, 32, device=DEV), torch.zeros(2, 8, 16, device=DEV)
    p = torch.zeros(4, 8, device=DEV)
    off, ids = torch.tensor([0, 2, 4], device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    bad = [lambda: lh.lh_lora(x, a, b[:, :4].contiguous()), lambda: lh.lh_lora(dy, a, b, offsets=off),
           lambda: lh.lh_lora(x, a, b, offsets=off[:0]), lambda: lh.lh_lora(x, a, b, offsets=off, adapter_ids=ids[:1]),
           lambda: lh.lh_lora(x, a, b, offsets=torch.tensor([0, 1, 2, 4], device=DEV)),
           lambda: lh.lh_lora(x, a, b, torch.ones(3, device=DEV), offsets=off), lambda: lh.lh_lora(x, a, b, adapter_ids=ids),
           lambda: lh.lh_lora(x, a, b, offsets=off, base=torch.zeros(4, 15, device=DEV)),
           lambda: lh.lh_lora(x, a, b, offsets=off, base=torch.zeros(3, 16, device=DEV)),
           lambda: lh.lh_lora(x, a, b, offsets=off, y=torch.zeros(3, 16, device=DEV)),
           lambda: lh.lh_lora(x.t(), a, b, offsets=off), lambda: lh.lh_lora(x, a.transpose(1, 2), b, offsets=off),
           lambda: lh.lh_lora(x, a, b, offsets=off, s=torch.zeros(4, 9, device=DEV)),
           lambda: lh.lh_lora(x, a, b, offsets=off.cpu()), lambda: lh.lh_lora(x, a, b, offsets=off, adapter_ids=ids.cpu()),
           lambda: lh.lh_lora(x, a, b, offsets=off, s=torch.zeros(4, 8)),
           lambda: lh.lh_lora(x, a, b, offsets=off, workspace=torch.zeros(1 << 16, dtype=torch.uint8)),
           lambda: lh.lh_lora_grad(x, a, b, offsets=off),
           lambda: lh.lh_lora_weight_grad(x, dy, None, None, 2), lambda: lh.lh_lora_weight_grad(x, dy, p, None, 2, offsets=off),
           lambda: lh.lh_lora_weight_grad(x[:3], dy, p, p, 2, offsets=off), lambda: lh.lh_lora_weight_grad(x, dy, p, p, 2, beta=1.0),
           lambda: lh.lh_lora_weight_grad(x, dy, p, p[:, :4].contiguous(), 2, offsets=off),
           lambda: lh.lh_lora_weight_grad(x, dy, p, p, 2, offsets=off, da=torch.zeros(2, 8, 31, device=DEV)),
           lambda: lh.lh_lora_weight_grad(x.to(torch.uint8), dy, p, p, 2, offsets=off, x_scale=torch.zeros(4, 2, dtype=torch.uint8, device=DEV))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail("call %d was taken" % i)
    wrong = [lambda: lh.lh_lora(x.half(), a, b, offsets=off), lambda: lh.lh_lora(x, a, b.to(BF16), offsets=off),
             lambda: lh.lh_lora(x, a.half(), b.half(), offsets=off), lambda: lh.lh_lora(x, a, b, offsets=off.int()),
             lambda: lh.lh_lora(x, a, b, offsets=off, adapter_ids=ids.float()),
             lambda: lh.lh_lora(x, a, b, offsets=off, base=torch.zeros(4, 16, device=DEV, dtype=BF16), out_dtype=F32),
             lambda: lh.lh_lora(x, a, b, offsets=off, out_dtype=torch.float16),
             lambda: lh.lh_lora_weight_grad(x, dy, p.to(BF16), p, 2, offsets=off),
             lambda: lh.lh_lora_weight_grad(x, dy, p, p, 2, offsets=off, out_dtype=torch.float16),
             lambda: lh.lh_lora_weight_grad(x, dy, p, p, 2, offsets=off, x_scale=torch.zeros(4, 1, dtype=torch.uint8, device=DEV))]
    for i, f in enumerate(wrong):
        with pytest.raises(TypeError):
            f()
            pytest.fail("call %d was taken" % i)
    with pytest.raises(lh.LHError):
        lh.lh_lora(x, torch.zeros(2, 257, 32, device=DEV), torch.zeros(2, 257, 16, device=DEV), offsets=off)
    with pytest.raises(lh.LHError):
        lh.lh_lora(x, a, b, offsets=off, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(lh.LHError):
        lh.lh_lora_weight_grad(x, dy, p, p, 1025, adapter_ids=torch.zeros(1, dtype=torch.int32, device=DEV))


def test_nothing_to_do(lh):
    for dt in (BF16, F32):
        a, b = torch.zeros(2, 8, 32, device=DEV, dtype=dt), torch.zeros(2, 8, 16, device=DEV, dtype=dt)
        x, base = torch.ones(4, 32, device=DEV, dtype=dt), torch.ones(4, 16, device=DEV, dtype=dt)
        assert lh.lh_lora(x[:0], a, b, offsets=torch.zeros(1, dtype=torch.int64, device=DEV)).shape == (0, 16)
        off = torch.tensor([0, 4], device=DEV)
        assert torch.equal(lh.lh_lora(x, a[:, :0], b[:, :0], offsets=off, base=base), base)                       # rank 0
        assert torch.equal(lh.lh_lora(x[:, :0], a[:, :, :0], b, offsets=off, base=base), base)                    # no inputs
        assert torch.equal(lh.lh_lora(x, a[:0], b[:0], offsets=off, adapter_ids=torch.zeros(1, dtype=torch.int32, device=DEV), base=base), base)
        y, s = lh.lh_lora(x, a, b[:, :, :0], offsets=off, s=True)                                                  # no outputs but s
        assert y.shape == (4, 0) and (s == 0).all()
        da, db = lh.lh_lora_weight_grad(x, base, s, s, 2, offsets=off, adapter_ids=torch.zeros(1, dtype=torch.int32, device=DEV))
        assert (da == 0).all() and (db == 0).all()
        assert lh.lh_lora_weight_grad(x, base[:, :0], s, s, 2, offsets=off, adapter_ids=torch.zeros(1, dtype=torch.int32, device=DEV))[1].shape == (2, 8, 0)

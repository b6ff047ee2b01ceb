"""Products with NVFP4 weights and their gradient against the definition in 64
bits (computed on the CPU from the nibbles' and codes' bit fields).

Tolerance, derived from the arithmetic: products are exact and added in fp32,
so a sum of n terms is off by at most lambda sqrt(n) 2^-24 sum |terms| (the
probabilistic bound with lambda = 8, failing with probability 2 exp(-32)),
plus two roundings for the scale, plus the rounding to the output's type (the
unit roundoff 2^-p of its p significant bits: 2^-8 for bf16, 2^-24 for fp32)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def units64(packed, codes):
    """r * c by the formats' fields, [..., c_in] in fp64."""
    p = packed.numpy()
    nib = np.stack([p & 15, p >> 4], axis=-1).reshape(*p.shape[:-1], -1).astype(np.int64)
    e, m = (nib >> 1) & 3, nib & 1
    r = np.where(e == 0, 0.5 * m, 2.0 ** (e - 1.0) * (1 + 0.5 * m)) * np.where(nib & 8, -1.0, 1.0)
    c = codes.numpy().astype(np.int64)
    e, m = c >> 3, c & 7
    s = np.where(e == 0, m * 2.0 ** -9, 2.0 ** (e - 7.0) * (1 + m / 8.0))
    return r * np.repeat(s, 16, axis=-1)


def weights(rng, g, c_out, c_in, wide=False):
    """Random nibbles and codes (all 126 when wide, else a middle range)."""
    packed = torch.from_numpy(rng.integers(0, 256, (g, c_out, c_in // 2), dtype=np.uint8))
    lo, hi = (1, 127) if wide else (0x28, 0x50)
    codes = torch.from_numpy(rng.integers(lo, hi, (g, c_out, c_in // 16), dtype=np.uint8))
    s = torch.from_numpy(rng.uniform(1e-4, 1e-2, g).astype(np.float32))
    return packed, codes, s


def tokens(rng, shape, dtype):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(dtype)


def near(y, x, w, scale, what):
    """y against scale * x @ w.T in 64 bits; x [t, n], w [m, n] fp64 arrays."""
    n = x.shape[1]
    ref, mass = scale * (x @ w.T), abs(scale) * (np.abs(x) @ np.abs(w).T)
    got = y.double().cpu().numpy()
    ulp = 2.0 ** -8 if y.dtype == BF16 else 2.0 ** -24
    tol = (8 * np.sqrt(n) * 2.0 ** -24 + 2.0 ** -23) * mass
    tol = tol + ulp * (np.abs(ref) + tol) + 1e-37
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), "%s: %d of %d outside, worst %.3g of its tolerance" % (
        what, bad.sum(), bad.size, np.max(np.abs(got - ref) / tol))


SIZES = [(1, 16, 16), (1, 1, 16), (2, 17, 48), (3, 64, 64), (5, 100, 272), (16, 128, 256), (17, 65, 1040),
         (33, 200, 128), (64, 256, 512), (65, 300, 320), (130, 513, 144), (300, 256, 768), (257, 1000, 256)]


@pytest.mark.parametrize("t,c_out,c_in", SIZES)
@pytest.mark.parametrize("xdt,ydt", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("workspace", [True, False])
def test_product_and_gradient(lh, t, c_out, c_in, xdt, ydt, workspace):
    print("case t=%d c_out=%d c_in=%d %s->%s ws=%s" % (t, c_out, c_in, xdt, ydt, workspace), flush=True)
    rng = np.random.default_rng([t, c_out, c_in])
    packed, codes, s = weights(rng, 1, c_out, c_in)
    x, dy = tokens(rng, (t, c_in), xdt), tokens(rng, (t, c_out), xdt)
    u = units64(packed, codes)[0]
    dev = [v.to(DEV) for v in (packed, codes, s)]
    y = lh.lh_linear_nvfp4(x.to(DEV), *dev, out_dtype=ydt, workspace=workspace)
    dx = lh.lh_linear_nvfp4_grad(dy.to(DEV), *dev, out_dtype=ydt, workspace=workspace)
    assert y.shape == (t, c_out) and dx.shape == (t, c_in) and y.dtype == dx.dtype == ydt
    near(y, x.double().numpy(), u, float(s[0]), "y")
    near(dx, dy.double().numpy(), u.T, float(s[0]), "dx")
    again = lh.lh_linear_nvfp4(x.to(DEV), *dev, out_dtype=ydt, workspace=workspace)
    assert torch.equal(y, again), "a second call gives other bits"


@pytest.mark.parametrize("t", [1, 4, 16, 40, 96, 200])
@pytest.mark.parametrize("c_out,c_in", [(48, 2048 + 16), (256, 4096), (520, 1536)])
def test_long_sums(lh, t, c_out, c_in):
    print("case t=%d %dx%d" % (t, c_out, c_in), flush=True)
    rng = np.random.default_rng([7, t, c_out])
    packed, codes, s = weights(rng, 1, c_out, c_in)
    u = units64(packed, codes)[0]
    dev = [v.to(DEV) for v in (packed, codes, s)]
    for dt in (BF16, F32):
        x, dy = tokens(rng, (t, c_in), dt), tokens(rng, (t, c_out), dt)
        near(lh.lh_linear_nvfp4(x.to(DEV), *dev, out_dtype=F32), x.double().numpy(), u, float(s[0]), "y")
        near(lh.lh_linear_nvfp4_grad(dy.to(DEV), *dev, out_dtype=F32), dy.double().numpy(), u.T, float(s[0]), "dx")


@pytest.mark.parametrize("t,c_out,c_in", [(1, 300, 4096), (20, 300, 512), (600, 700, 1056)])
def test_every_code_and_position(lh, t, c_out, c_in):
    """One-hot activations read the weights out one by one: exact."""
    rng = np.random.default_rng(5)
    packed, codes, _ = weights(rng, 1, c_out, c_in, wide=True)
    u = units64(packed, codes)[0]
    s = torch.ones(1)
    cols, rows = rng.permutation(c_in)[:t], rng.permutation(c_out)[:min(t, c_out)]
    for dt in (BF16, F32):
        x = torch.zeros((t, c_in), dtype=dt)
        x[torch.arange(t), torch.from_numpy(cols)] = 1.0
        y = lh.lh_linear_nvfp4(x.to(DEV), packed.to(DEV), codes.to(DEV), s.to(DEV))
        assert np.array_equal(y.double().cpu().numpy(), u[:, cols].T)
        dy = torch.zeros((len(rows), c_out), dtype=dt)
        dy[torch.arange(len(rows)), torch.from_numpy(rows)] = 1.0
        dx = lh.lh_linear_nvfp4_grad(dy.to(DEV), packed.to(DEV), codes.to(DEV), s.to(DEV))
        assert np.array_equal(dx.double().cpu().numpy(), u[rows])


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("t", [3, 19, 150])
def test_strides_offsets_and_neighbours(lh, dt, t):
    """Rows that start anywhere, outputs inside a larger buffer: what lies
    around input rows (NaN) is not read into the result, what lies around
    output rows is not written."""
    rng = np.random.default_rng([9, t])
    c_out, c_in = 133, 176
    packed, codes, s = weights(rng, 1, c_out, c_in)
    u = units64(packed, codes)[0]
    dev = [v.to(DEV) for v in (packed, codes, s)]
    for shift in (0, 1, 3):
        for n, w, f in ((c_in, u, lh.lh_linear_nvfp4), (c_out, u.T, lh.lh_linear_nvfp4_grad)):
            big = torch.full((t + 2, n + 11), float("nan"), dtype=dt, device=DEV)
            x = tokens(rng, (t, n), dt)
            big[1:t + 1, shift:shift + n] = x.to(DEV)
            m = w.shape[0]
            out = torch.full((t + 2, m + 9), 7.0, dtype=dt, device=DEV)
            y = out[1:t + 1, shift:shift + m]
            args = dict(y=y) if f is lh.lh_linear_nvfp4 else dict(dx=y)
            f(big[1:t + 1, shift:shift + n], *dev, **args)
            near(y, x.double().numpy(), w, float(s[0]), "shift %d" % shift)
            mask = torch.ones_like(out, dtype=torch.bool)
            mask[1:t + 1, shift:shift + m] = False
            assert bool((out[mask] == 7.0).all()), "written outside the output"


def test_groups_with_strides_and_x_scale(lh):
    rng = np.random.default_rng(11)
    g, t, c_out, c_in = 3, 21, 70, 96
    packed, codes, s = weights(rng, g, c_out, c_in)
    u = units64(packed, codes)
    xs = torch.tensor([0.5, 3.0, 1e-3])
    buf = tokens(rng, (g, t + 5, c_in), BF16)
    x = buf.to(DEV)[:, 2:2 + t]
    y = lh.lh_linear_nvfp4(x, packed.to(DEV), codes.to(DEV), s.to(DEV), x_scale=xs.to(DEV), out_dtype=F32)
    dy = tokens(rng, (g, t, c_out), BF16)
    dx = lh.lh_linear_nvfp4_grad(dy.to(DEV), packed.to(DEV), codes.to(DEV), s.to(DEV), out_dtype=F32)
    for i in range(g):
        near(y[i], buf[i, 2:2 + t].double().numpy(), u[i], float(s[i]) * float(xs[i]), "group %d" % i)
        near(dx[i], dy[i].double().numpy(), u[i].T, float(s[i]), "gradient, group %d" % i)


@pytest.mark.parametrize("counts", [[0, 5, 1, 0, 64, 17, 0], [300, 0, 0, 2], [1] * 70, [0, 0, 0], [40], [0] * 65 + [3],
                                    [16, 32, 15, 33, 128, 129]])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("bound", [False, True])
def test_ragged_rows(lh, counts, dt, bound):
    print("case counts=%s %s" % (counts[:8], dt), flush=True)
    rng = np.random.default_rng([13, len(counts)])
    g, c_out, c_in, tail = len(counts), 72, 96, 3
    off = np.concatenate([[0], np.cumsum(counts)])
    n = int(off[-1]) + tail
    packed, codes, s = weights(rng, g, c_out, c_in)
    u = units64(packed, codes)
    x, dy = tokens(rng, (n, c_in), dt), tokens(rng, (n, c_out), dt)
    dev = [torch.from_numpy(off).to(DEV), packed.to(DEV), codes.to(DEV), s.to(DEV)]
    most = max(counts) if bound else 0
    y = torch.full((n, c_out), 7.0, dtype=dt, device=DEV)
    dx = torch.full((n, c_in), 7.0, dtype=dt, device=DEV)
    lh.lh_linear_nvfp4_ragged(x.to(DEV), *dev, y=y, max_group_rows=most)
    lh.lh_linear_nvfp4_ragged_grad(dy.to(DEV), *dev, dx=dx, max_group_rows=most)
    for i in range(g):
        r = slice(int(off[i]), int(off[i + 1]))
        if off[i + 1] > off[i]:
            near(y[r], x[r].double().numpy(), u[i], float(s[i]), "group %d" % i)
            near(dx[r], dy[r].double().numpy(), u[i].T, float(s[i]), "gradient, group %d" % i)
    assert bool((y[int(off[-1]):] == 7.0).all()) and bool((dx[int(off[-1]):] == 7.0).all())


def test_a_wrong_row_bound_changes_nothing(lh):
    """max_group_rows shapes the work only: a bound far too small gives the same result."""
    rng = np.random.default_rng(17)
    off = torch.tensor([0, 250, 251, 400], dtype=torch.int64)
    packed, codes, s = weights(rng, 3, 80, 128)
    u = units64(packed, codes)
    x = tokens(rng, (400, 128), BF16)
    for most in (1, 20, 100, 250, 10 ** 6):
        y = lh.lh_linear_nvfp4_ragged(x.to(DEV), off.to(DEV), packed.to(DEV), codes.to(DEV), s.to(DEV),
                                      max_group_rows=most, out_dtype=F32)
        for i in range(3):
            r = slice(int(off[i]), int(off[i + 1]))
            near(y[r], x[r].double().numpy(), u[i], float(s[i]), "bound %d group %d" % (most, i))


def test_offsets_outside_the_buffer_stay_inside(lh):
    """Offsets are clamped, a decreasing pair is an empty group; the buffers
    are views inside larger ones whose surroundings must not change."""
    rng = np.random.default_rng(19)
    packed, codes, s = weights(rng, 3, 40, 64)
    u = units64(packed, codes)
    x = tokens(rng, (50, 64), BF16)
    out = torch.full((90, 40), 7.0, dtype=F32, device=DEV)
    off = torch.tensor([-5, 30, 20, 10 ** 9], dtype=torch.int64)      # groups 0..29, none, 20..49
    lh.lh_linear_nvfp4_ragged(x.to(DEV), off.to(DEV), packed.to(DEV), codes.to(DEV), s.to(DEV), y=out[20:70])
    near(out[20:40], x[:20].double().numpy(), u[0], float(s[0]), "group 0")
    near(out[50:70], x[30:].double().numpy(), u[2], float(s[2]), "group 2")
    assert bool((out[:20] == 7.0).all()) and bool((out[70:] == 7.0).all())


def test_empty_problems(lh):
    rng = np.random.default_rng(23)
    packed, codes, s = [v.to(DEV) for v in weights(rng, 1, 32, 64)]
    assert lh.lh_linear_nvfp4(torch.empty((0, 64), dtype=BF16, device=DEV), packed, codes, s).shape == (0, 32)
    assert lh.lh_linear_nvfp4_grad(torch.empty((0, 32), dtype=BF16, device=DEV), packed, codes, s).shape == (0, 64)
    none = torch.empty((1, 0, 32), dtype=torch.uint8, device=DEV)
    nsc = torch.empty((1, 0, 4), dtype=torch.uint8, device=DEV)
    assert lh.lh_linear_nvfp4(torch.ones((3, 64), dtype=BF16, device=DEV), none, nsc, s).shape == (3, 0)
    dx = torch.full((3, 64), 7.0, dtype=BF16, device=DEV)
    lh.lh_linear_nvfp4_grad(torch.empty((3, 0), dtype=BF16, device=DEV), none, nsc, s, dx=dx)
    assert bool((dx == 0).all())                                       # a sum over no outputs
    y = torch.full((3, 32), 7.0, dtype=F32, device=DEV)
    lh.lh_linear_nvfp4(torch.empty((3, 0), dtype=BF16, device=DEV), torch.empty((1, 32, 0), dtype=torch.uint8, device=DEV),
                       torch.empty((1, 32, 0), dtype=torch.uint8, device=DEV), s, y=y)
    assert bool((y == 0).all())
    off = torch.zeros(2, dtype=torch.int64, device=DEV)
    assert lh.lh_linear_nvfp4_ragged(torch.empty((0, 64), dtype=BF16, device=DEV), off, packed, codes, s).shape == (0, 32)


def test_a_token_with_nan_keeps_it_to_itself(lh):
    rng = np.random.default_rng(29)
    packed, codes, s = weights(rng, 1, 200, 160)
    u = units64(packed, codes)[0]
    for t in (2, 30, 140):
        for dt in (BF16, F32):
            x = tokens(rng, (t, 160), dt)
            x[t // 2, 5] = float("nan")
            y = lh.lh_linear_nvfp4(x.to(DEV), packed.to(DEV), codes.to(DEV), s.to(DEV), out_dtype=F32)
            keep = [i for i in range(t) if i != t // 2]
            near(y[keep], x[keep].double().numpy(), u, float(s[0]), "the other tokens")


@pytest.mark.parametrize("t,c_out,c_in", [(1, 40, 272), (2, 40, 272), (5, 64, 272), (1500, 512, 528), (2100, 512, 1056),
                                          (400, 1000, 272), (700, 512, 256), (4100, 1000, 272), (4100, 2048, 272),
                                          (32, 8192, 2064)])
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("workspace", [True, None])
def test_infinities_as_the_formula_has_them(lh, t, c_out, c_in, dt, workspace):
    """An infinite activation meets every weight: infinite of the weight's
    sign, NaN where the weight is zero, and nothing for the other tokens."""
    print("case t=%d %dx%d %s ws=%s" % (t, c_out, c_in, dt, workspace), flush=True)
    rng = np.random.default_rng([59, t, c_in])
    packed, codes, s = weights(rng, 1, c_out, c_in)
    packed[0, 0], packed[0, :, 3] = 0x31, 0x31                       # rows and columns without a zero
    u = torch.from_numpy(units64(packed, codes)[0]).to(DEV)
    s_ = float(s[0])
    dev = [v.to(DEV) for v in (packed, codes, s)]
    for n, w, f in ((c_in, u, lh.lh_linear_nvfp4), (c_out, u.t(), lh.lh_linear_nvfp4_grad)):
        x = torch.from_numpy(rng.standard_normal((t, n)).astype(np.float32)).to(DEV).to(dt)
        for i, (row, col) in enumerate(((0, 0), (t // 2, n - 1), (t - 1, 6), (t - 1, n // 2))):
            x[row, col] = float("inf") if i % 2 == 0 else -float("inf")
        y = f(x, *dev, out_dtype=F32, workspace=workspace).double()
        bad = torch.zeros(t, dtype=torch.bool)
        bad[[0, t // 2, t - 1]] = True
        assert bool(torch.isfinite(y[~bad.to(DEV)]).all())
        for r in {0, t // 2, t - 1}:
            ref = s_ * (x[r].double() * w).sum(1)
            assert torch.equal(torch.isnan(y[r]), torch.isnan(ref)) and torch.equal(torch.isinf(y[r]), torch.isinf(ref))
            assert torch.equal(y[r] == float("inf"), ref == float("inf"))


def test_large_row_strides(lh):
    """Rows more than 2^32 bytes from the buffer's start."""
    rng = np.random.default_rng(31)
    packed, codes, s = weights(rng, 1, 48, 64)
    u = units64(packed, codes)[0]
    ld, t = 1 << 28, 10
    x, dy = tokens(rng, (t, 64), BF16), tokens(rng, (t, 48), BF16)
    buf = torch.zeros(ld * (t - 1) + 4096 + 64, dtype=BF16, device=DEV)
    xv, yv = buf.as_strided((t, 64), (ld, 1)), buf.as_strided((t, 48), (ld, 1), 4096)
    xv.copy_(x.to(DEV))
    lh.lh_linear_nvfp4(xv, packed.to(DEV), codes.to(DEV), s.to(DEV), y=yv)
    near(yv, x.double().numpy(), u, float(s[0]), "y")
    yv.copy_(dy.to(DEV))
    lh.lh_linear_nvfp4_grad(yv, packed.to(DEV), codes.to(DEV), s.to(DEV), dx=xv)
    near(xv, dy.double().numpy(), u.T, float(s[0]), "dx")


def test_gradient_against_the_formula_and_differences(lh):
    """L(x) = sum(dy * y(x)): its difference quotients in x are dx (y is
    linear, so the quotient has no step error), and <dy, y(v)> = <dx, v>."""
    rng = np.random.default_rng(37)
    t, c_out, c_in = 6, 90, 112
    packed, codes, s = [v.to(DEV) for v in weights(rng, 1, c_out, c_in)]
    x, dy = tokens(rng, (t, c_in), F32).to(DEV), tokens(rng, (t, c_out), F32).to(DEV)
    dx = lh.lh_linear_nvfp4_grad(dy, packed, codes, s).double()
    y0 = lh.lh_linear_nvfp4(x, packed, codes, s).double()
    mass = (dy.double().abs() * y0.abs()).sum()
    for i, j in ((0, 0), (2, 17), (5, 111), (3, 64)):
        up = x.clone()
        up[i, j] += 64.0
        h = float(up[i, j].double() - x[i, j].double())
        quotient = ((lh.lh_linear_nvfp4(up, packed, codes, s).double() - y0) * dy.double()).sum() / h
        # fp32 sums of 112 terms on both sides, differenced
        tol = 4 * 8 * np.sqrt(c_in) * 2.0 ** -24 * (mass + abs(h) * dx.abs().max() * c_out) / abs(h) + 1e-6 * dx.abs().max()
        assert abs(quotient - dx[i, j]) <= tol, (i, j)
    v = tokens(rng, (t, c_in), F32).to(DEV)
    lhs = (dy.double() * lh.lh_linear_nvfp4(v, packed, codes, s).double()).sum()
    rhs = (dx * v.double()).sum()
    scale = (dx.abs() * v.double().abs()).sum()
    assert abs(lhs - rhs) <= 8 * np.sqrt(c_out + c_in) * 2.0 ** -24 * scale * 8


def test_another_stream(lh):
    rng = np.random.default_rng(41)
    packed, codes, s = weights(rng, 1, 64, 128)
    u = units64(packed, codes)[0]
    x = tokens(rng, (33, 128), F32)
    st = torch.cuda.Stream()
    dev = [v.to(DEV) for v in (x, packed, codes, s)]
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        y = lh.lh_linear_nvfp4(*dev)
    st.synchronize()
    near(y, x.double().numpy(), u, float(s[0]), "y")


def test_refusals(lh):
    rng = np.random.default_rng(43)
    packed, codes, s = [v.to(DEV) for v in weights(rng, 1, 32, 64)]
    x = torch.zeros((4, 64), dtype=BF16, device=DEV)
    with pytest.raises(ValueError):
        lh.lh_linear_nvfp4(x.cpu(), packed, codes, s)
    with pytest.raises(ValueError):
        lh.lh_linear_nvfp4(x[:, :48], packed, codes, s)
    with pytest.raises(ValueError):
        lh.lh_linear_nvfp4(x.t().contiguous().t(), packed, codes, s)
    with pytest.raises(TypeError):
        lh.lh_linear_nvfp4(x.half(), packed, codes, s)
    with pytest.raises(TypeError):
        lh.lh_linear_nvfp4(x, packed.int(), codes, s)
    with pytest.raises(ValueError):
        lh.lh_linear_nvfp4(x, packed, codes[..., :3], s)
    with pytest.raises(ValueError):
        lh.lh_linear_nvfp4(x, packed, codes, torch.cat([s, s]))
    with pytest.raises(ValueError):
        lh.lh_linear_nvfp4(x, packed, codes, s, y=torch.empty((4, 31), dtype=BF16, device=DEV))
    with pytest.raises(ValueError):
        lh.lh_linear_nvfp4_ragged(x, torch.zeros(3, dtype=torch.int64, device=DEV), packed, codes, s)
    with pytest.raises(TypeError):
        lh.lh_linear_nvfp4_ragged(x, torch.zeros(2, dtype=torch.int32, device=DEV), packed, codes, s)


def test_a_workspace_on_the_host_or_with_gaps_is_refused(lh):
    rng = np.random.default_rng(47)
    packed, codes, s = [v.to(DEV) for v in weights(rng, 1, 32, 64)]
    x = torch.zeros((40, 64), dtype=F32, device=DEV)
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty((1 << 20, 2), dtype=torch.uint8, device=DEV)[:, 0]):
        with pytest.raises(ValueError):
            lh.lh_linear_nvfp4(x, packed, codes, s, workspace=ws)
        with pytest.raises(ValueError):
            lh.lh_linear_nvfp4_grad(torch.zeros((40, 32), device=DEV), packed, codes, s, workspace=ws)
        with pytest.raises(ValueError):
            lh.lh_moe_sort(torch.zeros((4, 2), dtype=torch.int64, device=DEV), 3, workspace=ws)


@pytest.mark.parametrize("t", [1, 2, 5, 70])
def test_groups_side_by_side_in_wide_rows(lh, t):
    """The output as [tokens, groups, columns]: the same values as group by group."""
    g, c_out, c_in = 3, 48, 80
    rng = np.random.default_rng(53)
    packed, codes, s = [v.to(DEV) for v in weights(rng, g, c_out, c_in)]
    x = torch.from_numpy(rng.standard_normal((t, g, c_in)).astype(np.float32)).to(DEV).transpose(0, 1)
    wide = torch.full((t, g, c_out), 9.0, device=DEV)
    lh.lh_linear_nvfp4(x, packed, codes, s, y=wide.transpose(0, 1))
    assert torch.equal(wide.transpose(0, 1), lh.lh_linear_nvfp4(x.contiguous(), packed, codes, s))
    dy = torch.from_numpy(rng.standard_normal((t, g, c_out)).astype(np.float32)).to(DEV).transpose(0, 1)
    dwide = torch.full((t, g, c_in), 9.0, device=DEV)
    lh.lh_linear_nvfp4_grad(dy, packed, codes, s, dx=dwide.transpose(0, 1))
    assert torch.equal(dwide.transpose(0, 1), lh.lh_linear_nvfp4_grad(dy.contiguous(), packed, codes, s))
    with pytest.raises(lh.LHError):
        lh.lh_linear_nvfp4(x, packed, codes, s, y=torch.empty((t, c_out), device=DEV).expand(g, t, c_out))


LARGE = [(5, 300, 2064), (24, 4096, 1056), (40, 8192, 1056), (40, 8192, 1040), (300, 4096, 528), (300, 4096, 512),
         (1100, 4096, 1040), (1100, 4096, 1024), (200, 2048, 2064), (4099, 4000, 2064), (4096, 4096, 2048),
         (4100, 1000, 272), (4100, 512, 2064), (4100, 512, 2048), (4100, 2048, 272), (4100, 1000, 2064),
         (1500, 512, 528), (2000, 512, 1024), (2100, 512, 1056), (32, 8192, 2064), (400, 1000, 272), (1000, 512, 256),
         (400, 1000, 528), (700, 512, 1024), (700, 512, 256), (700, 1000, 1168), (1500, 512, 2048)]


@pytest.mark.parametrize("t,c_out,c_in", LARGE)
@pytest.mark.parametrize("dt", [BF16, F32])
def test_larger_layers(lh, t, c_out, c_in, dt):
    """Sizes at which tiles of 16 to 256 tokens and splits of the sum are
    chosen, whole and ragged at every end; the 64-bit reference is computed on
    the GPU here.  The workspace's contents must not matter."""
    print("case t=%d c_out=%d c_in=%d %s" % (t, c_out, c_in, dt), flush=True)
    gen = torch.Generator(device=DEV).manual_seed(t)
    packed = torch.randint(0, 256, (1, c_out, c_in // 2), dtype=torch.uint8, device=DEV, generator=gen)
    codes = torch.randint(0x28, 0x50, (1, c_out, c_in // 16), dtype=torch.uint8, device=DEV, generator=gen)
    s = torch.full((1,), 1e-3, device=DEV)
    u = torch.from_numpy(units64(packed.cpu(), codes.cpu())[0]).to(DEV)
    for n, m, w, grad in ((c_in, c_out, u, False), (c_out, c_in, u.t(), True)):
        x = torch.randn((t, n), device=DEV, generator=gen).to(dt)
        f = lh.lh_linear_nvfp4_grad if grad else lh.lh_linear_nvfp4
        size = lh.lh_linear_nvfp4_workspace_bytes(t, c_in, c_out, dtype=dt, grad=grad)
        ws = torch.full((max(size, 256),), 0xFF, dtype=torch.uint8, device=DEV)
        got = [f(x, packed, codes, s, workspace=ws), f(x, packed, codes, s), f(x, packed, codes, s, workspace=None)]
        assert torch.equal(got[0], got[1])
        x64, scale = x.double(), float(s[0])
        ref, mass = scale * (x64 @ w.t()), scale * (x64.abs() @ w.t().abs())
        ulp = 2.0 ** -8 if dt == BF16 else 2.0 ** -24
        tol = (8 * np.sqrt(n) * 2.0 ** -24 + 2.0 ** -23) * mass
        tol = tol + ulp * (ref.abs() + tol)
        for y in got[1:]:
            assert bool(((y.double() - ref).abs() <= tol).all()), "gradient" if grad else "product"


@pytest.mark.parametrize("n,c_out,c_in", [(128, 512, 512), (600, 512, 528), (9000, 300, 272), (20000, 512, 256),
                                          (6, 300, 528)])
def test_larger_ragged_calls(lh, n, c_out, c_in):
    print("case n=%d c_out=%d c_in=%d" % (n, c_out, c_in), flush=True)
    g = 16
    rng = np.random.default_rng(n)
    counts = rng.multinomial(n, rng.dirichlet(np.full(g, 0.4)))
    off = np.concatenate([[0], np.cumsum(counts)])
    packed, codes, s = weights(rng, g, c_out, c_in)
    u = torch.from_numpy(units64(packed, codes)).to(DEV)
    dev = [torch.from_numpy(off).to(DEV), packed.to(DEV), codes.to(DEV), s.to(DEV)]
    for dt in (BF16, F32):
        ulp = 2.0 ** -8 if dt == BF16 else 2.0 ** -24
        for k, f, w in ((c_in, lh.lh_linear_nvfp4_ragged, u), (c_out, lh.lh_linear_nvfp4_ragged_grad, u.transpose(1, 2))):
            x = torch.randn((n, k), device=DEV).to(dt)
            y = f(x, *dev, max_group_rows=int(counts.max()))
            for i in range(g):
                r = slice(int(off[i]), int(off[i + 1]))
                x64 = x[r].double()
                ref, mass = float(s[i]) * (x64 @ w[i].t()), float(s[i]) * (x64.abs() @ w[i].t().abs())
                tol = (8 * np.sqrt(k) * 2.0 ** -24 + 2.0 ** -23) * mass
                tol = tol + ulp * (ref.abs() + tol)
                assert bool(((y[r].double() - ref).abs() <= tol).all()), "group %d" % i

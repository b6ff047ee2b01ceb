"""Activations in 8 bits against the format's definition, value by value: the
shared power of two, the rounding to E4M3 (nearest, ties to even) and the way
back are exact operations, so everything is compared for equality."""
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


GRID = np.array([m * 2.0 ** -9 if e == 0 else 2.0 ** (e - 7) * (1 + m / 8) for e in range(16) for m in range(8)][:127])


def packed(x):
    """(codes, exponents + 127) of fp64 values by the definition."""
    rows, cols = x.shape
    codes = np.zeros((rows, cols), dtype=np.uint8)
    scales = np.zeros((rows, -(-cols // 32)), dtype=np.uint8)
    powers = 2.0 ** np.arange(-127.0, 128.0)
    mid = (GRID[1:] + GRID[:-1]) / 2
    for b in range(scales.shape[1]):
        part = x[:, 32 * b:32 * b + 32]
        most = np.where(np.isfinite(part), np.abs(part), 0).max(axis=1)
        k = np.searchsorted(448 * powers, most, side="left")
        q = np.abs(part) / powers[k][:, None]
        lo, hi = np.searchsorted(mid, q, side="left"), np.searchsorted(mid, q, side="right")
        c = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
        c = np.where(np.isfinite(part), c, 0x7f) + 128 * np.signbit(part)
        codes[:, 32 * b:32 * b + 32] = c
        scales[:, b] = k
    return codes, scales


def same(got, codes, scales):
    v, s = got[0].cpu().numpy(), got[1].cpu().numpy()
    assert np.array_equal(s, scales)
    nan = (codes & 0x7f) == 0x7f
    assert np.array_equal(v[~nan], codes[~nan]) and ((v[nan] & 0x7f) == 0x7f).all()


def back(codes, scales):
    mag = np.append(GRID, np.nan)[codes & 0x7f]
    return np.where(codes & 128, -mag, mag) * np.repeat(2.0 ** (scales.astype(np.float64) - 127), 32, axis=1)[:, :codes.shape[1]]


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 16), (3, 31), (2, 33), (7, 48), (5, 64), (4, 1000), (3, 1024), (2, 1025),
                                       (9, 2100), (300, 272)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_pack_and_unpack(lh, rows, cols, dt):
    rng = np.random.default_rng([rows, cols])
    x = rng.standard_normal((rows, cols)) * np.exp(3 * rng.standard_normal((rows, cols))) * np.exp(8 * rng.standard_normal((rows, 1)))
    x = torch.from_numpy(x.astype(np.float32)).to(dt)
    codes, scales = packed(x.double().numpy())
    got = lh.lh_checkpoint_pack(x.to(DEV))
    same(got, codes, scales)
    want = back(codes, scales)
    for out in (BF16, F32):
        y = lh.lh_checkpoint_unpack(*got, out_dtype=out)
        assert y.dtype == out and np.array_equal(y.double().cpu().numpy(), want)
    half = np.maximum(np.abs(x.double().numpy()) * 2.0 ** -4, np.repeat(2.0 ** (scales - 137.0), 32, axis=1)[:, :cols])
    assert (np.abs(want - x.double().numpy()) <= half).all()


def test_every_code(lh):
    """All 256 codes with all exponents, back to fp32 and bf16, and packed again where the block holds 448."""
    codes = torch.arange(256, dtype=torch.uint8).view(1, 256).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1).repeat(1, 8)
    y = lh.lh_checkpoint_unpack(codes.to(DEV), scales.to(DEV), out_dtype=F32)
    mag = np.append(GRID, np.nan)[codes.numpy() & 0x7f]
    with np.errstate(over="ignore"):
        want = (np.where(codes.numpy() & 128, -mag, mag) * 2.0 ** (np.arange(256)[:, None] - 127.0))
        want[255] = np.nan
        assert np.array_equal(y.double().cpu().numpy(), want.astype(np.float32).astype(np.float64), equal_nan=True)
        yb = lh.lh_checkpoint_unpack(codes.to(DEV), scales.to(DEV), out_dtype=BF16)
        assert torch.equal(torch.nan_to_num(yb, nan=7.0), torch.nan_to_num(y.to(BF16), nan=7.0))
    full = y[10:240].clone()
    full[:, ::32] = 448 * torch.exp2(torch.arange(10, 240, device=DEV).double() - 127).float()[:, None]
    got = lh.lh_checkpoint_pack(full)
    assert (got[1].cpu() == scales[10:240]).all()
    want = codes[10:240].clone()
    want[:, ::32] = 0x7e
    nan = (want & 0x7f) == 0x7f
    assert (got[0].cpu()[~nan] == want[~nan]).all() and ((got[0].cpu()[nan] & 0x7f) == 0x7f).all()


@pytest.mark.parametrize("dt", [BF16, F32])
def test_edges(lh, dt):
    """Zeros, subnormals, the largest numbers, maxima next to 1.75 * 2^k, infinities and NaN among others."""
    tiny, big = torch.finfo(dt).smallest_normal, torch.finfo(dt).max
    rows = [[0.0] * 40, [-0.0] * 40, [tiny / 4, tiny, -tiny * 3] + [0.0] * 37, [big, -big / 2, 1.0] + [0.0] * 37,
            [1.75, 1.0, 0.001] * 13 + [0.5], [1.75 * (1 + 2.0 ** -7), 1.0, 0.001] * 13 + [0.5], [448.0, 449.0, 3.0, 2.0 ** -9] * 10,
            [float("inf"), 1.0, -float("inf"), float("nan")] + [1.5] * 36, [float("nan")] * 40]
    x = torch.tensor(rows).to(dt)
    codes, scales = packed(x.double().numpy())
    same(lh.lh_checkpoint_pack(x.to(DEV)), codes, scales)
    got = lh.lh_checkpoint_unpack(*lh.lh_checkpoint_pack(x.to(DEV)), out_dtype=F32).cpu()
    assert torch.equal(torch.isnan(got), ~torch.isfinite(x))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_ties(lh, dt):
    """Midpoints of the grid go to the even code; beside them to the nearer one (bf16 holds the midpoints, fp32 their neighbours too)."""
    mid = (GRID[1:] + GRID[:-1]) / 2
    cols = [448.0] + mid[:31].tolist()
    x = np.array([[448.0] + mid[31 * i:31 * i + 31].tolist() + [0.0] * 31 for i in range(5)], dtype=object)
    x = np.array([list(r)[:32] for r in x], dtype=np.float64)
    assert len(cols) == 32
    if dt == F32:
        x = np.concatenate([x, x * (1 + 2.0 ** -20), x * (1 - 2.0 ** -20)])
    x[:, 0] = 448.0
    t = torch.from_numpy(x.astype(np.float32)).to(dt)
    codes, scales = packed(t.double().numpy())
    same(lh.lh_checkpoint_pack(torch.cat([t, -t]).to(DEV)), np.concatenate([codes, codes | 128]), np.concatenate([scales, scales]))


@pytest.mark.parametrize("dt", [BF16, F32])
def test_strides_and_alignment(lh, dt):
    rng = np.random.default_rng(2)
    for rows, cols, by, pad in ((5, 100, 1, 3), (3, 96, 3, 5), (4, 33, 0, 1), (6, 1, 0, 7)):
        wide = torch.full((rows * (cols + pad) + by,), 9.0, dtype=dt, device=DEV)
        v = wide[by:].view(rows, cols + pad)[:, :cols]
        v.copy_(torch.from_numpy(rng.standard_normal((rows, cols))).to(dt))
        codes, scales = packed(v.double().cpu().numpy())
        buf = torch.full((rows * cols + 8,), 7, dtype=torch.uint8, device=DEV)
        got = lh.lh_checkpoint_pack(v, values=buf[by:by + rows * cols].view(rows, cols))
        same(got, codes, scales)
        assert (buf[:by] == 7).all() and (buf[by + rows * cols:] == 7).all()
        v.fill_(0)
        assert lh.lh_checkpoint_unpack(*got, x=v) is v
        assert np.array_equal(v.double().cpu().numpy(), back(codes, scales))
        assert (wide == 9.0).sum() >= by + pad * (rows - 1)


def test_nothing_and_refusals(lh):
    x = torch.zeros(4, 40, device=DEV)
    v, s = lh.lh_checkpoint_pack(x[:0])
    assert v.shape == (0, 40) and s.shape == (0, 2) and lh.lh_checkpoint_unpack(v, s).shape == (0, 40)
    v, s = lh.lh_checkpoint_pack(x[:, :0])
    assert v.shape == (4, 0) and s.shape == (4, 0) and lh.lh_checkpoint_unpack(v, s).shape == (4, 0)
    v, s = lh.lh_checkpoint_pack(x)
    for f in (lambda: lh.lh_checkpoint_pack(x.t()), lambda: lh.lh_checkpoint_pack(x, values=v[:3]), lambda: lh.lh_checkpoint_pack(x, scales=s[:, :1]),
              lambda: lh.lh_checkpoint_unpack(v, s[:, :1].contiguous()), lambda: lh.lh_checkpoint_unpack(v[:, ::2], s),
              lambda: lh.lh_checkpoint_unpack(v, s, x=x[:3]), lambda: lh.lh_checkpoint_unpack(v, s.cpu())):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: lh.lh_checkpoint_pack(x.half()), lambda: lh.lh_checkpoint_unpack(v.int(), s),
              lambda: lh.lh_checkpoint_unpack(v, s, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            f()


def test_far_rows(lh):
    """Rows past 2^32 bytes."""
    x = torch.zeros((140000, 16384), dtype=BF16, device=DEV)
    x[-1] = torch.arange(16384, device=DEV).to(BF16)
    v, s = lh.lh_checkpoint_pack(x)
    codes, scales = packed(x[-1:].double().cpu().numpy())
    same((v[-1:], s[-1:]), codes, scales)
    assert (v[:-1] == 0).all()
    assert torch.equal(lh.lh_checkpoint_unpack(v, s)[-1].double().cpu(), torch.from_numpy(back(codes, scales)[0]))

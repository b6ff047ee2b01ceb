"""The adapters' tile kernels (many rows) at the sizes and segments where they can
go wrong: runs that begin and end inside a tile, several adapters a tile, rows of
no segment and of no adapter, ranks that fill no group of 16, odd widths, and the
one launch that takes many rows of a small rank both ways."""
import numpy as np
import pytest
import torch

from test_gpu_lora import BF16, DEV, F32, TYPES, check, expected, near, rand, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def runs(rng, rows, adapters):
    """Segments of 1 to 90 rows, empty ones among them, until the rows are used up but for a few."""
    cut, ids = [int(rng.integers(0, 3))], []
    while cut[-1] < rows - 5:
        cut.append(min(rows - 2, cut[-1] + int(rng.choice([0, 1, 3, 16, 17, 40, 64, 90]))))
        ids.append(int(rng.integers(-1, adapters)))
    return np.array(cut, dtype=np.int64), np.array(ids, dtype=np.int32)


@pytest.mark.parametrize("rank", [3, 16, 24, 40, 64, 100, 200])
@pytest.mark.parametrize("types", TYPES)
def test_runs(lh, rank, types):
    rng = np.random.default_rng([rank, 7])
    offsets, ids = runs(rng, 300, 3)
    # 300 rows of few long segments besides, so that the tiles are taken whatever the rank
    for c_in, c_out, off, who in ((200, 136, offsets, ids), (77, 101, np.array([0, 150, 299]), np.array([2, 0], dtype=np.int32))):
        check(lh, rng, 300, c_in, c_out, rank, 3, off, who, *types)


@pytest.mark.parametrize("rank,c_in,c_out", [(1, 64, 64), (5, 70, 130), (16, 264, 72), (12, 1000, 9)])
@pytest.mark.parametrize("ydt", [BF16, F32])
def test_both_ways_in_one_launch(lh, rank, c_in, c_out, ydt):
    rng = np.random.default_rng([rank, c_in])
    rows = 2085
    lengths = [0, 1, 15, 16, 17, 400, 3, 0, 700, 33, 31, 600]
    offsets = np.cumsum(lengths).astype(np.int64) + 2
    ids = np.array([1, 0, 2, -1, 1, 1, 0, 2, 7, 2, 0], dtype=np.int32)
    check(lh, rng, rows, c_in, c_out, rank, 3, offsets, ids, BF16, BF16, ydt)


@pytest.mark.parametrize("rank", [16, 64, 128])
def test_long_contractions(lh, rank):
    """Several workgroups a tile along the contraction, whose sums the second kernel adds."""
    rng = np.random.default_rng(rank)
    for types in ((BF16, BF16, BF16), (F32, F32, F32)):
        check(lh, rng, 290, 4100, 200, rank, 2, np.array([0, 100, 290]), np.array([1, 0], dtype=np.int32), *types)


@pytest.mark.parametrize("rows,rank", [(400, 16), (2100, 16), (400, 64)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_infinities_and_nan(lh, rows, rank, dt):
    """They stay in their row, and other adapters' never show."""
    rng = np.random.default_rng(rows)
    x, a, b = rand(rng, (rows, 80), dt), rand(rng, (2, rank, 80), dt), rand(rng, (2, rank, 70), dt)
    one = dict(adapter_ids=torch.ones(1, dtype=torch.int32, device=DEV))
    clean = lh.lh_lora(x.to(DEV), a.to(DEV), b.to(DEV), **one)
    x[1, 7], x[200, 79], x[rows - 1, 0] = float("inf"), float("nan"), -float("inf")
    a[0], b[0] = float("nan"), float("inf")
    y, s = lh.lh_lora(x.to(DEV), a.to(DEV), b.to(DEV), s=True, **one)
    assert torch.isinf(s[1]).all() and torch.isnan(s[200]).all() and torch.isinf(s[rows - 1]).all()
    others = [t for t in range(rows) if t not in (1, 200, rows - 1)]
    assert torch.equal(y[others], clean[others]) and not torch.isfinite(y[[1, 200, rows - 1]]).any()
    x1 = torch.ones(rows, 80, dtype=dt)
    x1[1, 7] = float("inf")
    y = lh.lh_lora(x1.to(DEV), a[1].abs().to(DEV), b[1].abs().to(DEV))
    assert (y[1] == float("inf")).all() and torch.isfinite(y[2:]).all()


def test_strides(lh):
    """Rows inside wider buffers at odd elements, in every kernel's sizes."""
    rng = np.random.default_rng(1)
    for rows, c_in, c_out, rank in ((300, 99, 77, 16), (2100, 99, 77, 16), (300, 99, 77, 64)):
        for dt in (BF16, F32):
            x, base = rand(rng, (rows, c_in), dt), rand(rng, (rows, c_out), dt)
            a, b = rand(rng, (2, rank, c_in), dt, 0.1), rand(rng, (2, rank, c_out), dt)
            offsets, ids = np.array([0, 130, rows]), np.array([1, 0], dtype=np.int32)
            s, st, y, yt = expected(x, a, b, [1.0, 1.0], base, rows_of(offsets, ids, rows, 2), dt, dt == BF16)
            wide = torch.full((rows, c_out + 5), 3.0, dtype=dt, device=DEV)
            xs = torch.full((rows, c_in + 3), float("nan"), dtype=dt, device=DEV)
            xs[:, 1:1 + c_in] = x.to(DEV)
            wide[:, 3:3 + c_out] = base.to(DEV)
            got = wide[:, 3:3 + c_out]
            lh.lh_lora(xs[:, 1:1 + c_in], a.to(DEV), b.to(DEV), base=got, y=got, offsets=torch.from_numpy(offsets).to(DEV),
                       adapter_ids=torch.from_numpy(ids).to(DEV))
            near(got, y, yt, "y")
            assert (wide[:, :3] == 3).all() and (wide[:, 3 + c_out:] == 3).all()


def test_overlapping_segments(lh):
    """Rows that several segments claim go to the first of them, in every kernel."""
    rng = np.random.default_rng(2)
    for rows, rank in ((40, 16), (400, 16), (2100, 16), (400, 64)):
        x, a, b = rand(rng, (rows, 64), BF16).to(DEV), rand(rng, (3, rank, 64), BF16).to(DEV), rand(rng, (3, rank, 48), BF16).to(DEV)
        off = torch.tensor([0, rows // 2, rows // 4, rows], device=DEV)     # the middle one is empty
        y = lh.lh_lora(x, a, b, offsets=off)
        clear = torch.tensor([0, rows // 2, rows], device=DEV)
        want = lh.lh_lora(x, a, b, offsets=clear, adapter_ids=torch.tensor([0, 2], device=DEV))
        assert torch.equal(y, want)

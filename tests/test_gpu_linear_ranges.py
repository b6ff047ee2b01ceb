"""Products with NVFP4 weights and their gradient at the ends of their ranges."""
import os
import sys

import numpy as np
import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_linear import units64, weights  # noqa: E402

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


# few, 16-, 32-, 64-, 128- and 256-token tiles, whole and ragged rows, parts and none
SIZES = [(1, 40, 272), (2, 40, 272), (5, 64, 272), (32, 8192, 2064), (40, 1000, 512), (700, 512, 256), (1500, 512, 528),
         (2100, 512, 1056), (4100, 1000, 272), (4100, 2048, 272)]


@pytest.mark.parametrize("t,c_out,c_in", SIZES)
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("workspace", [True, None])
def test_a_nan_reaches_every_output_of_its_token(lh, t, c_out, c_in, dt, workspace):
    print("case t=%d %dx%d %s ws=%s" % (t, c_out, c_in, dt, workspace), flush=True)
    rng = np.random.default_rng([61, t, c_in])
    packed, codes, s = weights(rng, 1, c_out, c_in)
    packed[0, 0, :] = 0                              # zero weights too: 0 x NaN is NaN
    dev = [v.to(DEV) for v in (packed, codes, s)]
    for n, f in ((c_in, lh.lh_linear_nvfp4), (c_out, lh.lh_linear_nvfp4_grad)):
        for bits in (0x7fc00000, -0x400000, 0x7f810000 if dt == BF16 else 0x7f800001):   # quiet, negative, signalling
            x = torch.from_numpy(rng.standard_normal((t, n)).astype(np.float32))
            rows = sorted({0, t // 2, t - 1})
            for r, col in zip(rows, (0, n - 1, n // 2)):
                x[r, col] = torch.tensor(bits, dtype=torch.int32).view(torch.float32)
            x = (x.view(torch.int32) >> 16).to(torch.int16).view(BF16) if dt == BF16 else x
            assert torch.isnan(x).any(1).nonzero().flatten().tolist() == rows
            y = f(x.to(DEV), *dev, out_dtype=F32, workspace=workspace).cpu()
            hit = torch.zeros(t, dtype=torch.bool)
            hit[rows] = True
            assert bool(torch.isnan(y[hit]).all()) and bool(torch.isfinite(y[~hit]).all())


@pytest.mark.parametrize("t,c_out,c_in", [(1, 300, 512), (2, 300, 512), (8, 512, 512), (40, 512, 512), (200, 512, 512),
                                          (600, 512, 512), (2100, 512, 512)])
@pytest.mark.parametrize("e", [-105, -112, -120, -127])
def test_tiny_activations(lh, t, c_out, c_in, e):
    """bf16 ones are exact down to the subnormal numbers.  Of fp32 ones below
    2^-110 what lies under 2^-133, the last place of a subnormal bf16, can be
    lost: less than 2^-133 |u| per product.  Besides, sums of n exact terms in
    fp32: 8 sqrt(n) 2^-24 of the terms' magnitudes (the probabilistic bound),
    two roundings for the scale, one for the output, and one half of the last
    place of a subnormal sum (2^-150) per addition."""
    rng = np.random.default_rng([67, t, e + 200])
    packed, _, _ = weights(rng, 1, c_out, c_in)
    codes = torch.from_numpy(rng.integers(0x60, 0x78, (1, c_out, c_in // 16), dtype=np.uint8))
    u = torch.from_numpy(units64(packed, codes)[0]).to(DEV)
    dev = [v.to(DEV) for v in (packed, codes, torch.full((1,), 2.0 ** 100))]
    for dt in (BF16, F32):
        for n, w, f in ((c_in, u, lh.lh_linear_nvfp4), (c_out, u.t().contiguous(), lh.lh_linear_nvfp4_grad)):
            x = torch.from_numpy(rng.standard_normal((t, n)) * 2.0 ** e).to(dt).to(DEV)
            ref, mass = x.double() @ w.t(), x.double().abs() @ w.abs().t()
            tol = (8 * n ** 0.5 * 2.0 ** -24 + 2.0 ** -22) * mass + 3 * n * 2.0 ** -150
            if dt == F32:
                tol = tol + 2.0 ** -133 * w.abs().sum(1)
            for workspace in (True, None):
                y = f(x, *dev, out_dtype=F32, workspace=workspace).double() / 2.0 ** 100
                assert bool(((y - ref).abs() <= tol).all()), "%s: worst %.3g of its tolerance" % (
                    dt, ((y - ref).abs() / tol).max().item())


def test_rows_to_pack_beyond_one_grid_dimension(lh):
    """(2^23 + 16) rows of 4112 bf16 are packed by more than 2^32 threads."""
    t, c_out, c_in = (1 << 23) + 16, 16, 4112
    if torch.cuda.mem_get_info()[0] < 180 << 30:
        pytest.skip("needs 145 GB of device memory")
    rng = np.random.default_rng(71)
    packed, codes, s = weights(rng, 1, c_out, c_in)
    u = torch.from_numpy(units64(packed, codes)[0])
    x = torch.zeros((t, c_in), dtype=BF16, device=DEV)
    rows = torch.tensor([0, 200000, 300001, t // 2, t - 70, t - 1])
    some = torch.from_numpy(rng.integers(-4, 5, (len(rows), c_in)).astype(np.float32)).to(BF16)
    x[rows.to(DEV)] = some.to(DEV)
    ones = torch.ones(1, device=DEV)
    y = lh.lh_linear_nvfp4(x, packed.to(DEV), codes.to(DEV), ones, out_dtype=F32)
    del x
    want, mass = some.double() @ u.t(), some.double().abs() @ u.abs().t()
    got = y[rows.to(DEV)].double().cpu()
    assert bool(((got - want).abs() <= 8 * c_in ** 0.5 * 2.0 ** -24 * mass).all())
    y[rows.to(DEV)] = 0.0
    assert not bool(y.any())

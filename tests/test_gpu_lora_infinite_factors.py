"""Infinities and NaN in the factors of adapters in use follow the formula, in the
kernels of few rows and of many alike.  s and the products are small whole numbers,
exact in every type, so that signs and zeros are the formula's; finite outputs are
whole numbers too, off by their own rounding alone (2^-8 for bf16)."""
import numpy as np
import pytest
import torch

from test_gpu_lora import BF16, DEV, F32, TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def follows(got, want, ydt):
    got = got.double().cpu().numpy()
    for what, p in (("NaN", np.isnan), ("infinity", np.isposinf), ("negative infinity", np.isneginf)):
        bad = p(got) != p(want)
        assert not bad.any(), "%s: %d of %d, at %s" % (what, bad.sum(), bad.size, np.argwhere(bad)[0])
    fine = np.isfinite(want)
    assert (np.abs(got[fine] - want[fine]) <= (2.0 ** -8 if ydt == BF16 else 0) * np.abs(want[fine])).all()


@pytest.mark.parametrize("rows,rank,k,m", [(5, 16, 24, 40), (400, 16, 72, 136), (400, 64, 40, 101), (400, 200, 40, 72), (2100, 16, 40, 72),
                                          (2100, 9, 40, 101)])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("grad", [False, True])
def test_factors(lh, rows, rank, k, m, types, grad):
    xdt, wdt, ydt = types
    rng = np.random.default_rng([rows, rank, grad])
    inf, nan = float("inf"), float("nan")
    x = rng.integers(-1, 2, (rows, k)).astype(np.float64)
    x[rng.random(rows) < 0.2] = 0
    inner, outer = rng.integers(-1, 2, (3, rank, k)).astype(np.float64), rng.integers(-3, 4, (3, rank, m)).astype(np.float64)
    outer[1, rank // 2, 3], outer[1, 0, 5], outer[1, rank - 1, m - 1] = inf, -inf, inf
    outer[1, 1, 7], outer[1, 2, 7], outer[1, 1, 9] = inf, -inf, nan
    outer[0, 1, 11], outer[0, :, 12] = -inf, inf
    inner[2, 3, 2], outer[2, :, :9] = inf, rng.integers(1, 4, (rank, 9))   # s is infinite, or NaN where x is zero there
    outer[2, 3, 4] = inf
    base = rng.integers(-9, 10, (rows, m)).astype(np.float64)
    offsets = np.array([0, rows // 4, rows // 2, 3 * rows // 4, rows])
    ids = np.array([1, 0, 2, 1])
    scale = np.array([2.0, 0.5, 1.0])
    want = base.copy()
    with np.errstate(invalid="ignore"):
        for t in range(rows):
            g = ids[np.searchsorted(offsets, t, side="right") - 1]
            s = (inner[g] * x[t]).sum(axis=1)
            want[t] += scale[g] * (s[:, None] * outer[g]).sum(axis=0)

    def dev(v, dt):
        return torch.from_numpy(v.astype(np.float32)).to(dt).to(DEV)

    a, b = (outer, inner) if grad else (inner, outer)
    f = lh.lh_lora_grad if grad else lh.lh_lora
    y = f(dev(x, xdt), dev(a, wdt), dev(b, wdt), dev(scale, F32), base=dev(base, ydt), out_dtype=ydt,
          offsets=torch.from_numpy(offsets).to(DEV), adapter_ids=torch.from_numpy(ids).to(DEV))
    assert np.isposinf(want).any() and np.isnan(want).any() and np.isfinite(want).any()
    follows(y, want, ydt)

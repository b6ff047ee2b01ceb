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

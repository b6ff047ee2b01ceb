"""Tensors whose strides mean nothing (no elements, or one column) are taken as
torch takes them: contiguous."""
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


def empty(*shape):
    """Without elements and with strides of zero, as numpy's empty arrays come."""
    t = torch.from_numpy(np.zeros(shape, dtype=np.float32)).to(DEV)
    return t.as_strided(shape, (0,) * len(shape))


def test_no_elements(lh):
    packed = torch.zeros((1, 32, 32), dtype=torch.uint8, device=DEV)
    codes = torch.ones((1, 32, 4), dtype=torch.uint8, device=DEV)
    s = torch.ones(1, device=DEV)
    off = torch.zeros(2, dtype=torch.int64, device=DEV)
    assert lh.lh_linear_nvfp4(empty(0, 64), packed, codes, s).shape == (0, 32)
    assert lh.lh_linear_nvfp4(empty(1, 0, 64), packed, codes, s, y=empty(1, 0, 32)).shape == (1, 0, 32)
    assert lh.lh_linear_nvfp4(empty(0, 5, 64), packed[:0], codes[:0], s[:0]).shape == (0, 5, 32)
    assert lh.lh_linear_nvfp4_grad(empty(0, 32), packed, codes, s).shape == (0, 64)
    assert lh.lh_linear_nvfp4_ragged(empty(0, 64), off, packed, codes, s).shape == (0, 32)
    assert lh.lh_linear_nvfp4_ragged_grad(empty(0, 32), off, packed, codes, s).shape == (0, 64)
    assert lh.lh_quantize_nvfp4(empty(0, 64), s)["values"].shape == (1, 0, 64)
    assert lh.lh_quantize_nvfp4(empty(0, 5, 64), s[:0])["values"].shape == (0, 5, 64)
    position = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    assert lh.lh_moe_dispatch(empty(0, 8), position, xs=empty(0, 8)).shape == (0, 8)
    assert lh.lh_moe_combine(empty(0, 8), position, y=empty(0, 8)).shape == (0, 8)
    assert [v.shape for v in lh.lh_moe_combine_grad(empty(0, 8), empty(0, 8), position)] == [(0, 8), (0, 2)]


@pytest.mark.parametrize("dt", [BF16, F32])
def test_one_column(lh, dt):
    """[n, 1] as the transpose of a row: its column stride is n."""
    n = 5
    col = torch.arange(1.0, n + 1, device=DEV).to(dt).view(1, n).t()
    assert col.stride(1) != 1 and col.is_contiguous()
    packed = torch.full((1, 1, 8), 0x22, dtype=torch.uint8, device=DEV)      # one output of sixteen weights 1
    codes = torch.full((1, 1, 1), 0x38, dtype=torch.uint8, device=DEV)       # scale 1
    s = torch.ones(1, device=DEV)
    assert torch.equal(lh.lh_linear_nvfp4_grad(col, packed, codes, s), col.expand(n, 16))
    y = torch.empty((1, n), dtype=dt, device=DEV).t()
    assert torch.equal(lh.lh_linear_nvfp4(col.expand(n, 16).contiguous(), packed, codes, s, y=y), 16 * col)
    position = torch.arange(n, dtype=torch.int32, device=DEV).view(n, 1)
    xs = lh.lh_moe_dispatch(col, position, xs=torch.empty((1, n), dtype=dt, device=DEV).t())
    assert torch.equal(xs, col) and torch.equal(lh.lh_moe_combine(xs, position), col)
    dys, dw = lh.lh_moe_combine_grad(col, xs, position)
    assert torch.equal(dys, col) and torch.equal(dw, col.float() ** 2)

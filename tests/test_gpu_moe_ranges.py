"""Routing at the ends of its ranges: buffers with more rows than assignments,
rows without columns, and more tokens than one grid dimension takes.  Rows are
moved, weighted by powers of two and dotted with small whole numbers, so every
result is exact."""
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


def leave_behind(shape, dtype):
    """The next allocation of this size finds NaN."""
    t = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
    torch.cuda.synchronize()
    del t


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("t,k,more", [(5, 2, 3), (64, 8, 512), (3, 0, 7), (0, 2, 4)])
def test_rows_without_an_assignment_have_no_gradient(lh, t, k, more, dt):
    print("case t=%d k=%d more=%d %s" % (t, k, more, dt), flush=True)
    rng = np.random.default_rng([t, k, more])
    c, n = 72, t * k
    position = torch.from_numpy(rng.permutation(n + more)[:n].astype(np.int32).reshape(t, k))
    dy = torch.from_numpy(rng.integers(-8, 9, (t, c)).astype(np.float32)).to(dt)
    ys = torch.from_numpy(rng.integers(-8, 9, (n + more, c)).astype(np.float32)).to(dt)
    w = torch.from_numpy(2.0 ** rng.integers(-3, 3, (t, k))).float()
    want = torch.zeros((n + more, c), dtype=dt)
    want[position.reshape(-1).long()] = (w.unsqueeze(-1) * dy.float().unsqueeze(1)).to(dt).reshape(n, c)
    leave_behind((n + more, c), dt)
    dys, dw = lh.lh_moe_combine_grad(dy.to(DEV), ys.to(DEV), position.to(DEV), w.to(DEV))
    assert torch.equal(dys.cpu(), want)
    assert torch.equal(dw.cpu(), (dy.float().unsqueeze(1) * ys[position.long()].float()).sum(-1))
    # a buffer of the caller's keeps what no assignment names
    mine = torch.full((n + more, c), 7.0, dtype=dt, device=DEV)
    lh.lh_moe_combine_grad(dy.to(DEV), ys.to(DEV), position.to(DEV), w.to(DEV), dys=mine)
    named = torch.zeros(n + more, dtype=torch.bool)
    named[position.reshape(-1).long()] = True
    assert torch.equal(mine.cpu()[named], want[named]) and bool((mine.cpu()[~named] == 7.0).all())


def test_rows_without_columns(lh):
    position = torch.tensor([[1, 0], [-4, 2]], dtype=torch.int32, device=DEV)
    leave_behind((2, 2), F32)
    dys, dw = lh.lh_moe_combine_grad(torch.empty((2, 0), device=DEV), torch.empty((4, 0), device=DEV), position)
    assert dys.shape == (4, 0) and dw.tolist() == [[0, 0], [0, 0]]
    assert lh.lh_moe_dispatch(torch.empty((2, 0), device=DEV), position).shape == (4, 0)
    assert lh.lh_moe_combine(torch.empty((4, 0), device=DEV), position).shape == (2, 0)

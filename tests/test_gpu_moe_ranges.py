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


def some(gen, rows, cols):
    return torch.randint(-8, 9, (rows, cols), generator=gen, device=DEV, dtype=torch.int8).to(BF16)


def test_gradients_of_many_tokens(lh):
    """One workgroup per token: 2^24 of them are 2^32 threads."""
    t, c = (1 << 24) + 3, 8
    gen = torch.Generator(device=DEV).manual_seed(1)
    position = torch.randperm(t, generator=gen, device=DEV).to(torch.int32).view(t, 1)
    dy, ys = some(gen, t, c), some(gen, t, c)
    w = torch.exp2(torch.randint(-3, 3, (t, 1), generator=gen, device=DEV).float())
    dys, dw = lh.lh_moe_combine_grad(dy, ys, position, w)
    at = position.view(-1).long()
    assert torch.equal(dys[at], (w * dy.float()).to(BF16))
    assert torch.equal(dw.view(-1), (dy.float() * ys[at].float()).sum(-1))


def test_rows_of_many_tokens(lh):
    """One wave per token: 2^26 of them are 2^32 threads.  (torch's own indexing
    of that many rows returns the first few alone: slices here.)"""
    t, c = (1 << 26) + 3, 8
    gen = torch.Generator(device=DEV).manual_seed(2)
    position = torch.randperm(t, generator=gen, device=DEV).to(torch.int32).view(t, 1)
    x = some(gen, t, c)
    xs = lh.lh_moe_dispatch(x, position)
    for i in range(0, t, 1 << 22):
        at = position[i:i + (1 << 22), 0]
        assert torch.equal(xs.index_select(0, at), x[i:i + (1 << 22)]), "rows from token %d on" % i
    y = lh.lh_moe_combine(xs, position)
    for i in range(0, t, 1 << 22):
        assert torch.equal(y[i:i + (1 << 22)], x[i:i + (1 << 22)]), "tokens from %d on" % i

"""Tokens sorted by expert and back, against plain loops in 64 bits.

Tolerances: rows that are only moved are exact; a sum of k products in fp32
is off by at most (k + 1) 2^-24 sum |terms| (every partial sum rounded once,
products fused), a product by half an ulp of its type, and a dot of n columns
by 8 sqrt(n) 2^-24 sum |terms| (the probabilistic bound, lambda = 8)."""
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


def sort64(ids, n_groups):
    flat = ids.reshape(-1)
    live = (flat >= 0) & (flat < n_groups)
    walk = np.array([a for g in range(n_groups) for a in np.nonzero(flat == g)[0]] if n_groups < 80 else
                    np.argsort(np.where(live, flat, n_groups), kind="stable")[:live.sum()], dtype=np.int64)
    dropped = np.nonzero(~live)[0]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[live], minlength=n_groups)[:n_groups])])
    order = np.concatenate([walk, -1 - dropped])
    position = np.empty(flat.size, dtype=np.int64)
    position[walk] = np.arange(len(walk))
    position[dropped] = -1 - np.arange(len(walk), flat.size)
    return offsets, order, position.reshape(ids.shape)


def make_ids(rng, t, k, n_groups, drop=0.1, skew=True):
    p = rng.dirichlet(np.full(n_groups, 0.3)) if skew and n_groups > 1 else np.full(n_groups, 1 / n_groups)
    ids = rng.choice(n_groups, (t, k), p=p)
    bad = rng.random((t, k)) < drop
    ids[bad] = rng.choice([-1, n_groups, -7, n_groups + 3], (t, k))[bad]
    return ids


@pytest.mark.parametrize("t,k,e", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (16, 8, 64), (64, 1, 2), (100, 7, 33), (511, 4, 1024),
                                   (1024, 2, 512), (1025, 8, 64), (4096, 8, 64), (5000, 5, 1000), (200000, 6, 17)])
@pytest.mark.parametrize("dt", [torch.int32, torch.int64])
def test_sort(lh, t, k, e, dt):
    print("case t=%d k=%d e=%d %s" % (t, k, e, dt), flush=True)
    rng = np.random.default_rng([t, k, e])
    for drop in (0.0, 0.2, 1.0):
        ids = make_ids(rng, t, k, e, drop)
        offsets, order, position = sort64(ids, e)
        got = lh.lh_moe_sort(torch.from_numpy(ids).to(dt).to(DEV), e)
        assert np.array_equal(got["offsets"].cpu().numpy(), offsets)
        assert np.array_equal(got["order"].cpu().numpy(), order)
        assert np.array_equal(got["position"].cpu().numpy(), position)


def test_sort_of_large_ids_and_nothing(lh):
    ids = torch.tensor([[2 ** 40, 1], [0, -2 ** 40]], dtype=torch.int64, device=DEV)
    got = lh.lh_moe_sort(ids, 3)
    assert got["offsets"].tolist() == [0, 1, 2, 2] and got["position"].tolist() == [[-3, 1], [0, -4]]
    for shape in ((0, 4), (5, 0)):
        got = lh.lh_moe_sort(torch.empty(shape, dtype=torch.int32, device=DEV), 3)
        assert got["offsets"].tolist() == [0, 0, 0, 0] and got["position"].shape == shape
    got = lh.lh_moe_sort(torch.zeros((2, 2), dtype=torch.int32, device=DEV), 0)
    assert got["offsets"].tolist() == [0] and got["position"].tolist() == [[-1, -2], [-3, -4]]


CASES = [(1, 1, 1, 8), (3, 2, 4, 1), (16, 8, 64, 2048), (7, 3, 5, 100), (50, 4, 16, 515), (33, 5, 8, 1030), (200, 2, 9, 64),
         (9, 12, 20, 4100)]


@pytest.mark.parametrize("t,k,e,c", CASES)
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_there_and_back_with_gradients(lh, t, k, e, c, dt, drop):
    print("case t=%d k=%d e=%d c=%d %s drop=%g" % (t, k, e, c, dt, drop), flush=True)
    rng = np.random.default_rng([t, k, e, c])
    ids = make_ids(rng, t, k, e, drop)
    _, _, pos = sort64(ids, e)
    n = t * k
    x, dy = [torch.from_numpy(rng.standard_normal((t, c)).astype(np.float32)).to(dt) for _ in range(2)]
    ys = torch.from_numpy(rng.standard_normal((n, c)).astype(np.float32)).to(dt)
    w = torch.from_numpy(rng.random((t, k)).astype(np.float32))
    position = lh.lh_moe_sort(torch.from_numpy(ids).to(DEV), e)["position"]
    ulp = 2.0 ** -8 if dt == BF16 else 2.0 ** -24

    xs = lh.lh_moe_dispatch(x.to(DEV), position, xs=torch.full((n, c), 7.0, dtype=dt, device=DEV)).cpu()
    want = torch.zeros((n, c), dtype=dt)
    for i in range(t):
        for j in range(k):
            if pos[i, j] >= 0:
                want[pos[i, j]] = x[i]
    assert torch.equal(xs, want)

    x64, dy64, ys64, w64 = (v.double().numpy() for v in (x, dy, ys, w))
    for weights in (w, None):
        y = lh.lh_moe_combine(ys.to(DEV), position, None if weights is None else weights.to(DEV))
        dys, dw = lh.lh_moe_combine_grad(dy.to(DEV), ys.to(DEV), position, None if weights is None else weights.to(DEV),
                                         dys=torch.full((n, c), 7.0, dtype=dt, device=DEV))
        ref, mass = np.zeros((t, c)), np.zeros((t, c))
        rdys = np.zeros((n, c))
        rdw, mdw = np.zeros((t, k)), np.zeros((t, k))
        for i in range(t):
            for j in range(k):
                p, wij = pos[i, j], w64[i, j] if weights is not None else 1.0
                if p < 0:
                    continue
                ref[i] += wij * ys64[p]
                mass[i] += np.abs(wij * ys64[p])
                rdys[p] = wij * dy64[i]
                rdw[i, j] = dy64[i] @ ys64[p]
                mdw[i, j] = np.abs(dy64[i]) @ np.abs(ys64[p])
        tol = (k + 1) * 2.0 ** -24 * mass
        assert (np.abs(y.double().cpu().numpy() - ref) <= tol + ulp * (np.abs(ref) + tol)).all()
        tol = 2.0 ** -24 * np.abs(rdys)
        assert (np.abs(dys.double().cpu().numpy() - rdys) <= tol + ulp * (np.abs(rdys) + tol)).all()
        assert (np.abs(dw.double().cpu().numpy() - rdw) <= 8 * np.sqrt(c) * 2.0 ** -24 * mdw + 1e-37).all()
    assert lh.lh_moe_combine_grad(dy.to(DEV), ys.to(DEV), position, w.to(DEV), dys=False)[0] is None
    only = lh.lh_moe_combine_grad(dy.to(DEV), ys.to(DEV), position, w.to(DEV), dweights=False)
    assert only[1] is None


def test_gradients_against_differences(lh):
    """L = sum(dy * combine(dispatch(x) * 1, w)): difference quotients in the
    weights and in the rows (the map is bilinear, so they have no step error
    beyond fp32 rounding)."""
    rng = np.random.default_rng(3)
    t, k, e, c = 5, 3, 4, 40
    ids = make_ids(rng, t, k, e, 0.2)
    position = lh.lh_moe_sort(torch.from_numpy(ids).to(DEV), e)["position"]
    ys, w, dy = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV) for s in ((t * k, c), (t, k), (t, c)))
    dys, dw = lh.lh_moe_combine_grad(dy, ys, position, w)

    def loss(ys, w):
        return (lh.lh_moe_combine(ys, position, w).double() * dy.double()).sum().item()

    base = loss(ys, w)
    mass = (dy.double().abs().sum() * ys.double().abs().max() * w.double().abs().max() * k).item()
    tol = 2 * (k + 2) * 2.0 ** -24 * mass / 8.0 + 1e-5
    for i in range(t):
        for j in range(k):
            up = w.clone()
            up[i, j] += 8.0
            assert abs((loss(ys, up) - base) / 8.0 - dw[i, j].item()) <= tol * 8
    for p, q in ((0, 0), (3, 39), (14, 7), (9, 20)):
        up = ys.clone()
        up[p, q] += 8.0
        assert abs((loss(up, w) - base) / 8.0 - dys[p, q].item()) <= tol * 8
    # dispatch's gradient is combine without weights: <dxs, dispatch(v)> = <combine(dxs), v>
    v, dxs = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV) for s in ((t, c), (t * k, c)))
    lhs = (dxs.double() * lh.lh_moe_dispatch(v, position).double()).sum()
    rhs = (lh.lh_moe_combine(dxs, position).double() * v.double()).sum()
    assert abs(lhs - rhs) <= (k + 1) * 2.0 ** -24 * (dxs.double().abs().sum() * v.double().abs().max())


def test_strides_and_surroundings(lh):
    rng = np.random.default_rng(5)
    t, k, e, c = 11, 2, 3, 77
    position = lh.lh_moe_sort(torch.from_numpy(make_ids(rng, t, k, e, 0.2)).to(DEV), e)["position"]
    for dt in (BF16, F32):
        big = torch.randn((t + 2, c + 9), device=DEV).to(dt)
        x = big[1:t + 1, 3:3 + c]
        rows = torch.full((t * k + 4, c + 5), 7.0, dtype=dt, device=DEV)
        xs = lh.lh_moe_dispatch(x, position, xs=rows[1:1 + t * k, 1:1 + c])
        assert torch.equal(xs, lh.lh_moe_dispatch(x.contiguous(), position))
        y = lh.lh_moe_combine(xs, position, y=torch.full((t + 1, c + 3), 7.0, dtype=dt, device=DEV)[:t, 2:2 + c])
        assert torch.equal(y, lh.lh_moe_combine(xs.contiguous(), position))
        keep = rows.clone()
        keep[1:1 + t * k, 1:1 + c] = 7.0
        assert bool((keep == 7.0).all())


def test_positions_outside_the_buffer_are_ignored(lh):
    position = torch.tensor([[0, 10 ** 6], [-(10 ** 6), 1]], dtype=torch.int32, device=DEV)
    x = torch.tensor([[1.0, 2.0], [3.0, 4.0]], device=DEV)
    xs = lh.lh_moe_dispatch(x, position, xs=torch.full((4, 2), 7.0, device=DEV))
    assert xs.tolist() == [[1, 2], [3, 4], [7, 7], [7, 7]]
    assert lh.lh_moe_combine(xs, position).tolist() == [[1, 2], [3, 4]]
    dys, dw = lh.lh_moe_combine_grad(x, xs, position, dys=torch.full((4, 2), 7.0, device=DEV))
    assert dys.tolist() == [[1, 2], [3, 4], [7, 7], [7, 7]] and dw.tolist() == [[5, 0], [0, 25]]


def test_empty(lh):
    z = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    assert lh.lh_moe_dispatch(torch.empty((0, 8), device=DEV), z).shape == (0, 8)
    assert lh.lh_moe_combine(torch.empty((0, 8), device=DEV), z).shape == (0, 8)
    none = torch.empty((3, 0), dtype=torch.int32, device=DEV)
    y = lh.lh_moe_combine(torch.empty((0, 8), device=DEV), none, y=torch.full((3, 8), 7.0, device=DEV))
    assert bool((y == 0).all())                       # tokens without any expert


def test_refusals(lh):
    ids = torch.zeros((4, 2), dtype=torch.int64, device=DEV)
    pos = lh.lh_moe_sort(ids, 3)["position"]
    x = torch.zeros((4, 8), device=DEV)
    with pytest.raises(TypeError):
        lh.lh_moe_sort(ids.float(), 3)
    with pytest.raises(ValueError):
        lh.lh_moe_sort(ids.cpu(), 3)
    with pytest.raises(ValueError):
        lh.lh_moe_sort(ids.t(), 3)
    with pytest.raises(lh.LHError):
        lh.lh_moe_sort(ids, 1025)
    with pytest.raises(ValueError):
        lh.lh_moe_dispatch(x[:3], pos)
    with pytest.raises(lh.LHError):
        lh.lh_moe_dispatch(x, pos, xs=torch.zeros((7, 8), device=DEV))
    with pytest.raises(TypeError):
        lh.lh_moe_dispatch(x, pos.long())
    with pytest.raises(TypeError):
        lh.lh_moe_dispatch(x.half(), pos)
    with pytest.raises(ValueError):
        lh.lh_moe_combine(x, pos, torch.ones((4, 3), device=DEV))
    with pytest.raises(TypeError):
        lh.lh_moe_combine_grad(x, torch.zeros((8, 8), dtype=BF16, device=DEV), pos)

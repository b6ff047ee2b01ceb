"""Offsets that decrease somewhere make segments overlap: a row is then the first
segment's that has it, in the product and in all gradients alike.  Tolerances as
in test_gpu_lora.py."""
import numpy as np
import pytest
import torch

from test_gpu_lora import BF16, DEV, F32, U, expected, f64, near, rand, wanted

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


def first_claims(offsets, ids, n_rows, n_adapters):
    """Each row's adapter: -1 none, -2 in no segment; the first segment that has the row says which."""
    g = np.full(n_rows, -2)
    for i in range(len(offsets) - 1):
        lo, hi = max(int(offsets[i]), 0), min(int(offsets[i + 1]), n_rows)
        part = g[lo:max(lo, hi)]
        part[part == -2] = int(ids[i]) if 0 <= ids[i] < n_adapters else -1
    return g


def lists(rows):
    rng = np.random.default_rng(rows)
    half, third = rows // 2, rows // 3
    yield "halves", [0, half, third, rows]
    yield "a hole inside a later segment", [third, half, 0, rows, 0]
    yield "holes within holes", [half, half + 9, third, third + 5, 3, 11, 0, rows - 1, 0, rows]
    yield "all rows again and again", [0, rows] * 20 + [0]
    yield "backwards", list(range(rows - 1, 0, -7))
    yield "backwards by pairs", [v for k in range(rows - 8, 0, -8) for v in (k, k + 5)] + [0, rows]
    yield "outside the rows", [-5, rows + 9, 4, half, -(1 << 40), third, 1 << 40, 7]
    yield "any", rng.integers(-9, rows + 9, 50).tolist()
    yield "many", rng.integers(0, rows + 1, 700).tolist()
    yield "many ups and downs", (np.arange(900) * rows // 900 + rng.integers(-20, 20, 900)).tolist()


@pytest.mark.parametrize("rows,adapters", [(60, 3), (333, 40), (1500, 5), (2600, 700)])
def test_all_calls_agree(lh, rows, adapters):
    rng = np.random.default_rng([rows, adapters])
    rank, c_in, c_out = 12, 72, 40
    x, dy = rand(rng, (rows, c_in), BF16), rand(rng, (rows, c_out), BF16)
    s, ds = rand(rng, (rows, rank), F32), rand(rng, (rows, rank), F32)
    a, b = rand(rng, (adapters, rank, c_in), BF16, c_in ** -0.5), rand(rng, (adapters, rank, c_out), BF16, 0.3)
    scale = rng.uniform(0.25, 2, adapters).astype(np.float32)
    old = [rand(rng, (adapters, rank, c), F32) for c in (c_in, c_out)]
    for name, offsets in lists(rows):
        print("case", rows, adapters, name, flush=True)
        offsets = np.array(offsets, dtype=np.int64)
        ids = rng.integers(-1, adapters, len(offsets) - 1).astype(np.int32)
        g = first_claims(offsets, ids, rows, adapters)
        kw = dict(scale=torch.from_numpy(scale).to(DEV), offsets=torch.from_numpy(offsets).to(DEV), adapter_ids=torch.from_numpy(ids).to(DEV))
        want_s, st, want_y, yt = expected(x, a, b, scale, None, g, BF16, False)
        y, got_s = lh.lh_lora(x.to(DEV), a.to(DEV), b.to(DEV), s=True, **kw)
        near(got_s[g > -2], want_s[g > -2], st[g > -2], "s")
        near(y[g > -2], want_y[g > -2], yt[g > -2], "y")
        nbytes = lh.lh_lora_weight_grad_workspace_bytes(rows, len(ids), adapters, rank, c_in, c_out)
        ws = torch.full((nbytes + 4096,), 0xff, dtype=torch.uint8, device=DEV)   # NaN to whoever reads what was not written
        out = [torch.full_like(o, float("nan")).to(DEV) for o in old]
        lh.lh_lora_weight_grad(x.to(DEV), dy.to(DEV), s.to(DEV), ds.to(DEV), adapters, da=out[0], db=out[1],
                               workspace=ws[:nbytes] if nbytes else None, **kw)
        added = [o.to(DEV) for o in old]
        lh.lh_lora_weight_grad(x.to(DEV), dy.to(DEV), s.to(DEV), ds.to(DEV), adapters, da=added[0], db=added[1], beta=0.5, **kw)
        assert (ws[nbytes:] == 0xff).all()
        for k, (p, v) in enumerate(((ds, x), (s, dy))):
            want, tol = wanted(p, v, scale, g, adapters)
            near(out[k], want, tol + U * (np.abs(want) + tol) + 1e-37, "da db"[3 * k:3 * k + 2])
            want, tol = wanted(p, v, scale, g, adapters, f64(old[k]), 0.5)
            near(added[k], want, tol + U * (np.abs(want) + tol) + 1e-37, "added to")


def test_the_same_bits_as_without_the_overlap(lh):
    rng = np.random.default_rng(1)
    for rows in (400, 3000):
        x, dy, p = rand(rng, (rows, 64), BF16).to(DEV), rand(rng, (rows, 48), BF16).to(DEV), rand(rng, (rows, 16), F32).to(DEV)
        over = torch.tensor([0, rows // 2, rows // 4, rows], device=DEV)
        clear = torch.tensor([0, rows // 2, rows], device=DEV)
        got = lh.lh_lora_weight_grad(x, dy, p, p, 3, offsets=over)
        want = lh.lh_lora_weight_grad(x, dy, p, p, 3, offsets=clear, adapter_ids=torch.tensor([0, 2], device=DEV))
        assert all(torch.equal(u, v) for u, v in zip(got, want))

"""Adapters beside a frozen projection as training and serving run them: the
product, the adapters, the rows in 8 bits, and all gradients together against
64 bits; captured in a graph; on another stream; the example's layer with an
adapter for every expert."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lh():
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import nvfp4_scale_calibration_amd as m
    return m


@pytest.fixture(scope="module")
def layer_example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_layer
    return moe_layer


def projection(lh, rng, c_out, c_in):
    w = torch.from_numpy((0.02 * rng.standard_normal((1, c_out, c_in))).astype(np.float32)).to(DEV)
    amax = lh.lh_absmax(w)
    idx, _, _ = lh.lh_select_scales(lh.LH_RULE_MAX, w, None, amax, best_err=False, best_amax=False)
    return lh.lh_fake_quant_nvfp4(w, idx, amax, packed=True, scale_e4m3=True, global_scale=True)


def rand(rng, *shape, dtype=BF16, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(dtype).to(DEV)


def step(lh, q, x, dy, a, b, scale, kw, ws=None):
    """One training step's calls; ws: the workspaces (adapters, adapters' gradient)."""
    w = (q["packed"], q["scale_e4m3"], q["global_scale"])
    wl = {} if ws is None else dict(workspace=ws[0])
    wg = {} if ws is None else dict(workspace=ws[1])
    wn = {} if ws is None else dict(workspace=None)
    y = lh.lh_linear_nvfp4(x, *w, **wn)
    y, s = lh.lh_lora(x, a, b, scale, base=y, y=y, s=True, **kw, **wl)
    values, scales = lh.lh_checkpoint_pack(x)
    dx = lh.lh_linear_nvfp4_grad(dy, *w, **wn)
    dx, ds = lh.lh_lora_grad(dy, a, b, scale, base=dx, dx=dx, ds=True, **kw, **wl)
    da, db = lh.lh_lora_weight_grad(values, dy, s, ds, a.shape[0], scale, x_scale=scales, **kw, **wg)
    return dict(y=y, s=s, dx=dx, ds=ds, da=da, db=db, values=values, scales=scales)


@pytest.mark.parametrize("rows,c_in,c_out,rank,dt", [(5, 64, 40, 4, BF16), (130, 272, 100, 16, BF16), (2100, 96, 64, 8, BF16),
                                                     (700, 128, 144, 40, BF16), (90, 80, 48, 8, F32)])
def test_training_step(lh, rows, c_in, c_out, rank, dt):
    """Against 64 bits, whose inputs are the roundings that the step makes on its
    way: y and dx of the projection are rounded (2^-8 for bf16) before the adapter
    adds to them, and rounded again after; da's x is the checkpoint's."""
    rng = np.random.default_rng([rows, c_in])
    q = projection(lh, rng, c_out, c_in)
    x, dy = rand(rng, rows, c_in, dtype=dt), rand(rng, rows, c_out, dtype=dt)
    a, b = rand(rng, 2, rank, c_in, dtype=dt, scale=c_in ** -0.5), rand(rng, 2, rank, c_out, dtype=dt, scale=0.1)
    scale = torch.tensor([0.5, 2.0], device=DEV)
    cut = rows // 3
    kw = dict(offsets=torch.tensor([0, cut, rows], device=DEV), adapter_ids=torch.tensor([1, 0], device=DEV))
    got = step(lh, q, x, dy, a, b, scale, kw)
    w, x64, dy64 = (t.double().cpu() for t in (q["w_q"][0], x, dy))
    kept = lh.lh_checkpoint_unpack(got["values"], got["scales"], out_dtype=F32).double().cpu()
    a64, b64 = a.double().cpu(), b.double().cpu()
    half = 2.0 ** -8 if dt == BF16 else 2.0 ** -24
    eps = 2.0 ** -17                                  # fp32 sums (8 sqrt(n) 2^-24 below it for n < 256), s cut to 16 bits
    for k, (g, sl) in enumerate(((1, slice(0, cut)), (0, slice(cut, rows)))):
        c = float(scale[g])
        for out, inp, lin, p, inner, outer in (("y", x64, w.t(), "s", a64[g], b64[g]), ("dx", dy64, w, "ds", b64[g], a64[g])):
            base, bm = inp[sl] @ lin, inp[sl].abs() @ lin.abs()
            r, rm = inp[sl] @ inner.t(), inp[sl].abs() @ inner.abs().t()
            assert ((got[p][sl].double().cpu() - r).abs() <= eps * rm + 1e-30).all(), p
            want, mass = base + c * (r @ outer), bm + c * (rm @ outer.abs())
            tol = 2 * eps * mass + half * (base.abs() + eps * bm)
            assert ((got[out][sl].double().cpu() - want).abs() <= tol + half * (want.abs() + tol)).all(), out
        s, ds = got["s"][sl].double().cpu(), got["ds"][sl].double().cpu()
        for out, p, v in (("da", ds, kept[sl]), ("db", s, dy64[sl])):
            tol = (8 * max(rows, 1) ** 0.5 + 3) * 2.0 ** -24 * c * (p.abs().t() @ v.abs())
            want = c * (p.t() @ v)
            assert ((got[out][g].double().cpu() - want).abs() <= tol + 2.0 ** -23 * want.abs() + 1e-30).all(), out


@pytest.mark.parametrize("rows,rank,segs", [(1, 16, 1), (9, 16, 9), (300, 16, 5), (2300, 8, 5), (500, 64, 3)])
def test_graph_replays_match_eager(lh, rows, rank, segs):
    rng = np.random.default_rng([3, rows])
    q = projection(lh, rng, 96, 128)
    x, dy = rand(rng, rows, 128), rand(rng, rows, 96)
    a, b = rand(rng, 4, rank, 128, scale=0.1), rand(rng, 4, rank, 96, scale=0.1)
    scale = torch.rand(4, device=DEV) + 0.5
    off = torch.from_numpy(np.sort(np.concatenate([[0, rows], rng.integers(0, rows + 1, segs - 1)]))).to(DEV)
    kw = dict(offsets=off, adapter_ids=torch.from_numpy(rng.integers(0, 4, segs)).to(DEV))
    u8 = dict(dtype=torch.uint8, device=DEV)
    ws = (torch.empty(max(lh.lh_lora_workspace_bytes(rows, segs, 128, 96, rank), lh.lh_lora_workspace_bytes(rows, segs, 128, 96, rank, grad=True), 256), **u8),
          torch.empty(max(lh.lh_lora_weight_grad_workspace_bytes(rows, segs, 4, rank, 128, 96), 256), **u8))
    eager = {k: v.clone() for k, v in step(lh, q, x, dy, a, b, scale, kw, ws).items()}
    assert all(torch.equal(v, eager[k]) for k, v in step(lh, q, x, dy, a, b, scale, kw, ws).items()), "a second call gives other bits"
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(lh, q, x, dy, a, b, scale, kw, ws)
    for rep in range(3):
        for v in out.values():                        # eager work between replays
            v.view(torch.uint8).fill_(0x55)
        for v in ws:
            v.fill_(0xAA)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, v in out.items():
            assert torch.equal(v, eager[k]), "replay %d: %s" % (rep, k)


def test_two_streams_at_once(lh):
    """Calls on two streams, each with tensors and a workspace of its own."""
    rng = np.random.default_rng(5)
    q = projection(lh, rng, 64, 96)
    sets = []
    for k in range(2):
        x, dy = rand(rng, 700, 96), rand(rng, 700, 64)
        a, b = rand(rng, 3, 16, 96, scale=0.1), rand(rng, 3, 16, 64, scale=0.1)
        kw = dict(offsets=torch.tensor([0, 100, 350, 700], device=DEV))
        sets.append((x, dy, a, b, torch.ones(3, device=DEV), kw))
    want = [step(lh, q, *v) for v in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(5):
        for k, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[k] = step(lh, q, *sets[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(got[k][n], want[k][n]) for n in want[k])


@pytest.mark.parametrize("tokens,experts,top_k,c_in,c_out,rank,refused", [(40, 6, 2, 64, 48, 4, 0.0), (600, 12, 3, 272, 130, 16, 0.2)])
def test_experts_adapters(lh, layer_example, tokens, experts, top_k, c_in, c_out, rank, refused):
    """The example's layer with an adapter for every expert: with b = 0 the layer
    without adapters, bit for bit; else the adapters' share of the output in 64
    bits (the experts' outputs are rounded to bf16 twice, 2^-8 each), and their
    gradients from the rows that the layer kept."""
    w, x, ids, weights, dy = layer_example.make(tokens, experts, top_k, c_in, c_out, seed=tokens)
    rng = np.random.default_rng(tokens)
    ids[torch.from_numpy(rng.random((tokens, top_k)) < refused).to(DEV)] = -1
    layer = layer_example.build_layer(lh, w, x, ids)
    a, b, scale = layer_example.make_adapters(experts, rank, c_in, c_out)
    plain, _ = layer_example.forward(lh, layer, x, ids, weights)
    same, _ = layer_example.forward(lh, layer, x, ids, weights, adapters=(a, torch.zeros_like(b), scale))
    assert torch.equal(plain, same)
    y, saved = layer_example.forward(lh, layer, x, ids, weights, adapters=(a, b, scale))
    dx, dweights, da, db = layer_example.backward(lh, layer, saved, weights, dy, (a, b, scale))
    assert dx.shape == x.shape and dweights.shape == weights.shape
    plan, ys, s, (values, scales) = saved
    kept = lh.lh_checkpoint_unpack(values, scales, out_dtype=F32).double().cpu()
    wq, wt, idc, x64, dy64 = layer["w_q"].double().cpu(), weights.double().cpu(), ids.cpu(), x.double().cpu(), dy.double().cpu()
    a64, b64, pos = a.double().cpu(), b.double().cpu(), plan["position"].cpu()
    ref, tol = torch.zeros(y.shape, dtype=torch.float64), torch.zeros(y.shape, dtype=torch.float64)
    rda, rdb = torch.zeros(da.shape, dtype=torch.float64), torch.zeros(db.shape, dtype=torch.float64)
    tda, tdb = rda.clone(), rdb.clone()
    for t in range(tokens):
        for k in range(top_k):
            e = int(idc[t, k])
            if e < 0:
                continue
            base, low = wq[e] @ x64[t], 2 * b64[e].t() @ (a64[e] @ x64[t])
            part = wq[e].abs() @ x64[t].abs() + 2 * b64[e].abs().t() @ (a64[e].abs() @ x64[t].abs())
            ref[t] += wt[t, k] * (base + low)
            tol[t] += wt[t, k] * (base.abs() * 2.0 ** -8 + (base + low).abs() * 2.0 ** -8 + part * 2.0 ** -15)
            dys = (wt[t, k] * dy64[t]).to(BF16).double()   # as the combination's gradient rounds it
            row = int(pos[t, k])
            rda[e] += 2 * torch.outer(b64[e] @ dys, kept[row])
            tda[e] += 2 * torch.outer(b64[e].abs() @ dys.abs(), kept[row].abs())
            rdb[e] += 2 * torch.outer(a64[e] @ x64[t], dys)
            tdb[e] += 2 * torch.outer(a64[e].abs() @ x64[t].abs(), dys.abs())
    assert ((y.double().cpu() - ref).abs() <= tol * 1.01 + ref.abs() * 2.0 ** -8 + 1e-30).all()
    # w dy is a product rounded to fp32 before bf16: where that changes the rounding, by one step of bf16 (2^-7)
    # in single terms; sums are fp32 (2^-16 of their mass covers 8 sqrt(n) 2^-24 for n < 1024, twice)
    assert ((da.double().cpu() - rda).abs() <= tda * 2.0 ** -7 + 1e-30).all()
    assert ((db.double().cpu() - rdb).abs() <= tdb * 2.0 ** -7 + 1e-30).all()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("power", [-126, -120, -100, 0, 60])
def test_checkpoints_of_any_magnitude(lh, dt, power):
    """The gradient takes a checkpoint's blocks at every exponent, the lowest among
    them (e = -127): against the values that come back in bf16, in 64 bits."""
    rng = np.random.default_rng(power + 200)
    rows, cols, rank = 70, 100, 8
    x = rng.uniform(1, 2, (rows, cols)) * 2.0 ** power * rng.choice([-1, 1], (rows, cols))
    x = torch.from_numpy(x.astype(np.float32)).to(dt).to(DEV)
    values, scales = lh.lh_checkpoint_pack(x)
    assert power > -119 or (scales == 0).all()
    ds = rand(rng, rows, rank, dtype=F32, scale=2.0 ** (-power / 2))
    da, _ = lh.lh_lora_weight_grad(values, x, None, ds, 1, x_scale=scales, db=False)
    kept, p = lh.lh_checkpoint_unpack(values, scales).double().cpu(), ds.double().cpu()
    want, mass = p.t() @ kept, p.abs().t() @ kept.abs()
    assert ((da[0].double().cpu() - want).abs() <= (8 * rows ** 0.5 + 6) * 2.0 ** -24 * mass).all()

"""The example's layer with an adapter for every expert and activations in NVFP4:
its rows are then in units of their global scale, which the adapters' share of the
output and their gradients have to carry.  Against 64 bits."""
import os
import sys

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


@pytest.fixture(scope="module")
def layer_example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import moe_layer
    return moe_layer


@pytest.mark.parametrize("tokens,experts,top_k,c_in,c_out,rank,refused", [(40, 6, 2, 64, 48, 4, 0.0), (600, 12, 3, 272, 130, 16, 0.2)])
def test_adapters_beside_quantized_activations(lh, layer_example, tokens, experts, top_k, c_in, c_out, rank, refused):
    """The adapters' inputs are the activations as the format holds them.  The
    experts' outputs are rounded to bf16 before the adapters add and after (2^-8
    each), the combination once more; sums are fp32 (2^-15 of their mass covers 8
    sqrt(n) 2^-24 twice over for n < 1024, and the products with the two scales).
    Gradients as in the layer without quantisation: the combination's gradient
    rounds w dy to bf16, by one step of it (2^-7) where a rounding changes."""
    w, x, ids, weights, dy = layer_example.make(tokens, experts, top_k, c_in, c_out, seed=tokens)
    rng = np.random.default_rng(tokens)
    ids[torch.from_numpy(rng.random((tokens, top_k)) < refused).to(DEV)] = -1
    layer = layer_example.build_layer(lh, w, x, ids)
    ad = layer_example.make_adapters(experts, rank, c_in, c_out)
    y, saved = layer_example.forward(lh, layer, x, ids, weights, quantize_x=True, adapters=ad)
    dx, dweights, da, db = layer_example.backward(lh, layer, saved, weights, dy, ad)
    plan, _, _, (values, scales) = saved[:4]
    q = lh.lh_quantize_nvfp4(x, layer["amax_x"], values=True, global_scale=True)
    unit = float(q["global_scale"].double())
    x64 = unit * q["values"][0].double().cpu()
    kept = unit * lh.lh_checkpoint_unpack(values, scales, out_dtype=F32).double().cpu()
    wq, wt, idc, dy64 = layer["w_q"].double().cpu(), weights.double().cpu(), ids.cpu(), dy.double().cpu()
    a64, b64, pos = ad[0].double().cpu(), ad[1].double().cpu(), plan["position"].cpu()
    ref, tol = torch.zeros(y.shape, dtype=torch.float64), torch.zeros(y.shape, dtype=torch.float64)
    rda, rdb = torch.zeros(da.shape, dtype=torch.float64), torch.zeros(db.shape, dtype=torch.float64)
    tda, tdb = rda.clone(), rdb.clone()
    rdx, tdx = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64)
    for t in range(tokens):
        for k in range(top_k):
            e = int(idc[t, k])
            if e < 0:
                continue
            base, low = wq[e] @ x64[t], 2 * b64[e].t() @ (a64[e] @ x64[t])
            part = wq[e].abs() @ x64[t].abs() + 2 * b64[e].abs().t() @ (a64[e].abs() @ x64[t].abs())
            ref[t] += wt[t, k] * (base + low)
            tol[t] += wt[t, k] * (base.abs() * 2.0 ** -8 + (base + low).abs() * 2.0 ** -8 + part * 2.0 ** -15)
            dys = (wt[t, k] * dy64[t]).to(BF16).double()
            ds, row = b64[e] @ dys, int(pos[t, k])
            rda[e] += 2 * torch.outer(ds, kept[row])
            tda[e] += 2 * torch.outer(b64[e].abs() @ dys.abs(), kept[row].abs())
            rdb[e] += 2 * torch.outer(a64[e] @ x64[t], dys)
            tdb[e] += 2 * torch.outer(a64[e].abs() @ x64[t].abs(), dys.abs())
            rdx[t] += wq[e].t() @ dys + 2 * a64[e].t() @ ds
            tdx[t] += wq[e].abs().t() @ dys.abs() + 2 * a64[e].abs().t() @ (b64[e].abs() @ dys.abs())
    assert ((y.double().cpu() - ref).abs() <= tol * 1.01 + ref.abs() * 2.0 ** -8 + 1e-30).all()
    assert ((da.double().cpu() - rda).abs() <= tda * 2.0 ** -7 + 1e-30).all()
    assert ((db.double().cpu() - rdb).abs() <= tdb * 2.0 ** -7 + 1e-30).all()
    assert ((dx.double().cpu() - rdx).abs() <= tdx * 2.0 ** -6 + 1e-30).all()   # and its own three roundings, 2^-8 each

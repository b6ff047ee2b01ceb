"""The calls together, as a layer uses them: the example's MoE layer against
the same layer in 64 bits with the weights the calibration returned, and the
new calls captured in a HIP graph, every replay against the eager result."""
import os
import sys

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
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


@pytest.mark.parametrize("tokens,experts,top_k,c_in,c_out,refused", [(40, 6, 2, 64, 48, 0.0), (130, 12, 3, 272, 130, 0.2),
                                                                     (3, 8, 2, 96, 33, 0.5)])
def test_layer_forward_and_backward(lh, layer_example, tokens, experts, top_k, c_in, c_out, refused):
    """The product of the packed weights is the product of the fake-quantised
    ones (r c S_g rounded twice in fp32, 2^-23 relative per weight), so the
    layer is compared with w_q in 64 bits.  Roundings on the way: the experts'
    outputs (bf16, 2^-8 each) meet weights that sum to at most 1, and y is
    rounded to bf16: 2 * 2^-8 of sum_k w |ys|, plus fp32 sums well below."""
    w, x, ids, weights, dy = layer_example.make(tokens, experts, top_k, c_in, c_out, seed=tokens)
    rng = np.random.default_rng(tokens)
    ids[torch.from_numpy(rng.random((tokens, top_k)) < refused).to(DEV)] = -1
    layer = layer_example.build_layer(lh, w, x, ids)
    y, saved = layer_example.forward(lh, layer, x, ids, weights)
    dx, dweights = layer_example.backward(lh, layer, saved, weights, dy)
    wq, x64, dy64 = layer["w_q"].double().cpu(), x.double().cpu(), dy.double().cpu()
    wt, idc = weights.double().cpu(), ids.cpu()
    ref, mass = torch.zeros((tokens, c_out), dtype=torch.float64), torch.zeros((tokens, c_out), dtype=torch.float64)
    rdx, mdx = torch.zeros((tokens, c_in), dtype=torch.float64), torch.zeros((tokens, c_in), dtype=torch.float64)
    rdw, mdw = torch.zeros((tokens, top_k), dtype=torch.float64), torch.zeros((tokens, top_k), dtype=torch.float64)
    for t in range(tokens):
        for k in range(top_k):
            e = int(idc[t, k])
            if e < 0:
                continue
            out = wq[e] @ x64[t]
            part = wq[e].abs() @ x64[t].abs()
            ref[t] += wt[t, k] * out
            mass[t] += wt[t, k] * (out.abs() * 2.0 ** -8 + part * 2.0 ** -18)   # rounding to bf16; fp32 sum
            rdx[t] += wt[t, k] * (dy64[t] @ wq[e])
            # dys = w dy rounded to bf16, dxs rounded to bf16
            mdx[t] += wt[t, k] * (dy64[t].abs() @ wq[e].abs()) * (2.0 ** -8 + 2.0 ** -18)
            mdx[t] += wt[t, k] * (dy64[t] @ wq[e]).abs() * 2.0 ** -8
            rdw[t, k] = dy64[t] @ out
            mdw[t, k] = dy64[t].abs() @ (out.abs() * 2.0 ** -8 + part * 2.0 ** -18) + dy64[t].abs() @ out.abs() * 2.0 ** -18
    assert ((y.double().cpu() - ref).abs() <= mass + (ref.abs() + mass) * 2.0 ** -8 + 1e-30).all()
    assert ((dx.double().cpu() - rdx).abs() <= mdx * 1.01 + (rdx.abs() + mdx) * 2.0 ** -8 + 1e-30).all()
    assert ((dweights.double().cpu() - rdw).abs() <= mdw * 1.01 + 1e-30).all()


def test_quantised_activations(lh, layer_example):
    """Activations in NVFP4: the product of the dequantised values, in 64 bits."""
    w, x, ids, weights, _ = layer_example.make(24, 4, 2, 96, 40, seed=7)
    layer = layer_example.build_layer(lh, w, x, ids)
    y, _ = layer_example.forward(lh, layer, x, ids, weights, quantize_x=True)
    q = lh.lh_quantize_nvfp4(x, layer["amax_x"], global_scale=True)
    xq = q["values"][0].double().cpu() * q["global_scale"].double().cpu()
    wq, wt, idc = layer["w_q"].double().cpu(), weights.double().cpu(), ids.cpu()
    ref, mass = torch.zeros(y.shape, dtype=torch.float64), torch.zeros(y.shape, dtype=torch.float64)
    for t in range(24):
        for k in range(2):
            e = int(idc[t, k])
            out, part = wq[e] @ xq[t], wq[e].abs() @ xq[t].abs()
            ref[t] += wt[t, k] * out
            mass[t] += wt[t, k] * (out.abs() * 2.0 ** -8 + part * 2.0 ** -18)
    assert ((y.double().cpu() - ref).abs() <= mass + (ref.abs() + mass) * 2.0 ** -8 + 1e-30).all()


@pytest.mark.parametrize("tokens", [1, 9, 300])
def test_graph_replays_match_eager(lh, layer_example, tokens):
    """Sort, dispatch, quantise, products, combine and the gradients in one
    graph (workspaces of the caller's): each replay equals the eager result."""
    w, x, ids, weights, dy = layer_example.make(tokens, 16, 4, 272, 96, seed=3)
    layer = layer_example.build_layer(lh, w, x, ids)
    n = tokens * 4
    u8 = dict(dtype=torch.uint8, device=DEV)
    ws_sort = torch.empty(max(lh.lh_moe_sort_workspace_bytes(tokens, 4, 16), 4), **u8)
    wsf = torch.empty(max(lh.lh_linear_nvfp4_workspace_bytes(n, 272, 96, 16, ragged=True), 256), **u8)
    wsg = torch.empty(max(lh.lh_linear_nvfp4_workspace_bytes(n, 272, 96, 16, grad=True, ragged=True), 256), **u8)
    dense = torch.empty(max(lh.lh_linear_nvfp4_workspace_bytes(tokens, 272, 96, dtype=torch.float32), 256), **u8)
    p0, c0, s0 = layer["packed"][:1].contiguous(), layer["scale_e4m3"][:1].contiguous(), layer["global_scale"][:1].contiguous()
    x32 = x.float()

    def step():
        plan = lh.lh_moe_sort(ids, 16, workspace=ws_sort)
        xs = lh.lh_moe_dispatch(x, plan["position"])
        ys = lh.lh_linear_nvfp4_ragged(xs, plan["offsets"], layer["packed"], layer["scale_e4m3"],
                                       layer["global_scale"], workspace=wsf)
        y = lh.lh_moe_combine(ys, plan["position"], weights)
        dys, dw = lh.lh_moe_combine_grad(dy, ys, plan["position"], weights)
        dxs = lh.lh_linear_nvfp4_ragged_grad(dys, plan["offsets"], layer["packed"], layer["scale_e4m3"],
                                             layer["global_scale"], workspace=wsg)
        dx = lh.lh_moe_combine(dxs, plan["position"])
        q = lh.lh_quantize_nvfp4(x, layer["amax_x"], packed=True, scale_e4m3=True, global_scale=True)
        yd = lh.lh_linear_nvfp4(x32, p0, c0, s0, workspace=dense)
        return dict(plan, xs=xs, y=y, dw=dw, dx=dx, yd=yd, **q)

    eager = {k: v.clone() for k, v in step().items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for rep in range(3):
        for v in out.values():      # eager work between replays
            v.view(torch.uint8).fill_(0x55)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for k, v in out.items():
            assert torch.equal(v, eager[k]), "replay %d: %s" % (rep, k)

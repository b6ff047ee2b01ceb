"""An MoE layer from calibration to a training step, through the library's calls.

    python3 examples/moe_layer.py [--tokens 4096] [--experts 64] [--top-k 8] [--c-in 2048] [--c-out 1024] [--rank 16]

1. Route tokens, sort them by expert (lh_moe_sort) and send their rows to the
   experts (lh_moe_dispatch).
2. Calibrate on those rows: per-expert Hessians (lh_accumulate_hessian_ragged),
   the 126-candidate sweep with packed weights (lh_scale_sweep_fake_quant).
3. The layer with NVFP4 weights: the experts' product on the sorted rows
   (lh_linear_nvfp4_ragged), rows back with the routing weights
   (lh_moe_combine); with activations in NVFP4 as well (lh_quantize_nvfp4).
4. Its gradients: to the routing weights and the experts' outputs
   (lh_moe_combine_grad), through the experts (lh_linear_nvfp4_ragged_grad) and
   back to the tokens (lh_moe_combine).
5. With --rank: a low-rank adapter for every expert beside its frozen weights
   (lh_lora, lh_lora_grad), trained from the experts' rows kept in 8 bits
   (lh_checkpoint_pack, lh_lora_weight_grad).

Random weights and activations stand in for a model's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def build_layer(lh, w, x, ids):
    """Calibrated NVFP4 weights of every expert from the tokens routed to it:
    dict(packed, scale_e4m3, global_scale, w_q, plan, xs, amax_x)."""
    experts = w.shape[0]
    plan = lh.lh_moe_sort(ids, experts)
    xs = lh.lh_moe_dispatch(x, plan["position"])
    nb = w.shape[2] // 16
    # experts without tokens keep the identity: the plain weight error decides for them
    h = torch.eye(16, device=w.device).expand(experts, nb, 16, 16).contiguous()
    lh.lh_accumulate_hessian_ragged(xs, plan["offsets"], h=h)
    amax = lh.lh_absmax(w)
    fq = lh.lh_scale_sweep_fake_quant(w, h, amax, best_err=False, best_amax=False, w_q=True, packed=True,
                                      scale_e4m3=True, global_scale=True)
    return dict(packed=fq["packed"], scale_e4m3=fq["scale_e4m3"], global_scale=fq["global_scale"], w_q=fq["w_q"],
                amax_x=lh.lh_absmax(x))


def forward(lh, layer, x, ids, weights, quantize_x=False, adapters=None):
    """y [tokens, c_out] and what the backward pass needs.  adapters: (a, b, scale), one for every expert."""
    experts = layer["packed"].shape[0]
    plan = lh.lh_moe_sort(ids, experts, order=False)
    x_scale = None
    if quantize_x:  # activations in units of their global scale, which the product multiplies back
        q = lh.lh_quantize_nvfp4(x, layer["amax_x"], values=True, global_scale=True)
        x, x_scale = q["values"][0], q["global_scale"].expand(experts).contiguous()
    xs = lh.lh_moe_dispatch(x, plan["position"])
    ys = lh.lh_linear_nvfp4_ragged(xs, plan["offsets"], layer["packed"], layer["scale_e4m3"], layer["global_scale"],
                                   x_scale=x_scale)
    # (rows of assignments without an expert are not written; nothing reads them)
    saved = (plan, ys)
    if adapters is not None:  # added in place; the rows are kept in 8 bits for the adapters' gradients
        a, b, scale = adapters
        if x_scale is not None:  # the adapters multiply the activations' units back as well
            scale = scale * x_scale
        ys, s = lh.lh_lora(xs, a, b, scale, offsets=plan["offsets"], base=ys, y=ys, s=True)
        saved = (plan, ys, s, lh.lh_checkpoint_pack(xs)) + (() if x_scale is None else (scale,))
    return lh.lh_moe_combine(ys, plan["position"], weights), saved


def backward(lh, layer, saved, weights, dy, adapters=None):
    """Gradients to the tokens, to the routing weights and, with adapters, to both factors of each."""
    plan, ys = saved[:2]
    dys, dweights = lh.lh_moe_combine_grad(dy, ys, plan["position"], weights)
    dxs = lh.lh_linear_nvfp4_ragged_grad(dys, plan["offsets"], layer["packed"], layer["scale_e4m3"],
                                         layer["global_scale"])
    if adapters is None:
        return lh.lh_moe_combine(dxs, plan["position"]), dweights
    s, (values, scales) = saved[2:4]
    scale = saved[4] if len(saved) > 4 else adapters[2]  # of the rows as they were kept: the tokens' gradient has no units
    dxs, ds = lh.lh_lora_grad(dys, *adapters, offsets=plan["offsets"], base=dxs, dx=dxs, ds=True)
    da, db = lh.lh_lora_weight_grad(values, dys, s, ds, adapters[0].shape[0], scale, offsets=plan["offsets"],
                                    x_scale=scales)
    return lh.lh_moe_combine(dxs, plan["position"]), dweights, da, db


def make(tokens, experts, top_k, c_in, c_out, seed=0, device="cuda:0"):
    gen = torch.Generator(device=device).manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device=device)

    w = (0.02 * rand(experts, c_out, c_in)).to(torch.bfloat16)
    x = (rand(tokens, c_in) * torch.exp(rand(c_in))).to(torch.bfloat16)
    top, ids = torch.topk(rand(tokens, experts) + rand(experts), top_k, dim=1)
    return w, x, ids, torch.softmax(top, dim=1), rand(tokens, c_out).to(torch.bfloat16)


def make_adapters(experts, rank, c_in, c_out, seed=1, device="cuda:0"):
    """(a, b, scale) as training finds them some steps on: neither factor is zero any more."""
    gen = torch.Generator(device=device).manual_seed(seed)
    a = torch.randn((experts, rank, c_in), generator=gen, device=device) * c_in ** -0.5
    b = torch.randn((experts, rank, c_out), generator=gen, device=device) * 0.02
    return a.to(torch.bfloat16), b.to(torch.bfloat16), torch.full((experts,), 2.0, device=device)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    ap.add_argument("--c-in", type=int, default=2048)
    ap.add_argument("--c-out", type=int, default=1024)
    ap.add_argument("--rank", type=int, default=16, help="rank of the experts' adapters (0: none)")
    a = ap.parse_args(argv)
    import nvfp4_scale_calibration_amd as lh

    w, x, ids, weights, dy = make(a.tokens, a.experts, a.top_k, a.c_in, a.c_out)
    layer = build_layer(lh, w, x, ids)
    exact = torch.zeros((a.tokens, a.c_out), device=x.device)
    for k in range(a.top_k):                       # the layer with unquantised weights, expert by expert
        for e in range(a.experts):
            t = ids[:, k] == e
            exact[t] += weights[t, k, None] * (x[t].float() @ w[e].float().t())
    norm = exact.norm()
    for quantize_x in (False, True):
        y, saved = forward(lh, layer, x, ids, weights, quantize_x)
        print("%s: relative output error against unquantised weights %.4f"
              % ("NVFP4 weights and activations" if quantize_x else "NVFP4 weights", float((y.float() - exact).norm() / norm)))
    dx, dweights = backward(lh, layer, saved, weights, dy)
    print("gradients: tokens %s, routing weights %s" % (tuple(dx.shape), tuple(dweights.shape)))

    def timed(f, n=20):
        for _ in range(3):
            f()
        ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        ev[0].record()
        for _ in range(n):
            f()
        ev[1].record()
        torch.cuda.synchronize()
        return ev[0].elapsed_time(ev[1]) / n * 1e3

    rows = a.tokens * a.top_k
    print("forward %.0f us, forward and backward %.0f us for %d rows on %d experts of %d x %d"
          % (timed(lambda: forward(lh, layer, x, ids, weights)),
             timed(lambda: backward(lh, layer, forward(lh, layer, x, ids, weights)[1], weights, dy)), rows, a.experts,
             a.c_out, a.c_in))
    if a.rank > 0:
        ad = make_adapters(a.experts, a.rank, a.c_in, a.c_out)
        _, _, da, db = backward(lh, layer, forward(lh, layer, x, ids, weights, adapters=ad)[1], weights, dy, ad)
        print("adapters of rank %d: gradients %s and %s, forward and backward with them %.0f us"
              % (a.rank, tuple(da.shape), tuple(db.shape),
                 timed(lambda: backward(lh, layer, forward(lh, layer, x, ids, weights, adapters=ad)[1], weights, dy, ad))))


if __name__ == "__main__":
    main()

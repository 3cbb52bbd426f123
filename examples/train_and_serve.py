"""Trains a small mixture-of-experts layer with its router, then serves it on 8-bit weights.

    python examples/train_and_serve.py [--steps 60] [--tokens 2048] [--f8]

A student layer (router, E experts) learns to reproduce a fixed teacher layer. One training step:

    logits = x @ R                          the router's own linear layer (torch)
    route      -> idx, prob, counts, losses
    MoeLayer.forward, .backward             out, dX, dprob
    MoeLayer.weight_grads                   dW1, dW2 of the experts, in fp32
    route_bwd  -> dlogits                   from dprob and the balance and z losses
    grad_norm, AdamW.step                   all weights in one launch, skipped unless finite

With --f8 the layer is F8MoeLayer: both directions on E4M3 codes of the BF16 weights with a scale
for every 128 x 128 block, made anew after each step (f8_prepare_weight).

Serving quantises the trained experts once (q8_prepare_weight) and runs Q8MoeLayer, for the whole
batch and for a single token. Needs a GB300 and the built library.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_grouped_gb300.gg as gg  # noqa: E402

E, H, F, K = 16, 256, 128, 2
AUX, ZCO, LR = 1e-2, 1e-3, 2e-3


def experts(g, scale):
    return [torch.randn(s, generator=g, device="cuda") * scale / s[2] ** 0.5
            for s in ((E, 2 * F, H), (E, H, F))]


def train(tokens: int, steps: int, seed: int = 0, log=print, f8: bool = False):
    """Returns dict(first, last, W1, W2, R, x, route, out, grads): losses, the trained layer, its
    outputs (with f8 those on the codes of W1 and W2) and the last step's gradients."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, H, generator=g, device="cuda").bfloat16()
    t1, t2 = experts(g, 1.5)
    tr = torch.randn(H, E, generator=g, device="cuda") / H ** 0.5
    layer = gg.MoeLayer(tokens, H, F, K, E)
    r = gg.route(x.float() @ tr, K, renormalize=True)
    target = layer.forward(x, r["idx"], r["prob"], t1.bfloat16(), t2.bfloat16()).float()
    weights = experts(g, 1.0)  # fp32 masters; the kernels read the BF16 copies W1 and W2
    weights.append(tr + 0.3 * torch.randn(H, E, generator=g, device="cuda") / H ** 0.5)
    R = weights[2]
    W1, W2, _ = half = [w.bfloat16() for w in weights]
    w1, w2 = (gg.f8_prepare_weight(W1), gg.f8_prepare_weight(W2)) if f8 else (W1, W2)
    student = gg.F8MoeLayer(tokens, H, F, K, E) if f8 else layer
    dW1, dW2, dR = grads = [torch.empty_like(w) for w in weights]
    opt = gg.AdamW(weights, grads, half=half, betas=(0.9, 0.99))
    norm = gg.GradPlan(grads)
    ws = gg.route_workspace(tokens, E, "cuda")
    losses = []
    for i in range(steps):
        logits = x.float() @ R
        r = gg.route(logits, K, renormalize=True, counts=True, losses=True, ws=ws)
        out = student.forward(x, r["idx"], r["prob"], w1, w2)
        err = out.float() - target
        losses.append(err.square().mean())
        dOut = (err * (2.0 / tokens)).bfloat16()
        _, dprob = student.backward(dOut, w1, w2, dprob=True)
        student.weight_grads(dW1, dW2)
        dlogits = gg.route_bwd(logits, r["idx"], dprob, renormalize=True, counts=r["counts"],
                               aux_coef=AUX, z_coef=ZCO)
        torch.mm(x.float().t(), dlogits, out=dR)
        opt.step(LR, grad_scale=gg.grad_norm(norm)[1:])
        if f8:
            gg.f8_prepare_weight(W1, *w1)
            gg.f8_prepare_weight(W2, *w2)
        if i % 20 == 0 or i == steps - 1:
            log(f"step {i:4d}  loss {losses[-1].item():.5f}  balance {r['losses'][0].item():.3f}"
                f"  busiest expert {int(r['counts'].max())} of {tokens * K} pairs")
    if student.status() != 0:
        raise RuntimeError(gg.status_string(student.status()))
    r = gg.route(x.float() @ R, K, renormalize=True)
    out = student.forward(x, r["idx"], r["prob"], w1, w2)
    return dict(first=losses[0].item(), last=losses[-1].item(), W1=W1, W2=W2, R=R,
                x=x, route=r, out=out, grads=grads)


def serve(trained, log=print):
    """Returns the relative distance of the 8-bit layer's outputs from the trained layer's, for the
    whole batch and for its first token alone."""
    W1, W2 = gg.q8_prepare_weight(trained["W1"]), gg.q8_prepare_weight(trained["W2"])
    x, r, ref = trained["x"], trained["route"], trained["out"].float()
    layer = gg.Q8MoeLayer(x.shape[0], H, F, K, E)
    out = layer.forward(x, r["idx"], r["prob"], W1, W2).float()
    one = layer.forward(x[:1], r["idx"][:1], r["prob"][:1], W1, W2).float()
    if layer.status() != 0:
        raise RuntimeError(gg.status_string(layer.status()))
    off = (float((out - ref).norm() / ref.norm()), float((one - ref[:1]).norm() / ref[:1].norm()))
    log(f"8-bit outputs against the trained layer's: {off[0]:.4f} (batch), {off[1]:.4f} (one token)")
    return off


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--f8", action="store_true", help="train on E4M3 codes of the weights")
    a = ap.parse_args()
    serve(train(a.tokens, a.steps, f8=a.f8))


if __name__ == "__main__":
    main()

"""Trains a small mixture-of-experts layer with its router, then serves it on 8-bit weights.

    python examples/train_and_serve.py [--steps 60] [--tokens 2048]

A student layer (router, E experts) learns to reproduce a fixed teacher layer. One training step:

    logits = x @ R                          the router's own linear layer (torch)
    route      -> idx, prob, counts, losses
    MoeLayer.forward, .backward             out, dX, dprob
    MoeLayer.weight_grads                   dW1, dW2 of the experts, in fp32
    route_bwd  -> dlogits                   from dprob and the balance and z losses

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


class Adam:
    """Adam on fp32 master weights; `half` is the BF16 copy that the kernels read."""

    def __init__(self, w):
        self.w, self.m, self.v, self.t = w, torch.zeros_like(w), torch.zeros_like(w), 0
        self.half = w.bfloat16()

    def step(self, g):
        self.t += 1
        self.m.lerp_(g, 0.1)
        self.v.lerp_(g * g, 0.01)
        m, v = self.m / (1 - 0.9 ** self.t), self.v / (1 - 0.99 ** self.t)
        self.w -= LR * m / (v.sqrt() + 1e-8)
        self.half.copy_(self.w)


def experts(g, scale):
    return [torch.randn(s, generator=g, device="cuda") * scale / s[2] ** 0.5
            for s in ((E, 2 * F, H), (E, H, F))]


def train(tokens: int, steps: int, seed: int = 0, log=print):
    """Returns dict(first, last, W1, W2, R, x, route, out): losses and the trained layer."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, H, generator=g, device="cuda").bfloat16()
    t1, t2 = experts(g, 1.5)
    tr = torch.randn(H, E, generator=g, device="cuda") / H ** 0.5
    layer = gg.MoeLayer(tokens, H, F, K, E)
    r = gg.route(x.float() @ tr, K, renormalize=True)
    target = layer.forward(x, r["idx"], r["prob"], t1.bfloat16(), t2.bfloat16()).float()
    W1, W2 = (Adam(w) for w in experts(g, 1.0))
    R = Adam(tr + 0.3 * torch.randn(H, E, generator=g, device="cuda") / H ** 0.5)
    ws = gg.route_workspace(tokens, E, "cuda")
    dW1, dW2 = (torch.empty_like(p.w) for p in (W1, W2))
    losses = []
    for i in range(steps):
        logits = x.float() @ R.w
        r = gg.route(logits, K, renormalize=True, counts=True, losses=True, ws=ws)
        out = layer.forward(x, r["idx"], r["prob"], W1.half, W2.half)
        err = out.float() - target
        losses.append(err.square().mean())
        dOut = (err * (2.0 / tokens)).bfloat16()
        _, dprob = layer.backward(dOut, W1.half, W2.half, dprob=True)
        layer.weight_grads(dW1, dW2)
        dlogits = gg.route_bwd(logits, r["idx"], dprob, renormalize=True, counts=r["counts"],
                               aux_coef=AUX, z_coef=ZCO)
        W1.step(dW1)
        W2.step(dW2)
        R.step(x.float().t() @ dlogits)
        if i % 20 == 0 or i == steps - 1:
            log(f"step {i:4d}  loss {losses[-1].item():.5f}  balance {r['losses'][0].item():.3f}"
                f"  busiest expert {int(r['counts'].max())} of {tokens * K} pairs")
    if layer.status() != 0:
        raise RuntimeError(gg.status_string(layer.status()))
    r = gg.route(x.float() @ R.w, K, renormalize=True)
    out = layer.forward(x, r["idx"], r["prob"], W1.half, W2.half)
    return dict(first=losses[0].item(), last=losses[-1].item(), W1=W1.half, W2=W2.half, R=R.w,
                x=x, route=r, out=out)


def serve(trained, log=print):
    """Returns the relative distance of the 8-bit layer's outputs from the BF16 layer's, for the
    whole batch and for its first token alone."""
    W1, W2 = gg.q8_prepare_weight(trained["W1"]), gg.q8_prepare_weight(trained["W2"])
    x, r, ref = trained["x"], trained["route"], trained["out"].float()
    layer = gg.Q8MoeLayer(x.shape[0], H, F, K, E)
    out = layer.forward(x, r["idx"], r["prob"], W1, W2).float()
    one = layer.forward(x[:1], r["idx"][:1], r["prob"][:1], W1, W2).float()
    if layer.status() != 0:
        raise RuntimeError(gg.status_string(layer.status()))
    off = (float((out - ref).norm() / ref.norm()), float((one - ref[:1]).norm() / ref[:1].norm()))
    log(f"8-bit outputs against BF16: {off[0]:.4f} (batch), {off[1]:.4f} (one token)")
    return off


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    serve(train(a.tokens, a.steps))


if __name__ == "__main__":
    main()

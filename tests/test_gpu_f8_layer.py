"""The expert layer on E4M3 weights, and a training step made of it: the layer's bits are those of
the calls it consists of (each held against the float64 oracle by itself), and a loop of router,
layer, weight gradients, gradient norm, AdamW and new codes gives the same bits captured as called.

Whole-layer gradients against the formula's: with both operands of a product quantised, every term
carries two independent errors of at most 2^-4 of itself, of standard deviation 2^-4 / sqrt(3) at
most, so a sum of terms of random sign is off by a factor of the 2-norm of at most
sqrt(2/3) 2^-4 = 0.051 for each product in a chain; the chains here are four products long at
most (x -> H1 -> A -> ... -> dX): 0.21 allowed. A wrong block's scale, a transposed weight or a
missing probability is off by 0.5 and more."""

import ctypes
import os
import sys

import numpy as np
import pytest
import torch

from oracle import adamw as oa

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


def _batch(T, H, F, k, E, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    idx = torch.rand(T, E, generator=g)
    if E > k:
        idx[:, E - 1] = -1  # the last expert gets no token
    idx = idx.topk(k, dim=1).indices.int().cuda()
    prob = (torch.rand(T, k, generator=g) + 0.1).cuda()
    W1 = (torch.randn(E, 2 * F, H, generator=g) * H ** -0.5).bfloat16().cuda()
    W2 = (torch.randn(E, H, F, generator=g) * F ** -0.5).bfloat16().cuda()
    dOut = torch.randn(T, H, generator=g).bfloat16().cuda()
    return x, idx, prob, W1, W2, dOut


def _by_hand(gg, x, idx, prob, w1, w2, dOut, k, E, P, act, mode):
    T, F = x.shape[0], w2[0].shape[2]
    ws = gg.workspace(T, k, E, "cuda")
    m = gg.permute(x, idx, prob, E, P, ws=ws)
    rc, off = gg.r_cap(T, k, E, P), m["offsets"]
    Xp = m["Xp"]
    if mode == 2:
        Xp = gg.permute_rows(x, m["row_of_slot"], m["slot_of_row"], off, k, E, P, rc, ws,
                             prob=prob)
    por = m["prob_of_row"]
    H1 = torch.zeros((rc, 2 * F), dtype=torch.bfloat16, device="cuda")
    A = gg.f8_grouped_fwd(Xp, *w1, off, 3 if act else 1, por if mode == 1 else None, H1_save=H1)
    Yp = gg.f8_grouped_fwd(A, *w2, off)
    out = gg.unpermute_combine(Yp, m["row_of_slot"], prob if mode == 0 else None, T, k, ws)
    dYp = gg.permute_rows(dOut, m["row_of_slot"], m["slot_of_row"], off, k, E, P, rc, ws)
    dot = torch.zeros((rc, gg.rowdot_stride(F)), device="cuda")
    dH = gg.f8_grouped_dgrad(dYp, *w2, off, 4 if act else 2, H1, None if mode == 2 else por,
                             rowdot=None if mode == 2 else dot)
    dXp = gg.f8_grouped_dgrad(dH, *w1, off)
    dprob = torch.zeros((T, k), device="cuda")
    if mode == 2:
        dX = gg.unpermute_combine(dXp, m["row_of_slot"], prob, T, k, ws, dot_src=x, dprob=dprob)
    else:
        dX = gg.unpermute_combine(dXp, m["row_of_slot"], None, T, k, ws, rowdot=dot, dprob=dprob,
                                  n_rowdot=gg.rowdot_blocks(F))
    return out, dX[0], dprob


SIZES = [(1, 64, 64, 1, 1, 1), (1, 128, 64, 2, 8, 1), (30, 192, 128, 2, 16, 8),
         (150, 128, 192, 3, 6, 1), (700, 320, 256, 2, 5, 16)]


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("T,H,F,k,E,P", SIZES)
def test_layer_is_its_calls(gg, T, H, F, k, E, P, act, mode):
    x, idx, prob, W1, W2, dOut = _batch(T, H, F, k, E, T)
    w1, w2 = gg.f8_prepare_weight(W1), gg.f8_prepare_weight(W2)
    layer = gg.F8MoeLayer(T, H, F, k, E, P, activation=act, prob_mode=mode)
    layer.ws8[256:] = 0x7F  # nothing of the scratch is used before it is written
    out = layer.forward(x, idx, prob, w1, w2)
    dX, dprob = layer.backward(dOut, w1, w2, dprob=True)
    assert layer.status() == 0
    want = _by_hand(gg, x, idx, prob, w1, w2, dOut, k, E, P, act, mode)
    for got, w in zip((out, dX, dprob), want):
        assert torch.equal(got, w)
    assert torch.equal(layer.backward(dOut, w1, w2), dX)


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("T,H,F,k,E,P", [(40, 256, 128, 2, 16, 1), (600, 256, 192, 2, 4, 16)])
def test_layer_gradients_against_autograd(gg, T, H, F, k, E, P, mode):
    x, idx, prob, W1, W2, dOut = _batch(T, H, F, k, E, 50 + T)
    layer = gg.F8MoeLayer(T, H, F, k, E, P, prob_mode=mode)
    w1, w2 = gg.f8_prepare_weight(W1), gg.f8_prepare_weight(W2)
    with pytest.raises(gg.GGError):
        layer.weight_grads()
    with pytest.raises(gg.GGError):
        layer.backward(dOut, w1, w2)
    got = [layer.forward(x, idx, prob, w1, w2)]
    got += layer.backward(dOut, w1, w2, dprob=True)
    got += layer.weight_grads(out_dtype=torch.float32)
    assert layer.status() == 0
    xs, ps, a1, a2 = (t.double().requires_grad_() for t in (x, prob, W1, W2))
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        p, e = ps[:, j:j + 1], idx[:, j].long()
        h = torch.einsum("th,tnh->tn", xs * p if mode == 2 else xs, a1[e])
        gate, up = h[:, :F], h[:, F:]
        y = torch.einsum("tf,thf->th", gate * torch.sigmoid(gate) * up, a2[e])
        out = out + (y if mode == 2 else p * y)
    (out * dOut.double()).sum().backward()
    for name, g, w in zip(("out", "dX", "dprob", "dW1", "dW2"), got,
                          (out.detach(), xs.grad, ps.grad, a1.grad, a2.grad)):
        assert float((g.double() - w).norm() / w.norm()) < 0.21, name
    for dW in got[3:]:
        assert (dW[E - 1] == 0).all()


def test_smaller_batches_and_none(gg):
    T, H, F, k, E = 64, 128, 64, 2, 8
    x, idx, prob, W1, W2, dOut = _batch(T, H, F, k, E, 3)
    w1, w2 = gg.f8_prepare_weight(W1), gg.f8_prepare_weight(W2)
    layer = gg.F8MoeLayer(T, H, F, k, E)
    for n in (64, 1, 0, 17):
        a = x[:n], idx[:n], prob[:n]
        fresh = gg.F8MoeLayer(max(n, 1), H, F, k, E)
        out, alone = layer.forward(*a, w1, w2), fresh.forward(*a, w1, w2)
        dX, dp = layer.backward(dOut[:n], w1, w2, dprob=True)
        assert out.shape == dX.shape == (n, H) and dp.shape == (n, k)
        assert torch.equal(out, alone) and torch.equal(dX, fresh.backward(dOut[:n], w1, w2))
    with pytest.raises(gg.GGError):
        layer.forward(torch.cat([x, x]), torch.cat([idx, idx]), torch.cat([prob, prob]), w1, w2)


def test_layer_refuses(gg):
    T, H, F, k, E = 8, 128, 64, 2, 4
    x, idx, prob, W1, W2, dOut = _batch(T, H, F, k, E, 4)
    w1, w2 = gg.f8_prepare_weight(W1), gg.f8_prepare_weight(W2)
    layer = gg.F8MoeLayer(T, H, F, k, E)
    with pytest.raises(TypeError):
        layer.forward(x, idx, prob, (W1, w1[1]), w2)
    with pytest.raises(ValueError):
        layer.forward(x, idx, prob, w2, w1)
    with pytest.raises(ValueError):
        layer.forward(x.cpu(), idx, prob, w1, w2)
    with pytest.raises(ValueError):
        layer.forward(x, idx, prob, w1, (w2[0].cpu(), w2[1].cpu()))
    layer.forward(x, idx, prob, w1, w2)
    with pytest.raises(ValueError):
        layer.backward(dOut[:4], w1, w2)
    with pytest.raises(ValueError):
        layer.backward(dOut, w1, w2, dX=torch.empty_like(x).cpu())
    # what the binding cannot ask for
    opt = gg.GGOptions(0, 0, 1)
    ptr = [t.data_ptr() for t in (x, idx, prob, *w1, *w2)]
    assert gg.LIB.gg_moe_mlp_fwd_f8(*ptr, T, H, F, k, E, 1, ctypes.byref(opt), x.data_ptr(),
                                    ctypes.byref(layer.buf), layer.ws8.data_ptr(),
                                    layer.ws8.numel(), None) == 1
    assert gg.LIB.gg_moe_mlp_fwd_f8(*ptr, T, H, F, k, E, 1, None, x.data_ptr(),
                                    ctypes.byref(layer.buf), layer.ws8.data_ptr(),
                                    layer.ws8.numel() - 1, None) == 4


def _loop(gg, T, H, F, k, E, seed, bits):
    """A training step over fixed buffers, and everything that it changes."""
    x, idx, prob, W1, W2, dOut = _batch(T, H, F, k, E, seed)
    g = torch.Generator().manual_seed(seed)
    R = (torch.randn(H, E, generator=g) * H ** -0.5).cuda()
    master = [W1.float(), W2.float(), R]
    half = [W1, W2, torch.empty_like(R, dtype=torch.bfloat16)]
    grads = [torch.zeros_like(w) for w in master]
    opt = gg.AdamW(master, grads, half=half, state_bits=bits, betas=(0.9, 0.99),
                   weight_decay=0.01, seed=5)
    plan = gg.GradPlan(grads)
    w1, w2 = gg.f8_prepare_weight(W1), gg.f8_prepare_weight(W2)
    layer = gg.F8MoeLayer(T, H, F, k, E)
    ws = gg.route_workspace(T, E, "cuda")
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    lr = torch.full((1,), 1e-2, device="cuda")
    norm = torch.zeros(2, device="cuda")
    out = torch.zeros_like(x)

    def once():
        step.add_(1)
        logits = x.float() @ R
        r = gg.route(logits, k, renormalize=True, counts=True, losses=True, ws=ws)
        layer.forward(x, r["idx"], r["prob"], w1, w2, out)
        err = ((out.float() - dOut.float()) * (2.0 / T)).bfloat16()
        _, dprob = layer.backward(err, w1, w2, dprob=True)
        layer.weight_grads(grads[0], grads[1])
        dlogits = gg.route_bwd(logits, r["idx"], dprob, renormalize=True, counts=r["counts"],
                               aux_coef=1e-2)
        torch.mm(x.float().t(), dlogits, out=grads[2])
        gg.grad_norm(plan, 1.0, out=norm)
        opt.step(lr, step=step, grad_scale=norm[1:])
        gg.f8_prepare_weight(W1, *w1)
        gg.f8_prepare_weight(W2, *w2)

    state = master + half + [norm, out, step] + list(w1) + list(w2) + opt.m + opt.v
    return once, state, dict(layer=layer, grads=grads, master=master, half=half, opt=opt,
                             norm=norm, w=(w1, w2))


def _bits(ts):
    return [t.detach().contiguous().view(torch.uint8).clone() for t in ts]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("T", [24, 500])
def test_training_steps_captured_as_called(gg, T, bits):
    size = (T, 128, 192, 2, 12, 9, bits)
    once, state, _ = _loop(gg, *size)
    for _ in range(4):
        once()
    want = _bits(state)
    once2, state2, own = _loop(gg, *size)
    once2()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        once2()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert own["layer"].status() == 0
    for a, b in zip(want, _bits(state2)):
        assert torch.equal(a, b)


def test_training_step_against_its_oracle(gg):
    """The first step's weights, bit for bit, from the gradients that the layer gave."""
    once, _, own = _loop(gg, 200, 128, 64, 2, 6, 11, 32)
    before = [w.cpu().numpy().copy() for w in own["master"]]
    once()
    grads = [g.cpu().numpy() for g in own["grads"]]
    total = float(np.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in grads)))
    norm, scale = own["norm"].tolist()
    assert abs(norm - total) <= 2.0 ** -20 * total
    for i, (w, g) in enumerate(zip(before, grads)):
        zero = np.zeros(g.size, np.float32)
        new = oa.step(w.ravel(), g.ravel(), zero, zero.copy(), lr=float(np.float32(1e-2)), t=1,
                      beta1=0.9, beta2=0.99, weight_decay=0.01, grad_scale=scale)
        np.testing.assert_array_equal(own["master"][i].cpu().numpy().ravel(), new[0])
    for (q, s), W in zip(own["w"], own["half"]):
        want = gg.f8_prepare_weight(W)
        assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8))
        assert torch.equal(s, want[1])


def test_example_trains_on_codes(gg):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_and_serve as ex
    finally:
        sys.path.pop(0)
    t = ex.train(256, 3, f8=True, log=lambda *_: None)
    for w in (t["W1"], t["W2"], t["R"], t["out"]):
        assert torch.isfinite(w.float()).all()


def test_example_on_codes_takes_its_steps_on_them(gg):
    """A step whose gradients are not finite is skipped and leaves the weights finite, so: the loss
    is finite, every step moves the weights, and what is returned comes from the codes. The first
    step's expert gradients stand beside those of BF16 at the same weights, three products down the
    chain and behind a difference (outputs less the teacher's, which are independent of them, so that
    it is no smaller than the outputs): 0.21 as above."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import train_and_serve as ex
    finally:
        sys.path.pop(0)
    runs = [ex.train(256, n, f8=True, log=lambda *_: None) for n in (1, 2, 3)]
    for t in runs:
        assert np.isfinite([t["first"], t["last"]]).all()
    assert runs[0]["first"] == runs[1]["first"] == runs[2]["first"]
    assert len({t["last"] for t in runs}) == 3
    for a, b in zip(runs, runs[1:]):
        for w in ("W1", "W2", "R"):
            assert float((a[w] != b[w]).float().mean()) > 0.2
    t = runs[2]
    layer = gg.F8MoeLayer(256, ex.H, ex.F, ex.K, ex.E)
    want = layer.forward(t["x"], t["route"]["idx"], t["route"]["prob"],
                         gg.f8_prepare_weight(t["W1"]), gg.f8_prepare_weight(t["W2"]))
    assert torch.equal(t["out"], want)
    bf16 = ex.train(256, 1, log=lambda *_: None)
    for got, ref in zip(runs[0]["grads"][:2], bf16["grads"][:2]):
        assert float((got - ref).norm() / ref.norm()) < 0.21

"""The router, the experts' weight gradients and the 8-bit layer as a program uses them: the whole
layer's weight gradients against float64 autograd for every option, the 8-bit layer against its
integer oracle, and the training example end to end."""

import ctypes
import os
import sys

import numpy as np
import pytest
import torch

from oracle import q8 as qo

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
    idx[:, E - 1] = -1  # the last expert gets no token
    idx = idx.topk(k, dim=1).indices.int().cuda()
    prob = (torch.rand(T, k, generator=g) + 0.1).cuda()
    W1 = (torch.randn(E, 2 * F, H, generator=g) * H ** -0.5).bfloat16().cuda()
    W2 = (torch.randn(E, H, F, generator=g) * F ** -0.5).bfloat16().cuda()
    dOut = torch.randn(T, H, generator=g).bfloat16().cuda()
    return x, idx, prob, W1, W2, dOut


@pytest.mark.parametrize("mode", [0, 1, 2])
@pytest.mark.parametrize("act,P,recompute", [(0, 1, False), (1, 16, False), (0, 1, True)])
def test_layer_weight_gradients_against_autograd(gg, mode, act, P, recompute):
    # Every operand of the two products has been rounded to BF16 (dH from BF16 H1 and an fp32
    # gradient; the weighted activation): relative errors of 2^-9 in each factor, independent
    # from element to element, so the tensors agree to a few 2^-9 in the 2-norm (1e-2 allowed).
    T, H, F, k, E = 150, 128, 192, 3, 6
    x, idx, prob, W1, W2, dOut = _batch(T, H, F, k, E, 7 + mode)
    layer = gg.MoeLayer(T, H, F, k, E, P, activation=act, prob_mode=mode, recompute_h1=recompute)
    with pytest.raises(gg.GGError):
        layer.weight_grads()
    layer.forward(x, idx, prob, W1, W2)
    layer.backward(dOut, W1, W2)
    dW1, dW2 = layer.weight_grads(out_dtype=torch.float32)
    assert layer.status() == 0
    a1, a2 = (w.double().requires_grad_() for w in (W1, W2))
    alpha = 1.702 if act else 1.0
    out = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for j in range(k):
        p = prob.double()[:, j:j + 1]
        xin = x.double() * (p if mode == 2 else 1.0)
        h = torch.einsum("th,tnh->tn", xin, a1[idx[:, j].long()])
        gate, up = h[:, :F], h[:, F:]
        y = torch.einsum("tf,thf->th", gate * torch.sigmoid(alpha * gate) * up,
                         a2[idx[:, j].long()])
        out = out + (y if mode == 2 else p * y)
    (out * dOut.double()).sum().backward()
    for got, want in ((dW1, a1.grad), (dW2, a2.grad)):
        assert (got[E - 1] == 0).all()
        assert float((got.double() - want).norm() / want.norm()) < 1e-2
    # again, in BF16, onto a base, and in place: the same sums
    again = layer.weight_grads(out_dtype=torch.float32)
    assert torch.equal(again[0], dW1) and torch.equal(again[1], dW2)
    b1, b2 = layer.weight_grads()
    assert torch.equal(b1, dW1.bfloat16()) and torch.equal(b2, dW2.bfloat16())
    acc1, acc2 = torch.ones_like(dW1), torch.ones_like(dW2)
    layer.weight_grads(acc1, acc2, base1=acc1, base2=acc2)
    assert torch.equal(acc1, dW1 + 1) and torch.equal(acc2, dW2 + 1)


def test_layer_weight_gradients_of_a_smaller_batch(gg):
    T, H, F, k, E = 90, 64, 64, 2, 4
    x, idx, prob, W1, W2, dOut = _batch(T, H, F, k, E, 3)
    big, small = gg.MoeLayer(T, H, F, k, E), gg.MoeLayer(40, H, F, k, E)
    got = []
    for layer in (big, small):
        layer.forward(x[:40].contiguous(), idx[:40].contiguous(), prob[:40].contiguous(), W1, W2)
        layer.backward(dOut[:40].contiguous(), W1, W2)
        got.append(layer.weight_grads())
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("T", [1, 5, 300])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("mode", [0, 1])
def test_8bit_layer_matches_oracle(gg, T, act, mode):
    # The activation is rounded to BF16 before its rows are quantised: where that rounding moves a
    # value across a code's boundary the code differs by one of 127 from the oracle's, a
    # perturbation of the kind and size the quantiser makes anyway (2-norm 1e-2 allowed, the
    # quantiser itself makes about 1e-2).
    H, F, k, E = 192, 128, 3, 7
    x, idx, prob, W1, W2, _ = _batch(T, H, F, k, E, 20 + T)
    layer = gg.Q8MoeLayer(T + 3, H, F, k, E, activation=act, prob_mode=mode)
    q1, q2 = gg.q8_prepare_weight(W1), gg.q8_prepare_weight(W2)
    out = layer.forward(x, idx, prob, q1, q2)
    assert layer.status() == 0
    w1, w2 = qo.quantize_rows(W1.float().cpu().numpy()), qo.quantize_rows(W2.float().cpu().numpy())
    np.testing.assert_array_equal(q1[0].cpu().numpy(), w1[0])
    eid = idx.cpu().numpy().reshape(-1)
    order = np.argsort(eid, kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(eid, minlength=E))])
    rows = x.float().cpu().numpy()[order // k]
    pr = prob.cpu().numpy().reshape(-1)[order]
    xq, xs = qo.quantize_rows(rows)
    a = qo.grouped_gemm(xq, xs, *w1, off, 1.702 if act else 1.0, pr if mode == 1 else None)
    a = torch.from_numpy(a).bfloat16().float().numpy()
    aq, asc = qo.quantize_rows(a)
    y = qo.grouped_gemm(aq, asc, *w2, off)
    want = np.zeros((T, H))
    np.add.at(want, order // k, y * (pr[:, None] if mode == 0 else 1.0))
    err = np.linalg.norm(out.double().cpu().numpy() - want) / np.linalg.norm(want)
    assert err < 1e-2


def test_8bit_layer_refusals(gg):
    L = gg.LIB
    p = ctypes.c_void_p(1 << 40)
    T, H, F, k, E = 8, 64, 64, 2, 4
    n = L.gg_q8_buffers_size(T, H, F, k, E)
    assert L.gg_q8_buffers_size(T, 96, F, k, E) == 0 and L.gg_q8_buffers_size(-1, H, F, k, E) == 0
    b = gg.GGQ8Buffers()
    assert L.gg_q8_buffers_bind(p, n - 1, T, H, F, k, E, ctypes.byref(b)) == 4
    assert L.gg_q8_buffers_bind(ctypes.c_void_p((1 << 40) + 16), n, T, H, F, k, E,
                                ctypes.byref(b)) == 3
    assert L.gg_q8_buffers_bind(p, n, T, H, F, k, E, ctypes.byref(b)) == 0
    sizes = dict(Xq=16 * H, Xs=64, A=32 * F, Aq=16 * F, As=64, Yp=32 * H, offsets=4 * (E + 1),
                 row_of_slot=64, slot_of_row=64, prob_of_row=64, ws=b.ws_bytes)
    spans = sorted((getattr(b, m), getattr(b, m) + s) for m, s in sizes.items())
    assert all(x[1] <= y[0] for x, y in zip(spans, spans[1:]))
    assert spans[0][0] >= 1 << 40 and spans[-1][1] <= (1 << 40) + n
    n0 = gg.launch_count()

    def call(opt=None, W=p, x=p, buf=b, h=H):
        o = None if opt is None else ctypes.byref(gg.GGOptions(*opt))
        return L.gg_moe_mlp_fwd_q8(x, p, p, W, p, p, p, T, h, F, k, E, o, p, ctypes.byref(buf),
                                   None)

    assert call((0, 2, 0)) == 1 and call((0, 0, 1)) == 1 and call((2, 0, 0)) == 1
    assert call(W=None) == 1 and call(x=None) == 1 and call(buf=gg.GGQ8Buffers()) == 1
    assert call(h=96) == 2
    assert L.gg_moe_mlp_wgrad(T, H, F, k, E, 1, None, 0, None, p, None, p, None, p, 1 << 20,
                              None) == 1
    assert gg.launch_count() == n0
    layer = gg.Q8MoeLayer(T, H, F, k, E)
    x = torch.zeros(T + 1, H, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(gg.GGError):
        layer.forward(x, None, None, None, None)


def test_training_example_learns_and_serves(gg):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_and_serve as ex

    t = ex.train(512, 40, log=lambda *_: None)
    assert t["last"] < 0.5 * t["first"]
    batch, one = ex.serve(t, log=lambda *_: None)
    assert batch < 0.05 and one < 0.1

"""The router's oracle against closed forms and differences (CPU), and the host-side checks of
gg_route / gg_route_bwd (no kernel runs here)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import router as ro

VARIANTS = [(sig, ren) for sig in (False, True) for ren in (False, True)]


@pytest.fixture(scope="module")
def gg():
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


@pytest.mark.parametrize("sig,ren", VARIANTS)
def test_backward_is_the_derivative_of_the_objective(sig, ren):
    # central differences of a smooth function: truncation h^2 |f'''| / 6 ~ 1e-8 for h = 1e-4
    rng = np.random.default_rng(5)
    T, E, k = 5, 7, 3
    x = rng.standard_normal((T, E))
    x[2, 4] = -np.inf
    f = ro.route_forward(x, k, sig, ren, 1.7)
    dprob = rng.standard_normal((T, k))
    args = dict(sigmoid=sig, renorm=ren, scale=1.7, aux=0.3, z=0.2)
    dx, _ = ro.route_backward(x, f["idx"], f["counts"], dprob, **args)
    h = 1e-4
    for t in range(T):
        for e in range(E):
            if np.isneginf(x[t, e]):
                assert dx[t, e] == 0
                continue
            lo, hi = x.copy(), x.copy()
            lo[t, e] -= h
            hi[t, e] += h
            fd = (ro.route_objective(hi, f["idx"], f["counts"], dprob, **args)
                  - ro.route_objective(lo, f["idx"], f["counts"], dprob, **args)) / (2 * h)
            assert abs(fd - dx[t, e]) < 1e-6


@pytest.mark.parametrize("sig,ren", VARIANTS)
def test_oracle_matches_autograd(sig, ren):
    rng = np.random.default_rng(6)
    T, E, k = 9, 12, 4
    x = torch.tensor(rng.standard_normal((T, E)), requires_grad=True)
    f = ro.route_forward(x.detach().numpy(), k, sig, ren)
    idx = torch.from_numpy(f["idx"].astype(np.int64))
    s = torch.sigmoid(x) if sig else torch.softmax(x, 1)
    prob = s.gather(1, idx)
    if ren:
        prob = prob / prob.sum(1, keepdim=True)
    share = s / s.sum(1, keepdim=True)
    balance = E * (torch.from_numpy(f["counts"] / (T * k)) * share.mean(0)).sum()
    zl = torch.logsumexp(x, 1).square().mean()
    np.testing.assert_allclose(f["prob"], prob.detach().numpy(), rtol=1e-12)
    np.testing.assert_allclose(f["losses"], [balance.item(), zl.item()], rtol=1e-12)
    dprob = rng.standard_normal((T, k))
    ((torch.from_numpy(dprob) * prob).sum() + 0.4 * balance + 0.1 * zl).backward()
    dx, _ = ro.route_backward(x.detach().numpy(), f["idx"], f["counts"], dprob, sig, ren,
                              aux=0.4, z=0.1)
    np.testing.assert_allclose(dx, x.grad.numpy(), rtol=1e-9, atol=1e-14)


def test_balance_loss_is_one_when_even():
    # every expert picked equally often with equal scores: f_e = P_e = 1 / E
    f = ro.route_forward(np.zeros((4, 4)) + np.eye(4) * 0, 4)
    np.testing.assert_allclose(f["losses"][0], 1.0)


def test_ties_nan_and_dead_rows_in_the_oracle():
    x = np.array([[1.0, 3.0, 3.0, 1.0], [np.nan, 5.0, 5.0, 9.0], [-np.inf] * 4,
                  [0.0, -0.0, 0.0, -1.0]])
    f = ro.route_forward(x, 3)
    np.testing.assert_array_equal(f["idx"], [[1, 2, 0], [0, 3, 1], [0, 1, 2], [0, 1, 2]])
    assert np.isnan(f["prob"][1]).all() and (f["prob"][2] == 0).all()


def test_validation_rejects_before_launch(gg):
    L = gg.LIB
    p = ctypes.c_void_p(1 << 40)
    odd = ctypes.c_void_p((1 << 40) + 2)
    ws = ctypes.c_void_p(1 << 41)
    n = L.gg_route_workspace_size(64, 16)
    assert n >= 256 and L.gg_route_workspace_size(-1, 16) == 0
    assert L.gg_route_workspace_size(64, 0) == 0
    # the scratch stops growing with the batch
    assert L.gg_route_workspace_size(1 << 20, 16) == L.gg_route_workspace_size(1 << 24, 16)
    n0 = gg.launch_count()

    def fwd(logits=p, dtype=0, T=64, E=16, k=4, score=0, idx=p, prob=p, counts=p, losses=p, w=ws,
            wb=n):
        return L.gg_route(logits, dtype, T, E, k, score, 0, 1.0, idx, prob, counts, losses, w, wb,
                          None)

    assert fwd(T=-1) == 1 and fwd(E=0) == 1 and fwd(k=0) == 1
    assert fwd(k=17) == 1 and fwd(E=64, k=33) == 1      # k <= E and k <= 32
    assert fwd(dtype=2) == 1 and fwd(score=2) == 1 and fwd(score=-1) == 1
    assert fwd(E=1025) == 2
    assert fwd(logits=None) == 1 and fwd(idx=None) == 1 and fwd(prob=None) == 1
    assert fwd(logits=odd) == 3 and fwd(prob=odd) == 3 and fwd(counts=odd) == 3
    assert fwd(w=None) == 1 and fwd(wb=n - 1) == 4
    assert fwd(w=ctypes.c_void_p((1 << 41) + 8)) == 3

    def bwd(logits=p, dtype=0, T=64, E=16, k=4, score=0, idx=p, dprob=p, counts=p, aux=0.5, out=p,
            w=ws, wb=256):
        return L.gg_route_bwd(logits, dtype, T, E, k, score, 0, 1.0, idx, dprob, counts, aux, 0.0,
                              out, w, wb, None)

    assert bwd(k=17) == 1 and bwd(dtype=7) == 1 and bwd(score=2) == 1 and bwd(E=2000) == 2
    assert bwd(idx=None) == 1 and bwd(dprob=None) == 1 and bwd(out=None) == 1
    assert bwd(counts=None) == 1                         # the balance loss needs the counts
    assert bwd(out=odd) == 3 and bwd(logits=odd) == 3 and bwd(wb=16) == 4
    assert gg.launch_count() == n0


def test_binding_refuses_wrong_tensors(gg):
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        gg.route(x, 2)                                   # not on a GPU
    with pytest.raises(TypeError):
        gg.route(x.to(torch.float16), 2)
    with pytest.raises(ValueError):
        gg.route(x, 2, idx=torch.zeros(4, 3, dtype=torch.int32))
    with pytest.raises(TypeError):
        gg.route_bwd(x, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))

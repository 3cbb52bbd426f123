"""CPU checks of the E4M3 products with scales per block of 128: the oracle's codes against
torch's E4M3, its gradient against differences, and the refusals that come before any launch."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import f8 as of
from oracle.adamw import E4M3


@pytest.fixture(scope="module")
def gg():
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


def test_codes_are_torch_e4m3():
    r = np.random.default_rng(0)
    y = np.concatenate([r.uniform(-448, 448, 20000), r.normal(size=20000) * 0.01, E4M3[:127],
                        (E4M3[:126] + E4M3[1:127]) / 2, [0.0, -0.0]]).astype(np.float32)
    want = torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(of.encode(y), want)


@pytest.mark.parametrize("K", [64, 128, 192, 1024])
def test_quantised_rows_are_near(K):
    """Half a step: 2^-4 of the value, or of the smallest normal code's scale."""
    x = np.random.default_rng(K).normal(size=(40, K)).astype(np.float32)
    x[3] = 0
    Q, S = of.quantize_rows(x)
    v = of.rows_value(Q, S)
    s = np.repeat(S.T.astype(np.float64), 128, axis=1)[:, :K]
    assert (np.abs(v - x) <= 2.0 ** -4 * np.maximum(np.abs(x), s * 2.0 ** -6) * 1.001).all()
    assert (v[3] == 0).all() and (S[:, 3] > 0).all()


def test_nonfinite_blocks():
    x = np.ones((3, 256), np.float32)
    x[0, 5], x[1, 200] = np.nan, -np.inf
    Q, S = of.quantize_rows(x)
    assert np.isnan(S[0, 0]) and np.isnan(S[1, 1]) and np.isfinite(S).sum() == 4
    assert (Q[0, :128] == 0).all() and (Q[1, 128:] == 0).all()


def test_gradient_is_the_derivative():
    """The products are linear: dA against central differences of <dC, C>."""
    r = np.random.default_rng(3)
    W = r.normal(size=(2, 192, 320)).astype(np.float32)
    Wq, Ws = of.quantize_weight(W)
    off = [0, 3, 5]
    d, S = of.quantize_rows(r.normal(size=(5, 192)).astype(np.float32))
    dA, _ = of.product(d, S, Wq, Ws, off, grad=True)
    x = r.normal(size=(5, 320))
    w = of.weight_value(Wq, Ws)
    dv = of.rows_value(d, S)
    for i, c in ((0, 0), (2, 319), (4, 130)):
        def loss(h):
            y = x.copy()
            y[i, c] += h
            return sum((dv[t] * (w[0 if t < 3 else 1] @ y[t])).sum() for t in range(5))
        assert abs((loss(0.5) - loss(-0.5)) - dA[i, c]) < 1e-9 * max(1, abs(dA[i, c]))


def test_gated_gradient_is_the_derivative():
    r = np.random.default_rng(4)
    g, u, acc, p = r.normal(size=(6, 8)), r.normal(size=(6, 8)), r.normal(size=(6, 8)), r.random(6)
    for alpha in (1.0, 1.702):
        dg, du, dot = of.glu_bwd(acc, g, u, alpha, p)
        h = 1e-5

        def f(g, u, p):
            return (acc * p[:, None] * of.glu(g, u, alpha)).sum(axis=1)
        for j in range(8):
            e = np.zeros(8)
            e[j] = h
            np.testing.assert_allclose((f(g + e, u, p) - f(g - e, u, p)) / (2 * h), dg[:, j],
                                       atol=1e-8)
            np.testing.assert_allclose((f(g, u + e, p) - f(g, u - e, p)) / (2 * h), du[:, j],
                                       atol=1e-8)
        np.testing.assert_allclose((f(g, u, p + h) - f(g, u, p - h)) / (2 * h), dot.sum(axis=1),
                                   atol=1e-8)


class TestRefusals:
    """The pointers are never used."""

    def _fwd(self, gg, **kw):
        a = dict(A=1 << 12, Wq=1 << 13, Ws=1 << 14, off=1 << 15, E=4, R=100, K=128, N=256, epi=0,
                 C=1 << 16, H1=None, prob=None, ws=1 << 17, nbytes=1 << 30)
        a.update(kw)
        return gg.LIB.gg_f8_grouped_fwd(a["A"], a["Wq"], a["Ws"], a["off"], a["E"], a["R"], a["K"],
                                        a["N"], a["epi"], a["C"], a["H1"], a["prob"], a["ws"],
                                        a["nbytes"], None)

    def _grad(self, gg, **kw):
        a = dict(dC=1 << 12, Wq=1 << 13, Ws=1 << 14, off=1 << 15, E=4, R=100, K=128, N=256, epi=0,
                 H1=None, prob=None, dA=1 << 16, dot=None, ws=1 << 17, nbytes=1 << 30)
        a.update(kw)
        return gg.LIB.gg_f8_grouped_dgrad(a["dC"], a["Wq"], a["Ws"], a["off"], a["E"], a["R"],
                                          a["K"], a["N"], a["epi"], a["H1"], a["prob"], a["dA"],
                                          a["dot"], a["ws"], a["nbytes"], None)

    @pytest.mark.parametrize("kw,code", [
        (dict(A=None), 1), (dict(Wq=None), 1), (dict(Ws=None), 1), (dict(off=None), 1),
        (dict(C=None), 1), (dict(ws=None), 1), (dict(E=0), 1), (dict(R=-1), 1), (dict(K=0), 1),
        (dict(N=-64), 1), (dict(epi=2), 1), (dict(epi=9), 1), (dict(H1=1 << 12), 1),
        (dict(prob=1 << 12), 1), (dict(K=96), 2), (dict(N=100), 2), (dict(E=1025), 2),
        (dict(epi=1, N=192), 2), (dict(A=4104), 3), (dict(Wq=8200), 3), (dict(Ws=16386), 3),
        (dict(C=65544), 3), (dict(epi=1, H1=4104), 3), (dict(epi=3, prob=4098), 3),
        (dict(off=32770), 3), (dict(ws=131076), 3), (dict(nbytes=256), 4),
        (dict(R=0x7FFFFFFF, N=1 << 22, E=1024), 2), (dict(R=0x7FFFFFFF - 100, N=64), 2),
        (dict(N=0x7FFFFFFF - 127, K=64), 2), (dict(N=64, K=0x7FFFFFFF - 63), 2)])
    def test_forward(self, gg, kw, code):
        assert self._fwd(gg, **kw) == code

    @pytest.mark.parametrize("kw,code", [
        (dict(dC=None), 1), (dict(dA=None), 1), (dict(Wq=None), 1), (dict(epi=1), 1),
        (dict(epi=2), 1), (dict(H1=1 << 12), 1), (dict(dot=1 << 12), 1), (dict(prob=1 << 12), 1),
        (dict(K=32), 2), (dict(N=65), 2),
        (dict(epi=2, H1=1 << 12, K=(1 << 30) - 64, N=64), 2), (dict(K=0x7FFFFFFF - 63, N=64), 2),
        (dict(dC=4100), 3), (dict(dA=65540), 3),
        (dict(epi=2, H1=4100), 3), (dict(epi=2, H1=1 << 12, dot=4112), 3), (dict(nbytes=300), 4)])
    def test_gradient(self, gg, kw, code):
        assert self._grad(gg, **kw) == code

    def test_workspace_counts_the_width(self, gg):
        L = gg.LIB
        need = L.gg_f8_workspace_size(100, 256)
        assert need == 256 + (4 * 2 * 100 + 255) // 256 * 256 + (100 * 256 + 255) // 256 * 256
        assert L.gg_f8_workspace_size(-1, 64) == L.gg_f8_workspace_size(1, 0) == 0
        assert self._grad(gg, nbytes=L.gg_f8_workspace_size(100, 256) - 1) == 4
        assert self._fwd(gg, nbytes=L.gg_f8_workspace_size(100, 128) - 1) == 4

    def test_codes_and_weights(self, gg):
        L = gg.LIB
        a = 1 << 12

        def gemm(Aq=a, As=a, K=128, epi=0, nbytes=256):
            return L.gg_f8_grouped_gemm(Aq, As, a, a, a, 4, 10, K, 256, epi, a, None, None, a,
                                        nbytes, None)
        assert gemm(Aq=None) == gemm(As=None) == gemm(epi=4) == 1
        assert gemm(K=100) == 2 and gemm(As=a + 2) == 3 and gemm(nbytes=255) == 4

        def weight(W=a, E=2, N=64, K=64, Wq=a, Ws=a):
            return L.gg_f8_prepare_weight(W, E, N, K, Wq, Ws, None)
        assert weight(W=None) == weight(E=0) == weight(Ws=None) == 1
        assert weight(K=65) == weight(E=1025) == weight(N=65535 * 128 + 64) == 2
        assert weight(W=a + 8) == weight(Wq=a + 4) == weight(Ws=a + 1) == 3

        def rows(src=a, T=4, K=64, ros=None, k=1, R=4, Q=a, S=a, ws=a, nbytes=256):
            return L.gg_f8_quantize_rows(src, T, K, ros, k, R, Q, S, ws, nbytes, None)
        assert rows(src=None) == rows(T=5) == rows(ros=a, k=33) == rows(ros=a, k=0) == 1
        assert rows(ws=None) == rows(T=-1) == 1
        assert rows(K=72) == 2 and rows(S=a + 2) == 3 and rows(nbytes=8) == 4

    def test_weights_too_wide_to_count(self, gg):
        a = 1 << 12
        for K in (0x7FFFFFFF - 63, 0x7FFFFFFF - 511):
            assert gg.LIB.gg_f8_prepare_weight(a, 1, 64, K, a, a, None) == 2

    def _layer(self, gg, backward=False, opt=(0, 0, 0), T=20, H=128, F=64, k=2, E=4, P=1, null=None,
               buf=None, nbytes=None, **kw):
        L, a = gg.LIB, 1 << 12
        b = gg.GGBuffers()
        assert L.gg_moe_buffers_bind(1 << 20, 1 << 40, 20, 128, 64, 2, 4, 1, ctypes.byref(b)) == 0
        for name, v in (buf or {}).items():
            setattr(b, name, v)
        names = ["dOut", "x", "prob"] if backward else ["x", "idx", "prob"]
        args = dict.fromkeys(names + ["W1q", "W1s", "W2q", "W2s"], a)
        tail = dict.fromkeys(["dX", "dprob"] if backward else ["out"], a)
        ws = dict(ws=a)
        for d in (args, tail, ws):
            d.update({n: v for n, v in kw.items() if n in d})
            d.update({n: None for n in d if n == null})
        need = L.gg_moe_f8_workspace_size(T, H, F, k, E, P) if nbytes is None else nbytes
        o = gg.GGOptions(*opt)
        f = L.gg_moe_mlp_bwd_f8 if backward else L.gg_moe_mlp_fwd_f8
        return f(*args.values(), T, H, F, k, E, P, ctypes.byref(o), *tail.values(),
                 ctypes.byref(b), ws["ws"], need, None)

    @pytest.mark.parametrize("backward", [False, True])
    @pytest.mark.parametrize("kw,code", [
        (dict(null="W1q"), 1), (dict(null="W1s"), 1), (dict(null="W2q"), 1), (dict(null="W2s"), 1),
        (dict(null="x", opt=(0, 2, 0)), 1), (dict(null="prob", opt=(0, 2, 0), back=True), 1),
        (dict(null="out", fwd=True), 1), (dict(null="dOut", back=True), 1),
        (dict(null="dX", back=True), 1), (dict(null="ws"), 1), (dict(opt=(0, 0, 1)), 1),
        (dict(opt=(2, 0, 0)), 1), (dict(opt=(0, 3, 0)), 1), (dict(T=-1), 1), (dict(P=0), 1),
        (dict(buf=dict(H1=None)), 1), (dict(buf=dict(rowdot=None)), 1), (dict(H=96), 2),
        (dict(F=32), 2), (dict(T=1 << 30, k=4, E=1, buf=dict(ws_bytes=1 << 60), nbytes=0), 2),
        (dict(buf=dict(dXp=(1 << 20) + 8)), 3), (dict(buf=dict(H1=(1 << 20) + 8)), 3),
        (dict(W1q=4104), 3), (dict(W2s=4098), 3), (dict(out=4104, fwd=True), 3),
        (dict(dX=4104, back=True), 3), (dict(ws=4104), 3), (dict(nbytes=255), 4)])
    def test_layer(self, gg, backward, kw, code):
        kw = dict(kw)
        only = {"back": True, "fwd": False}
        for name, side in only.items():
            if kw.pop(name, False) and side != backward:
                return
        assert self._layer(gg, backward, **kw) == code

    def test_layer_workspace(self, gg):
        L = gg.LIB
        rows = gg.r_cap(30, 2, 6, 16)
        assert L.gg_moe_f8_workspace_size(30, 128, 192, 2, 6, 16) == L.gg_f8_workspace_size(
            rows, 384)
        assert L.gg_moe_f8_workspace_size(30, 512, 192, 2, 6, 16) == L.gg_f8_workspace_size(
            rows, 512)
        assert L.gg_moe_f8_workspace_size(30, 0, 192, 2, 6, 16) == 0
        assert L.gg_moe_f8_workspace_size(1 << 30, 64, 64, 4, 1, 1) == 0

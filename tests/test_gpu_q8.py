"""GPU parity of the 8-bit expert products (gg_q8_*) with the integer oracle.

Codes and scales are compared exactly (the same fp32 operations). Products are exact integers, and
fp32 sums of them too below 2^24; above, an addition is off by at most 2^-23 of the running sum, so
an accumulator over K codes by at most (K / 16) 2^-23 of the sum of magnitudes. Then a few fp32
roundings (8 * 2^-24 of the value; the fast exponential and divide of the gate: 2^-18), and one
BF16 rounding (2^-9 of the value, 2^-8 allowed)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import q8 as qo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


def _f64(t):
    return t.double().cpu().numpy()


def _random(counts, N, K, spare, seed, lo=-127):
    """Codes and scales as another program may have made them."""
    r = np.random.default_rng(seed)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R = int(off[-1]) + spare
    Aq = r.integers(-127, 128, (R, K)).astype(np.int8)
    Wq = r.integers(lo, 128, (len(counts), N, K)).astype(np.int8)
    As = (r.random(R) * 1e-2).astype(np.float32)
    Ws = ((r.random((len(counts), N)) + 0.1) * 1e-3).astype(np.float32)
    return Aq, As, Wq, Ws, off


def _dev(*arrays):
    return [torch.from_numpy(a).cuda() for a in arrays]


def _check(got, Aq, As, Wq, Ws, off, alpha=0.0, prob=None):
    K = Aq.shape[1]
    n = int(off[-1])
    want = qo.grouped_gemm(Aq, As, Wq, Ws, off, alpha, prob)[:n]
    mag = qo.grouped_gemm(np.abs(Aq.astype(np.int16)), As, np.abs(Wq.astype(np.int16)), Ws, off)[:n]
    # exact sums where no partial sum can pass 2^24
    big = K * 127 * 128 > 2 ** 24
    acc = (K / 16) * 2.0 ** -23 * mag if big else 0.0 * mag
    if alpha:
        F = want.shape[1]
        v = qo.grouped_gemm(Aq, As, Wq, Ws, off)[:n]
        # d(act(g) u) <= |u| * 1.2 |dg| + |act(g)| |du|, |act(g)| <= |g|
        acc = acc[:, :F] * 1.2 * np.abs(v[:, F:]) + np.abs(v[:, :F]) * acc[:, F:]
        if prob is not None:
            acc = acc * np.asarray(prob, np.float64)[:n, None]
    tol = acc + (2.0 ** -8 + 2.0 ** -18) * np.abs(want) + 1e-30
    err = np.abs(_f64(got)[:n] - want)
    assert np.isfinite(want).all() and (err <= tol).all(), (err - tol).max()


CASES = [
    # counts, N, K, rows past the last expert's
    ([1], 64, 64, 0),
    ([0, 1, 0], 128, 128, 0),
    ([8, 0, 3, 1], 192, 320, 4),
    ([1] * 9, 256, 2048, 0),
    ([17, 0, 33, 9, 64], 320, 192, 0),
    ([130, 256, 1, 0, 300], 128, 1088, 7),
    ([500, 2], 640, 256, 0),
    ([0, 0], 64, 64, 3),
    ([5] * 60, 64, 128, 0),
    ([700], 384, 4096, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_plain_matches_oracle(gg, case):
    counts, N, K, spare = CASES[case]
    Aq, As, Wq, Ws, off = _random(counts, N, K, spare, 50 + case, lo=-128)
    dA, dS, dW, dT, dO = _dev(Aq, As, Wq, Ws, off)
    ws = gg.workspace(0, 1, len(counts), "cuda")
    C = torch.full((Aq.shape[0], N), 3.0, dtype=torch.bfloat16, device="cuda")
    gg.q8_grouped_gemm(dA, dS, dW, dT, dO, C=C, ws=ws)
    assert gg.read_status(ws) == 0 and (C[int(off[-1]):] == 3).all()
    _check(C, Aq, As, Wq, Ws, off)
    assert torch.equal(C, gg.q8_grouped_gemm(dA, dS, dW, dT, dO, C=C.clone(), ws=ws))


@pytest.mark.parametrize("case", [c for c in range(len(CASES)) if CASES[c][1] % 128 == 0])
@pytest.mark.parametrize("alpha", [1.0, 1.702])
@pytest.mark.parametrize("weighted", [False, True])
def test_gated_matches_oracle(gg, case, alpha, weighted):
    counts, N, K, spare = CASES[case]
    Aq, As, Wq, Ws, off = _random(counts, N, K, spare, 80 + case)
    prob = np.random.default_rng(1).random(Aq.shape[0]).astype(np.float32) if weighted else None
    epi = gg.GG_EPI_SWIGLU if alpha == 1.0 else gg.GG_EPI_QGEGLU
    dA, dS, dW, dT, dO = _dev(Aq, As, Wq, Ws, off)
    C = gg.q8_grouped_gemm(dA, dS, dW, dT, dO, epi,
                           prob_of_row=None if prob is None else torch.from_numpy(prob).cuda())
    assert C.shape == (Aq.shape[0], N // 2)
    _check(C, Aq, As, Wq, Ws, off, alpha, prob)


# few rows per expert on average, yet more in one than are multiplied in one go
HEAVY = [
    ([40] + [0] * 7, 192, 320, 0),
    ([0] * 20 + [21] + [1] * 11, 64, 64, 0),
    ([0, 100, 3, 0, 0, 9, 0, 0, 16], 128, 1088, 5),
    ([33] + [0] * 600 + [1, 0, 17], 64, 192, 2),
    ([1] + [0] * 1022 + [1], 128, 128, 0),
]


@pytest.mark.parametrize("case", range(len(HEAVY)))
def test_one_expert_with_most_of_few_rows(gg, case):
    counts, N, K, spare = HEAVY[case]
    Aq, As, Wq, Ws, off = _random(counts, N, K, spare, 150 + case, lo=-128)
    dA, dS, dW, dT, dO = _dev(Aq, As, Wq, Ws, off)
    ws = gg.workspace(0, 1, len(counts), "cuda")
    C = torch.full((Aq.shape[0], N), 3.0, dtype=torch.bfloat16, device="cuda")
    gg.q8_grouped_gemm(dA, dS, dW, dT, dO, C=C, ws=ws)
    assert gg.read_status(ws) == 0 and (C[int(off[-1]):] == 3).all()
    _check(C, Aq, As, Wq, Ws, off)
    if N % 128 == 0:
        C = gg.q8_grouped_gemm(dA, dS, dW, dT, dO, gg.GG_EPI_SWIGLU, ws=ws)
        _check(C, Aq, As, Wq, Ws, off, 1.0)


@pytest.mark.parametrize("seed,gated", [(0, False), (1, True), (2, False), (3, True)])
def test_many_blocks_of_mixed_sizes(gg, seed, gated):
    # several work items per SM pair, from one token to 256, in every order
    r = np.random.default_rng(900 + seed)
    counts = r.choice([0, 1, 31, 33, 64, 70, 128, 129, 150, 190, 193, 224, 240, 256, 257, 300, 513],
                      48).tolist()
    N, K = (2048, 192) if gated else (1536, 320)
    Aq, As, Wq, Ws, off = _random(counts, N, K, 3, 950 + seed)
    dA, dS, dW, dT, dO = _dev(Aq, As, Wq, Ws, off)
    ws = gg.workspace(0, 1, len(counts), "cuda")
    epi = gg.GG_EPI_SWIGLU if gated else gg.GG_EPI_NONE
    C = gg.q8_grouped_gemm(dA, dS, dW, dT, dO, epi, ws=ws)
    assert gg.read_status(ws) == 0
    _check(C, Aq, As, Wq, Ws, off, 1.0 if gated else 0.0)


@pytest.mark.parametrize("K", [128, 256, 320, 512, 576, 1024, 1088, 2112, 4096, 8192])
def test_quantised_rows_of_every_width(gg, K):
    g = torch.Generator().manual_seed(K)
    x = torch.randn(19, K, generator=g) * torch.exp(torch.randn(19, 1, generator=g) * 4)
    x = x.bfloat16()
    x[7, K - 1] = 1e4
    x[9, K - 3] = float("-inf")
    Q, S = gg.q8_quantize_rows(x.cuda(), gg.workspace(0, 1, 1, "cuda"))
    q, s = qo.quantize_rows(x.float().numpy())
    np.testing.assert_array_equal(Q.cpu().numpy(), q)
    ok = np.isfinite(s)
    np.testing.assert_array_equal(S.cpu().numpy().view(np.int32)[ok], s.view(np.int32)[ok])
    assert not ok[9] and ok.sum() == 18 and np.isnan(S.cpu().numpy()[9])


@pytest.mark.parametrize("R,K", [(1, 64), (5, 192), (300, 2048), (33, 4160)])
def test_quantised_rows_match_bit_for_bit(gg, R, K):
    g = torch.Generator().manual_seed(R + K)
    x = torch.randn(R, K, generator=g) * torch.exp(torch.randn(R, 1, generator=g) * 4)
    if R > 4:
        x[1] = 0.0
        x[2] = 1e-38            # below the floor of the scale
        x[3, 5] = float("inf")
        x[4, 7] = float("nan")
    x = x.bfloat16()
    ws = gg.workspace(0, 1, 1, "cuda")
    Q, S = gg.q8_quantize_rows(x.cuda(), ws)
    q, s = qo.quantize_rows(x.float().numpy())
    np.testing.assert_array_equal(Q.cpu().numpy(), q)
    np.testing.assert_array_equal(S.cpu().numpy().view(np.int32)[np.isfinite(s)],
                                  s.view(np.int32)[np.isfinite(s)])
    np.testing.assert_array_equal(np.isnan(S.cpu().numpy()), np.isnan(s))
    if K % 64 == 0 and R >= 64:
        Wq, Ws = gg.q8_prepare_weight(x[:64].reshape(1, 64, K).cuda())
        np.testing.assert_array_equal(Wq[0].cpu().numpy(), q[:64])


def test_quantised_rows_through_the_permutes_map(gg):
    T, K, k, E = 37, 128, 3, 5
    g = torch.Generator().manual_seed(4)
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    idx = torch.randint(0, E, (T, k), generator=g, dtype=torch.int32).cuda()
    m = gg.permute(x, idx, torch.rand(T, k, generator=g).cuda(), E)
    Q, S = gg.q8_quantize_rows(x, m["ws"], m["row_of_slot"], k)
    Qp, Sp = gg.q8_quantize_rows(m["Xp"], m["ws"])
    assert torch.equal(Q, Qp) and torch.equal(S, Sp) and gg.read_status(m["ws"]) == 0
    bad = m["row_of_slot"].clone()
    bad[4], bad[9] = T * k, -1
    Q2, S2 = torch.zeros_like(Q), torch.zeros_like(S)
    gg.q8_quantize_rows(x, m["ws"], bad, k, Q=Q2, S=S2)
    assert gg.read_status(m["ws"]) == 18
    skipped = m["row_of_slot"][[4, 9]].long()
    Q[skipped], S[skipped] = 0, 0
    assert torch.equal(Q2, Q) and torch.equal(S2, S)


@pytest.mark.parametrize("counts", [[1], [3, 0, 2], [40, 1, 0, 90], [300, 200]])
def test_bf16_rows_in_one_call(gg, counts):
    g = torch.Generator().manual_seed(sum(counts))
    R, K, N = sum(counts), 256, 384
    A = torch.randn(R + 2, K, generator=g).bfloat16()
    W = (torch.randn(len(counts), N, K, generator=g) * 0.05).bfloat16()
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    Wq, Ws = gg.q8_prepare_weight(W.cuda())
    wq, wsc = qo.quantize_rows(W.float().numpy())
    np.testing.assert_array_equal(Wq.cpu().numpy(), wq)
    q, s = qo.quantize_rows(A.float().numpy())
    (dO,) = _dev(off)
    for epi, alpha in ((0, 0.0), (1, 1.0), (3, 1.702)):
        C = gg.q8_grouped_fwd(A.cuda(), Wq, Ws, dO, epi)
        _check(C, q, s, wq, wsc, off, alpha)


def test_rows_that_are_not_finite_give_nan_alone(gg):
    A = torch.randn(6, 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    A[1, 3], A[4, 0] = float("nan"), float("-inf")
    W = torch.randn(2, 64, 64, generator=torch.Generator().manual_seed(4)).bfloat16()
    Wq, Ws = gg.q8_prepare_weight(W.cuda())
    off = torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda")
    C = gg.q8_grouped_fwd(A.cuda(), Wq, Ws, off)
    assert torch.isnan(C).all(1).tolist() == [False, True, False, False, True, False]
    assert torch.isfinite(C[[0, 2, 3, 5]]).all()


def test_bad_offsets_write_nothing(gg):
    Aq, As, Wq, Ws, off = _random([10, 20], 64, 64, 0, 3)
    dA, dS, dW, dT = _dev(Aq, As, Wq, Ws)
    for bad in ([0, 20, 10], [1, 10, 30], [0, 10, 31]):
        C = torch.full((30, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ws = gg.workspace(0, 1, 2, "cuda")
        gg.q8_grouped_gemm(dA, dS, dW, dT, torch.tensor(bad, dtype=torch.int32).cuda(), C=C, ws=ws)
        assert gg.read_status(ws) == 17 and (C == 7).all()


def test_side_stream_and_graph_replay(gg):
    Aq, As, Wq, Ws, off = _random([20, 0, 70], 128, 128, 0, 5)
    A = torch.randn(90, 128, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    dW, dT, dO = _dev(Wq, Ws, off)
    ws = gg.q8_workspace(90, 128, "cuda")
    C = gg.q8_grouped_fwd(A, dW, dT, dO, ws=ws)
    want = C.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gg.q8_grouped_fwd(A, dW, dT, dO, C=C, ws=ws)
    C.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(C, want)


def test_host_refusals(gg):
    L = gg.LIB
    p, mis, ws = (ctypes.c_void_p(v) for v in (1 << 40, (1 << 40) + 8, 1 << 41))
    n0 = gg.launch_count()
    assert L.gg_q8_workspace_size(-1, 64) == 0 and L.gg_q8_workspace_size(4, 0) == 0
    assert L.gg_q8_workspace_size(100, 64) == 256 + 512 + 6400

    def gemm(A=p, s=p, W=p, t=p, off=p, E=4, R=64, K=64, N=128, epi=0, pr=None, C=p, w=ws, wb=256):
        return L.gg_q8_grouped_gemm(A, s, W, t, off, E, R, K, N, epi, pr, C, w, wb, None)

    def fwd(A=p, W=p, off=p, E=4, R=64, K=64, N=128, epi=0, pr=None, C=p, w=ws, wb=1 << 20):
        return L.gg_q8_grouped_fwd(A, W, p, off, E, R, K, N, epi, pr, C, w, wb, None)

    assert gemm(E=0) == 1 and gemm(R=-1) == 1 and gemm(epi=2) == 1 and gemm(epi=4) == 1
    assert gemm(A=None) == 1 and gemm(s=None) == 1 and gemm(W=None) == 1 and gemm(t=None) == 1
    assert gemm(off=None) == 1 and gemm(C=None) == 1 and gemm(pr=p) == 1
    assert gemm(K=96) == 2 and gemm(N=96) == 2 and gemm(E=1025) == 2 and gemm(N=192, epi=1) == 2
    assert gemm(A=mis) == 3 and gemm(W=mis) == 3 and gemm(C=mis) == 3 and gemm(t=mis) == 3
    assert gemm(w=None) == 1 and gemm(wb=16) == 4
    assert fwd(A=None) == 1 and fwd(K=96) == 2 and fwd(A=mis) == 3 and fwd(wb=256) == 4
    Q = L.gg_q8_quantize_rows
    assert Q(p, 8, 96, None, 1, 8, p, p, ws, 256, None) == 2
    assert Q(p, 9, 64, None, 1, 8, p, p, ws, 256, None) == 1     # more rows than places
    assert Q(p, 8, 64, p, 33, 64, p, p, ws, 256, None) == 1
    assert Q(None, 8, 64, None, 1, 8, p, p, ws, 256, None) == 1
    assert Q(mis, 8, 64, None, 1, 8, p, p, ws, 256, None) == 3
    W = L.gg_q8_prepare_weight
    assert W(p, 0, 64, 64, p, p, None) == 1 and W(p, 2, 64, 72, p, p, None) == 2
    assert W(p, 2, 64, 64, mis, p, None) == 3 and W(p, 2, 64, 64, None, p, None) == 1
    assert gg.launch_count() == n0
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    Wq = torch.zeros(2, 128, 64, dtype=torch.int8, device="cuda")
    Ws = torch.zeros(2, 128, device="cuda")
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        gg.q8_grouped_fwd(x, Wq.float(), Ws, off)
    with pytest.raises(TypeError):
        gg.q8_grouped_fwd(x.float(), Wq, Ws, off)
    with pytest.raises(ValueError):
        gg.q8_grouped_fwd(x, Wq, Ws[:1], off)
    with pytest.raises(ValueError):
        gg.q8_grouped_fwd(x[:, :32].contiguous(), Wq, Ws, off)


def test_empty_batch(gg):
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    Wq = torch.zeros(2, 128, 64, dtype=torch.int8, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert gg.q8_grouped_fwd(x, Wq, torch.zeros(2, 128, device="cuda"), off).shape == (0, 128)


@pytest.mark.parametrize("counts", [[5, 0, 3], [300, 0, 70]])
def test_scales_whose_product_leaves_the_fp32_range(gg, counts):
    # Scales of 1e-24 and 1e-19: their product, 1e-43, has six bits left in fp32, yet the results
    # (sums near 8e6, exact) are normal numbers. Scales of 1e25 and 1e20: their product is
    # infinite, the result of a row of zero codes is zero.
    K, N = 1024, 128
    Aq, As, Wq, Ws, off = _random(counts, N, K, 0, 300)
    Aq, Wq = np.abs(Aq) | 64, np.abs(Wq) | 64
    As, Ws = (As * 1e-22).astype(np.float32) + np.float32(1e-24), (Ws * 1e-16).astype(np.float32)
    assert (As.astype(np.float64).min() * Ws.min() < 2.0 ** -143)
    dA, dS, dW, dT, dO = _dev(Aq, As, Wq, Ws, off)
    _check(gg.q8_grouped_gemm(dA, dS, dW, dT, dO), Aq, As, Wq, Ws, off)
    Aq[1::2] = 0
    As[1::2], Ws[:] = 1e25, 1e20
    dA, dS, dT = _dev(Aq, As, Ws)
    C = gg.q8_grouped_gemm(dA, dS, dW, dT, dO)
    assert (C[1::2] == 0).all()
    _check(C, Aq, As, Wq, Ws, off)


@pytest.mark.parametrize("K", [64, 320, 1024])
@pytest.mark.parametrize("N", [128, 4096])
@pytest.mark.parametrize("epi,weighted", [(0, False), (1, False), (1, True), (3, False),
                                          (3, True)])
def test_a_rows_bits_do_not_depend_on_the_kernel(gg, K, N, epi, weighted):
    # the sizes choose the kernel by the rows there is room for: the same rows, with room for few
    # and for many, where every sum is exact (K * 127 * 127 < 2^24)
    counts = [9, 0, 40, 1, 33, 2, 0, 8, 64, 70]
    Aq, As, Wq, Ws, off = _random(counts, N, K, 4000, 500 + K)
    prob = np.random.default_rng(2).random(Aq.shape[0]).astype(np.float32)
    n = int(off[-1])
    assert n > 16 * len(counts)
    got = []
    for room, E in ((n + 4000, 10), (n, 60)):
        pad = np.zeros((E - 10, N, K), np.int8)
        offs = np.concatenate([off, np.full(E - 10, n, np.int32)])
        dev = _dev(Aq[:room], As[:room], np.concatenate([Wq, pad]),
                   np.concatenate([Ws, np.ones((E - 10, N), np.float32)]), offs, prob[:room])
        got.append(gg.q8_grouped_gemm(*dev[:5], epi, prob_of_row=dev[5] if weighted else None)[:n])
    assert torch.equal(got[0], got[1])

"""GPU parity of the E4M3 products with scales per block of 128.

Codes and scales are compared bit for bit. Products: two E4M3 codes multiply exactly in fp32. A
block of 128 is four MMAs of 32, each aligning its terms (2^-22 of their magnitudes) and truncating
one addition (2^-23): 1.5 * 2^-20 of the block's terms, 2^-19 allowed. Each block then costs the
rounding of its scales' product and of one fused addition, 2^-24 of the terms each. BF16 results
are rounded once more: 2^-8 of their value. In the gated activations the exponent a g is rounded
(2^-24 of it, and again times log2 e), which the exponential turns into 2^-22 |a g| of the sigmoid;
its quotient and the products are 2^-20."""

import math

import numpy as np
import pytest
import torch

from oracle import f8 as of

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ALPHA = {1: 1.0, 2: 1.0, 3: 1.702, 4: 1.702}


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _codes(t):
    return t.view(torch.uint8).cpu().numpy()


def _rows(R, K, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * std
    x[:, ::37] *= 9.0
    return x.bfloat16().cuda()


def _weight(gg, E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(E, N, K, generator=g) * 0.05 *
         torch.rand(E, N, 1, generator=g)).bfloat16().cuda()
    return gg.f8_prepare_weight(W)


def _offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()


def _sum_tol(mag, red):
    return (2.0 ** -19 + U * (2 + 2 * -(-red // 128))) * mag


def _act_tol(ag):
    return 2.0 ** -20 + 2.0 ** -22 * np.abs(ag)


def _near(got, want, tol, what):
    err = np.abs(got - want)
    assert np.isfinite(got).all(), what
    assert (err <= tol).all(), f"{what}: {float((err - tol).max())}, {int((err > tol).sum())}"


# ------------------------------------------------------------------ codes

@pytest.mark.parametrize("K", [64, 128, 192, 320, 1024, 2048, 4096, 4160, 8256])
def test_row_codes(gg, K):
    x = _rows(77, K, K)
    x[5] = 0
    x[6, ::3] = 1e-38
    x[7, 60], x[8, K - 1] = math.nan, -math.inf
    x[9] *= 1e30
    ws = gg.f8_workspace(0, 64, "cuda")
    Q, S = gg.f8_quantize_rows(x, ws)
    q, s = of.quantize_rows(x.float().cpu().numpy())
    np.testing.assert_array_equal(S.cpu().numpy(), s)
    np.testing.assert_array_equal(_codes(Q), q)


def test_row_codes_go_to_their_rows(gg):
    T, K, k, R = 50, 192, 3, 170
    x = _rows(T, K, 1)
    r = np.random.default_rng(1).permutation(R)[:T * k].astype(np.int32)
    r[7], r[20] = -1, R
    ws = gg.f8_workspace(0, 64, "cuda")
    Q = torch.full((R, K), 7.0, device="cuda").to(torch.float8_e4m3fn)
    S = torch.full((2, R), 3.0, device="cuda")
    gg.f8_quantize_rows(x, ws, torch.from_numpy(r).cuda(), k, R, Q, S)
    assert gg.read_status(ws) == 18
    q, s = of.quantize_rows(x.float().cpu().numpy())
    wq, wsc = np.full((R, K), int(_codes(Q)[-1, 0]), np.uint8), np.full((2, R), 3.0, np.float32)
    wq[:] = 0x4E  # 7.0
    for i, to in enumerate(r):
        if 0 <= to < R:
            wq[to], wsc[:, to] = q[i // k], s[:, i // k]
    np.testing.assert_array_equal(_codes(Q), wq)
    np.testing.assert_array_equal(S.cpu().numpy(), wsc)


@pytest.mark.parametrize("E,N,K", [(1, 64, 64), (3, 192, 320), (2, 256, 128), (1, 1856, 192)])
def test_weight_codes(gg, E, N, K):
    W = torch.randn(E, N, K, generator=torch.Generator().manual_seed(N)).bfloat16().cuda()
    W[0, :64, :64] = 0
    W[0, N - 1, K - 1] = math.inf
    Wq, Ws = gg.f8_prepare_weight(W)
    q, s = of.quantize_weight(W.float().cpu().numpy())
    np.testing.assert_array_equal(Ws.cpu().numpy(), s)
    np.testing.assert_array_equal(_codes(Wq), q)


# ------------------------------------------------------------------ products

COUNTS = [
    [1], [0, 5, 0, 0, 1], [33, 31, 32, 64], [255, 256, 257], [1000, 0, 3, 300], [2] * 40,
    [129, 513, 90], [20, 0] + [1] * 9,
]
SHAPES = [(64, 64), (128, 128), (256, 192), (320, 448), (576, 1024), (1088, 64)]


def _ids(x):
    return "x".join(map(str, x)) if len(x) < 6 else f"{len(x)}of{x[0]}"


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=_ids)
def test_forward_plain(gg, counts, N, K):
    E, spare = len(counts), 9
    R = sum(counts) + spare
    x, off = _rows(R, K, 1), _offsets(counts)
    Wq, Ws = _weight(gg, E, N, K, 2)
    ws = gg.f8_workspace(R, K, "cuda")
    C = torch.full((R, N), 5.0, dtype=torch.bfloat16, device="cuda")
    gg.f8_grouped_fwd(x, Wq, Ws, off, C=C, ws=ws)
    assert gg.read_status(ws) == 0
    q, s = of.quantize_rows(x.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy())
    n = R - spare
    _near(_np(C)[:n], y[:n], _sum_tol(mag[:n], K) + 2.0 ** -8 * np.abs(y[:n]), "C")
    assert (C[n:] == 5.0).all()
    # the same from codes
    Q, S = gg.f8_quantize_rows(x, ws)
    got = gg.f8_grouped_gemm(Q, S, Wq, Ws, off)
    np.testing.assert_array_equal(_np(got)[:n], _np(C)[:n])


@pytest.mark.parametrize("epi", [1, 3])
@pytest.mark.parametrize("keep,weighted", [(True, True), (False, False), (True, False)])
@pytest.mark.parametrize("N,K", [(128, 64), (256, 192), (384, 320), (640, 1024)])
@pytest.mark.parametrize("counts", [[1], [0, 33, 300, 2], [257, 64, 0], [3, 0, 12, 1, 2, 1]],
                         ids=_ids)
def test_forward_gated(gg, counts, N, K, keep, weighted, epi):
    E, spare, F = len(counts), 5, N // 2
    R = sum(counts) + spare
    x, off = _rows(R, K, 3), _offsets(counts)
    Wq, Ws = _weight(gg, E, N, K, 4)
    prob = torch.rand(R, generator=torch.Generator().manual_seed(5)).cuda() if weighted else None
    H1 = torch.full((R, N), 5.0, dtype=torch.bfloat16, device="cuda") if keep else None
    C = torch.full((R, F), 5.0, dtype=torch.bfloat16, device="cuda")
    gg.f8_grouped_fwd(x, Wq, Ws, off, epi, prob_of_row=prob, C=C, H1_save=H1)
    q, s = of.quantize_rows(x.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy())
    n = R - spare
    y, tol = y[:n], _sum_tol(mag[:n], K)
    if keep:
        _near(_np(H1)[:n], y, tol + 2.0 ** -8 * np.abs(y), "H1")
        assert (H1[n:] == 5.0).all()
    g, u, tg, tu = y[:, :F], y[:, F:], tol[:, :F], tol[:, F:]
    p = _np(prob)[:n, None] if weighted else 1.0
    want = of.glu(g, u, ALPHA[epi]) * p
    # |act'| <= 1.13, |act| <= |g|
    bound = p * (1.13 * tg * (np.abs(u) + tu) + np.abs(g) * tu) + \
        (_act_tol(ALPHA[epi] * g) + 2.0 ** -8) * np.abs(want)
    _near(_np(C)[:n], want, bound + 1e-30, "C")
    assert (C[n:] == 5.0).all()


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=_ids)
def test_gradient_plain(gg, counts, N, K):
    E, spare = len(counts), 9
    R = sum(counts) + spare
    d, off = _rows(R, N, 6), _offsets(counts)
    Wq, Ws = _weight(gg, E, N, K, 7)
    dA = torch.full((R, K), 5.0, dtype=torch.bfloat16, device="cuda")
    gg.f8_grouped_dgrad(d, Wq, Ws, off, dA=dA)
    q, s = of.quantize_rows(d.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy(), grad=True)
    n = R - spare
    _near(_np(dA)[:n], y[:n], _sum_tol(mag[:n], N) + 2.0 ** -8 * np.abs(y[:n]), "dA")
    assert (dA[n:] == 5.0).all()


@pytest.mark.parametrize("epi", [2, 4])
@pytest.mark.parametrize("weighted,dots", [(True, True), (False, True), (True, False)])
@pytest.mark.parametrize("N,K", [(64, 64), (192, 128), (320, 384), (1024, 320)])
@pytest.mark.parametrize("counts", [[1], [0, 33, 300, 2], [257, 64, 0]], ids=_ids)
def test_gradient_gated(gg, counts, N, K, weighted, dots, epi):
    E, spare = len(counts), 5
    R = sum(counts) + spare
    d, off, H1 = _rows(R, N, 8), _offsets(counts), _rows(R, 2 * K, 9)
    Wq, Ws = _weight(gg, E, N, K, 10)
    prob = torch.rand(R, generator=torch.Generator().manual_seed(11)).cuda() if weighted else None
    dA = torch.full((R, 2 * K), 5.0, dtype=torch.bfloat16, device="cuda")
    rowdot = torch.full((R, gg.rowdot_stride(K)), 5.0, device="cuda") if dots else None
    gg.f8_grouped_dgrad(d, Wq, Ws, off, epi, H1=H1, prob_of_row=prob, dA=dA, rowdot=rowdot)
    q, s = of.quantize_rows(d.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy(), grad=True)
    n = R - spare
    y, tol = y[:n], _sum_tol(mag[:n], N)
    h = _np(H1)[:n]
    g, u, a = h[:, :K], h[:, K:], ALPHA[epi]
    p = _np(prob)[:n] if weighted else np.ones(n)
    dg, du, dot = of.glu_bwd(y, g, u, a, p)
    slope = np.abs(u) * np.abs(of.sigmoid(a * g) * (1 + a * g * (1 - of.sigmoid(a * g))))
    # in s (1 + a g (1 - s)) the sum cancels: its own terms' errors count, not the result's
    rel = _act_tol(a * g)
    rest = p[:, None] * np.abs(y * u) * of.sigmoid(a * g) * (rel + 2.0 ** -22) * \
        (1 + np.abs(a * g))
    _near(_np(dA)[:n, :K], dg, p[:, None] * tol * slope + rest + (rel + 2.0 ** -8) * np.abs(dg) +
          1e-30, "dg")
    act = np.abs(g * of.sigmoid(a * g))
    _near(_np(dA)[:n, K:], du, p[:, None] * tol * act + (rel + 2.0 ** -8) * np.abs(du) + 1e-30,
          "du")
    assert (dA[n:] == 5.0).all()
    if dots:
        blocks = gg.rowdot_blocks(K)
        got = _np(rowdot)
        assert (got[n:] == 5.0).all() and (got[:, blocks:] == 5.0).all()
        # 128 rounded additions of the block's terms beside the sums' own error
        term = (tol * act * np.abs(u)) + (rel + 128 * U) * np.abs(dot)
        for b in range(blocks):
            cols = slice(128 * b, 128 * b + 128)
            _near(got[:n, b], dot[:, cols].sum(1), term[:, cols].sum(1) + 1e-30, f"rowdot {b}")


def test_codes_made_elsewhere(gg):
    """Any codes and scales, the largest among them."""
    r = np.random.default_rng(12)
    R, N, K, E = 40, 128, 256, 2
    def codes(*shape):
        c = r.integers(0, 256, shape).astype(np.uint8)
        c[(c & 127) == 127] = 0x7E
        return torch.from_numpy(c).cuda().view(torch.float8_e4m3fn)
    Q, Wq = codes(R, K), codes(E, N, K)
    S = torch.from_numpy(r.uniform(-2, 2, (2, R)).astype(np.float32)).cuda()
    Ws = torch.from_numpy((10.0 ** r.uniform(-6, 3, (E, 1, 2))).astype(np.float32)).cuda()
    off = _offsets([15, 25])
    C = gg.f8_grouped_gemm(Q, S, Wq, Ws, off)
    y, mag = of.product(_codes(Q), S.cpu().numpy(), _codes(Wq), Ws.cpu().numpy(),
                        off.cpu().numpy())
    _near(_np(C), y, _sum_tol(mag, K) + 2.0 ** -8 * np.abs(y), "C")


def test_nonfinite_rows_stay_among_themselves(gg):
    R, N, K = 70, 192, 320
    x, off = _rows(R, K, 13), _offsets([30, 40])
    Wq, Ws = _weight(gg, 2, N, K, 14)
    clean = gg.f8_grouped_fwd(x, Wq, Ws, off)
    x[3, 200], x[30, 0], x[69, 319] = math.nan, math.inf, -math.inf
    got = gg.f8_grouped_fwd(x, Wq, Ws, off)
    bad = [3, 30, 69]
    assert torch.isnan(got[bad]).all()
    keep = [i for i in range(R) if i not in bad]
    assert torch.equal(got[keep], clean[keep])


def test_rows_behind_the_last_expert_may_hold_anything(gg):
    R, N, K = 300, 128, 128
    off = _offsets([200, 50])
    Wq, Ws = _weight(gg, 2, N, K, 15)
    x = _rows(R, K, 16)
    a = gg.f8_grouped_fwd(x, Wq, Ws, off)[:250].clone()
    x[250:] = math.nan
    C = torch.full((R, N), 5.0, dtype=torch.bfloat16, device="cuda")
    gg.f8_grouped_fwd(x, Wq, Ws, off, C=C)
    assert torch.equal(C[:250], a) and (C[250:] == 5.0).all()


@pytest.mark.parametrize("offsets", [[0, 5, 3], [1, 2, 4], [0, 2, 99], [0, -1, 4]])
def test_bad_offsets_are_reported(gg, offsets):
    off = torch.tensor(offsets, dtype=torch.int32).cuda()
    Wq, Ws = _weight(gg, 2, 64, 64, 17)
    ws = gg.f8_workspace(10, 64, "cuda")
    C = torch.full((10, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    gg.f8_grouped_fwd(_rows(10, 64, 18), Wq, Ws, off, C=C, ws=ws)
    assert gg.read_status(ws) == 17 and (C == 5.0).all()
    ws.zero_()
    gg.f8_grouped_dgrad(_rows(10, 64, 18), Wq, Ws, off, dA=C, ws=ws)
    assert gg.read_status(ws) == 17 and (C == 5.0).all()


def test_no_rows(gg):
    Wq, Ws = _weight(gg, 2, 128, 64, 19)
    off = _offsets([0, 0])
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert gg.f8_grouped_fwd(empty, Wq, Ws, off).shape == (0, 128)
    C = torch.full((4, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    gg.f8_grouped_fwd(_rows(4, 64, 20), Wq, Ws, off, C=C)
    assert (C == 5.0).all()


@pytest.mark.parametrize("counts", [[3, 1, 0, 8], [500, 700, 3, 0]], ids=_ids)
def test_captured_and_repeated_calls_give_the_same_bits(gg, counts):
    R, N, K = sum(counts), 256, 320
    x, off = _rows(R, K, 21), _offsets(counts)
    d, H1 = _rows(R, N, 22), _rows(R, 2 * K, 23)
    Wq, Ws = _weight(gg, len(counts), N, K, 24)
    ws, ws2 = gg.f8_workspace(R, K, "cuda"), gg.f8_workspace(R, N, "cuda")
    C = torch.zeros((R, N // 2), dtype=torch.bfloat16, device="cuda")
    dA = torch.zeros((R, 2 * K), dtype=torch.bfloat16, device="cuda")
    rowdot = torch.zeros((R, gg.rowdot_stride(K)), device="cuda")

    def both():
        gg.f8_grouped_fwd(x, Wq, Ws, off, 1, C=C, ws=ws)
        gg.f8_grouped_dgrad(d, Wq, Ws, off, 2, H1=H1, dA=dA, rowdot=rowdot, ws=ws2)

    both()
    first = [t.clone() for t in (C, dA, rowdot)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        for t in (C, dA, rowdot):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, w in zip((C, dA, rowdot), first):
            assert torch.equal(t, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for t in (C, dA, rowdot):
            t.zero_()
        both()
    side.synchronize()
    for t, w in zip((C, dA, rowdot), first):
        assert torch.equal(t, w)


def test_many_experts_and_items(gg):
    """More work items than clusters, every one with several steps."""
    r = np.random.default_rng(25)
    counts = r.integers(0, 700, 60).tolist()
    R, N, K = sum(counts), 576, 448
    x, off = _rows(R, K, 26), _offsets(counts)
    Wq, Ws = _weight(gg, 60, N, K, 27)
    C = gg.f8_grouped_fwd(x, Wq, Ws, off)
    q, s = of.quantize_rows(x.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy())
    _near(_np(C), y, _sum_tol(mag, K) + 2.0 ** -8 * np.abs(y), "C")
    d = _rows(R, N, 28)
    dA = gg.f8_grouped_dgrad(d, Wq, Ws, off)
    q, s = of.quantize_rows(d.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy(), grad=True)
    _near(_np(dA), y, _sum_tol(mag, N) + 2.0 ** -8 * np.abs(y), "dA")


@pytest.mark.parametrize("N,K", [(64, 1024), (192, 3904), (128, 64)])
def test_row_sums_of_items_side_by_side(gg, N, K):
    """Items of different heights, one after the other: the two halves of a block's tokens are
    summed by warps that need not be at the same item."""
    counts = [100, 40, 128, 33, 65, 1, 97, 64] * 6
    R = sum(counts)
    d, H1, off = _rows(R, N, 46), _rows(R, 2 * K, 47, 0.7), _offsets(counts)
    p = torch.rand(R, generator=torch.Generator().manual_seed(48)).cuda()
    Wq, Ws = _weight(gg, len(counts), N, K, 49)
    blocks, stride = gg.rowdot_blocks(K), gg.rowdot_stride(K)
    got = []
    for _ in range(10):
        rowdot = torch.zeros((R, stride), device="cuda")
        gg.f8_grouped_dgrad(d, Wq, Ws, off, 2, H1, p, rowdot=rowdot)
        got.append(rowdot[:, :blocks])
    assert all(torch.equal(g, got[0]) for g in got)
    q, s = of.quantize_rows(d.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy(), grad=True)
    act = np.abs(_np(H1)[:, :K]) * np.abs(_np(H1)[:, K:])
    _, _, dot = of.glu_bwd(y, _np(H1)[:, :K], _np(H1)[:, K:])
    tol = _sum_tol(mag, N) * act + (2 * _act_tol(_np(H1)[:, :K]) + K * U) * np.abs(y) * act
    _near(_np(got[0]).sum(axis=1), dot.sum(axis=1), tol.sum(axis=1), "rowdot")


@pytest.mark.parametrize("most", [2, 12, 300])
def test_most_experts(gg, most):
    """1024 experts, some empty: the few-row kernel and both of the other's orientations."""
    r = np.random.default_rng(most)
    counts = r.integers(0, most, 1024)
    counts[[0, 1023]] = 0, most
    R, N, K = int(counts.sum()), 128, 192
    x, off = _rows(R, K, 40), _offsets(counts)
    Wq, Ws = _weight(gg, 1024, N, K, 41)
    C = gg.f8_grouped_fwd(x, Wq, Ws, off)
    q, s = of.quantize_rows(x.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy())
    _near(_np(C), y, _sum_tol(mag, K) + 2.0 ** -8 * np.abs(y), "C")
    d = _rows(R, N, 42)
    dA = gg.f8_grouped_dgrad(d, Wq, Ws, off)
    q, s = of.quantize_rows(d.float().cpu().numpy())
    y, mag = of.product(q, s, _codes(Wq), Ws.cpu().numpy(), off.cpu().numpy(), grad=True)
    _near(_np(dA), y, _sum_tol(mag, N) + 2.0 ** -8 * np.abs(y), "dA")


def test_two_streams_with_workspaces_of_their_own(gg):
    """Two calls under way at once, each with its own workspace and result."""
    counts = [700, 0, 300, 24]
    R, N, K = sum(counts), 512, 1024
    off, (Wq, Ws) = _offsets(counts), _weight(gg, 4, N, K, 43)
    xs = [_rows(R, K, 44), _rows(R, K, 45)]
    want = [gg.f8_grouped_fwd(x, Wq, Ws, off) for x in xs]
    ws = [gg.f8_workspace(R, K, "cuda") for _ in xs]
    got = [torch.zeros_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                gg.f8_grouped_fwd(xs[i], Wq, Ws, off, C=got[i], ws=ws[i])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g, w)


def test_binding_refuses(gg):
    R, N, K = 10, 128, 64
    x, off = _rows(R, K, 29), _offsets([4, 6])
    Wq, Ws = _weight(gg, 2, N, K, 30)
    with pytest.raises(TypeError):
        gg.f8_grouped_fwd(x.float(), Wq, Ws, off)
    with pytest.raises(TypeError):
        gg.f8_grouped_fwd(x, Wq.view(torch.uint8), Ws, off)
    with pytest.raises(ValueError):
        gg.f8_grouped_fwd(x, Wq, Ws[:, :, :0], off)
    with pytest.raises(ValueError):
        gg.f8_grouped_fwd(x, Wq, Ws, off[:2])
    with pytest.raises(ValueError):
        gg.f8_grouped_fwd(x[:, ::2], Wq, Ws, off)
    with pytest.raises(ValueError):
        gg.f8_grouped_fwd(torch.cat([x, x], 1)[:, :K], Wq, Ws, off)
    with pytest.raises(ValueError):
        gg.f8_grouped_fwd(x, Wq, Ws, off, prob_of_row=torch.ones(R - 1, device="cuda"))
    with pytest.raises(ValueError):
        gg.f8_grouped_fwd(x, Wq, Ws, off.cpu())
    with pytest.raises(gg.GGError):
        gg.f8_grouped_fwd(x, Wq, Ws, off, ws=gg.f8_workspace(R - 5, K, "cuda"))
    with pytest.raises(gg.GGError):
        gg.f8_grouped_fwd(x, Wq, Ws, off, H1_save=torch.empty((R, N), dtype=torch.bfloat16,
                                                              device="cuda"))
    with pytest.raises(gg.GGError):
        gg.f8_grouped_dgrad(_rows(R, N, 31), Wq, Ws, off, gg.GG_EPI_SWIGLU_BWD)
    with pytest.raises(ValueError):
        gg.f8_grouped_dgrad(_rows(R, N, 31), Wq, Ws, off, gg.GG_EPI_SWIGLU_BWD,
                            H1=_rows(R, K, 32))

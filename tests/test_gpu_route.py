"""GPU parity of the router (gg_route, gg_route_bwd) with its 64-bit oracle.

Picks and counts are compared exactly. Probabilities are held to 1e-5 of their value: the
argument of the exponential is rounded once (up to 2^-24 of logits up to 30 apart, 2e-6), the
exponential, division and scaling round to a few units, and a sum of at most 1024 terms in 32
lanes adds at most 37 roundings of 2^-24 (2.2e-6). Gradients are held to 2e-5 of the sum of the
magnitudes of their terms, for the same reasons with two such factors, and BF16 ones to half a
unit in the last place (2^-9 of their value) more."""

import numpy as np
import pytest
import torch

from oracle import router as ro

pytestmark = pytest.mark.gpu

REL, GRAD_REL, BF16_REL, TINY = 1e-5, 2e-5, 2.0 ** -8, 1e-30
VARIANTS = [(sig, ren) for sig in (False, True) for ren in (False, True)]


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


def _logits(seed, T, E, dtype, masked=0, dead=0.0):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, E)) * 2
    if masked:
        x[:, rng.permutation(E)[:masked]] = -np.inf
    x[rng.random(T) < dead] = -np.inf
    t = torch.from_numpy(x).to(dtype).cuda()
    return t, t.double().cpu().numpy()


def _check_forward(gg, t, x, k, sig, ren, scale):
    T, E = x.shape
    r = gg.route(t, k, int(sig), ren, scale, counts=True, losses=True)
    f = ro.route_forward(x, k, sig, ren, scale)
    np.testing.assert_array_equal(r["idx"].cpu().numpy(), f["idx"])
    np.testing.assert_array_equal(r["counts"].cpu().numpy(), f["counts"])
    np.testing.assert_allclose(r["prob"].cpu().numpy(), f["prob"], rtol=REL, atol=TINY)
    np.testing.assert_allclose(r["losses"].cpu().numpy(), f["losses"], rtol=REL, atol=TINY)
    bare = gg.route(t, k, int(sig), ren, scale)  # without statistics: the same answers
    assert torch.equal(bare["idx"], r["idx"])
    np.testing.assert_allclose(bare["prob"].cpu().numpy(), f["prob"], rtol=REL, atol=TINY)
    return r, f


def _check_backward(gg, t, x, r, f, sig, ren, scale, seed):
    T, k = f["idx"].shape
    dprob = torch.randn(T, k, generator=torch.Generator().manual_seed(seed)).cuda()
    got = gg.route_bwd(t, r["idx"], dprob, int(sig), ren, scale, counts=r["counts"],
                       aux_coef=0.7, z_coef=0.3)
    want, mag = ro.route_backward(x, f["idx"], f["counts"], dprob.double().cpu().numpy(), sig, ren,
                                  scale, 0.7, 0.3)
    tol = GRAD_REL * mag + TINY
    if t.dtype == torch.bfloat16:
        tol = tol + BF16_REL * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("sig,ren", VARIANTS)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (7, 5, 5), (33, 32, 2), (300, 60, 4),
                                   (129, 257, 32), (64, 1024, 8), (5000, 64, 6)])
def test_matches_oracle(gg, T, E, k, sig, ren):
    for dtype in (torch.float32, torch.bfloat16):
        t, x = _logits(T + E + k, T, E, dtype)
        r, f = _check_forward(gg, t, x, k, sig, ren, 1.0 if k % 2 else 2.5)
        _check_backward(gg, t, x, r, f, sig, ren, 1.0 if k % 2 else 2.5, 3)


@pytest.mark.parametrize("sig,ren", VARIANTS)
def test_masked_experts_and_dead_rows(gg, sig, ren):
    # more picks than experts left in every row, and rows with none left
    for dtype in (torch.float32, torch.bfloat16):
        t, x = _logits(11, 200, 40, dtype, masked=37, dead=0.2)
        r, f = _check_forward(gg, t, x, 6, sig, ren, 1.0)
        assert (r["prob"][torch.isneginf(t).all(1)] == 0).all()
        _check_backward(gg, t, x, r, f, sig, ren, 1.0, 4)


def test_equal_logits_go_to_the_lower_id(gg):
    t = torch.tensor([[2.0, 7.0, 7.0, 2.0, 7.0], [0.0, -0.0, 0.0, -0.0, -1.0]]).cuda()
    r = gg.route(t, 4)
    assert r["idx"].tolist() == [[1, 2, 4, 0], [0, 1, 2, 3]]
    # many ties: BF16 logits of few values
    x = torch.randint(0, 4, (500, 96), generator=torch.Generator().manual_seed(1)).bfloat16()
    f = ro.route_forward(x.double().numpy(), 20)
    np.testing.assert_array_equal(gg.route(x.cuda(), 20)["idx"].cpu().numpy(), f["idx"])


def test_nan_and_infinities_keep_valid_ids(gg):
    t = torch.zeros(3, 70)
    t[0, 40] = float("nan")
    t[1, 50] = float("inf")
    t[2, 60] = torch.finfo(torch.float32).min
    for sig in (0, 1):
        r = gg.route(t.cuda(), 3, sig, counts=True, losses=True)
        assert r["idx"].tolist() == [[40, 0, 1], [50, 0, 1], [0, 1, 2]]
        assert int(r["counts"].sum()) == 9
        assert torch.isfinite(r["prob"][2]).all()
        if not sig:
            assert torch.isnan(r["prob"][:2]).all()


@pytest.mark.parametrize("E", [29, 33, 64, 65, 70, 127, 128, 130, 200, 254, 256, 257, 300,
                               511, 512])
@pytest.mark.parametrize("k", [1, 3, 8, 16])
def test_picks_among_many_equal_logits(gg, E, k):
    # few values, infinities and NaN among them, in rows that start at any element; NaN is the
    # largest, and equals go to the lower id
    rng = np.random.default_rng(E * 100 + k)
    few = np.array([-np.inf, -2.0, -0.0, 0.0, 0.0, 1.0, 1.5, np.inf, np.nan])
    x = few[rng.integers(0, rng.integers(1, 10, (203, 1)), (203, E))]
    x[5] = -np.inf
    x[6] = np.nan
    x[7, E - 1] = 3.0
    rank = np.where(np.isnan(x), 1e6, np.clip(x, -1e5, 1e5))
    want = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    for dtype in (torch.float32, torch.bfloat16):
        for shift in (0, 1, 4):
            room = torch.empty(203 * E + shift, dtype=dtype, device="cuda")
            t = room[shift:].view(203, E)
            t.copy_(torch.from_numpy(x))
            r = gg.route(t, k, 1, counts=True)
            np.testing.assert_array_equal(r["idx"].cpu().numpy(), want)
            np.testing.assert_array_equal(r["counts"].cpu().numpy(),
                                          np.bincount(want.ravel(), minlength=E))
            assert torch.equal(gg.route(t, k, 1)["idx"], r["idx"])


@pytest.mark.parametrize("T,E,k", [(700, 70, 8), (700, 128, 8), (301, 200, 5), (300, 255, 8),
                                   (300, 256, 12), (40, 96, 16), (200, 512, 8), (201, 390, 10)])
def test_wide_rows_match_oracle(gg, T, E, k):
    for dtype in (torch.float32, torch.bfloat16):
        t, x = _logits(T + E + k, T, E, dtype, masked=E // 9, dead=0.05)
        for sig, ren in VARIANTS:
            r, f = _check_forward(gg, t, x, k, sig, ren, 1.5)
            _check_backward(gg, t, x, r, f, sig, ren, 1.5, 3)


def test_extreme_logits_stay_finite(gg):
    for dtype in (torch.float32, torch.bfloat16):
        lim = torch.finfo(dtype).max
        t = torch.tensor([[lim, -lim, 0.0, lim], [-lim] * 4], dtype=dtype).cuda()
        for sig, ren in VARIANTS:
            r = gg.route(t, 2, int(sig), ren)
            assert torch.isfinite(r["prob"]).all()
            d = gg.route_bwd(t, r["idx"], torch.ones(2, 2, device="cuda"), int(sig), ren)
            assert torch.isfinite(d).all()


def test_gradient_against_differences_of_the_kernel(gg):
    # The kernel's own losses and probabilities in FP32: a central difference of step 1/16
    # carries a truncation error below h^2/6 * max|f'''| ~ 1e-3 and a rounding error below
    # 2 * 1e-5 / (2 h) = 1.6e-4 per unit of the objective's terms.
    T, E, k = 4, 10, 3
    t, x = _logits(8, T, E, torch.float32)
    dprob = torch.randn(T, k, generator=torch.Generator().manual_seed(9)).cuda()
    h = 1.0 / 16
    for sig, ren in VARIANTS:
        r = gg.route(t, k, int(sig), ren, counts=True, losses=True)
        d = gg.route_bwd(t, r["idx"], dprob, int(sig), ren, counts=r["counts"], aux_coef=0.5,
                         z_coef=0.1).double().cpu().numpy()

        def f(dt, e):
            y = t.clone()
            y[:, e] += dt
            q = gg.route(y, k, int(sig), ren, counts=True, losses=True)
            if not torch.equal(q["idx"], r["idx"]):
                return None  # a pick changed: the objective jumps there
            return q["prob"].double().cpu().numpy()

        for e in range(E):
            hi, lo = f(h, e), f(-h, e)
            if hi is None or lo is None:
                continue
            only, _ = ro.route_backward(x, r["idx"].cpu().numpy(), r["counts"].cpu().numpy(),
                                        np.zeros((T, k)), sig, ren, 1.0, 0.5, 0.1)
            fd = ((hi - lo) / (2 * h) * dprob.double().cpu().numpy()).sum(1) + only[:, e]
            assert np.abs(fd - d[:, e]).max() < 5e-3


def test_empty_batch_and_lone_outputs(gg):
    t = torch.empty(0, 16, device="cuda")
    r = gg.route(t, 2, counts=True, losses=True)
    assert r["counts"].tolist() == [0] * 16 and r["losses"].tolist() == [0.0, 0.0]
    assert gg.route_bwd(t, r["idx"], r["prob"]).shape == (0, 16)
    t, x = _logits(2, 40, 16, torch.float32)
    f = ro.route_forward(x, 2)
    only = gg.route(t, 2, counts=True)
    assert only["losses"] is None
    np.testing.assert_array_equal(only["counts"].cpu().numpy(), f["counts"])
    only = gg.route(t, 2, losses=True)
    np.testing.assert_allclose(only["losses"].cpu().numpy(), f["losses"], rtol=REL)


def test_in_place_gradient_bad_ids_and_repeatability(gg):
    t, x = _logits(21, 3000, 48, torch.bfloat16)
    r = gg.route(t, 4, counts=True, losses=True)
    again = gg.route(t, 4, counts=True, losses=True)
    for n in r:
        assert torch.equal(r[n], again[n])
    dprob = torch.randn(3000, 4, generator=torch.Generator().manual_seed(2)).cuda()
    d = gg.route_bwd(t, r["idx"], dprob, counts=r["counts"], aux_coef=0.1, z_coef=0.1)
    ws = gg.route_workspace(3000, 48, "cuda")
    buf = t.clone()
    gg.route_bwd(buf, r["idx"], dprob, counts=r["counts"], aux_coef=0.1, z_coef=0.1, dlogits=buf,
                 ws=ws)
    assert torch.equal(buf, d) and gg.read_status(ws) == 0
    # an id outside [0, E) adds nothing and is reported
    bad = r["idx"].clone()
    bad[17, 2], bad[18, 0] = 48, -1
    cut = dprob.clone()
    cut[17, 2], cut[18, 0] = 0.0, 0.0
    got = gg.route_bwd(t, bad, dprob, dlogits=torch.empty_like(t), ws=ws)
    want = gg.route_bwd(t, r["idx"], cut)
    assert gg.read_status(ws) == 16
    assert torch.equal(got, want)


def test_side_stream_and_graph_replay(gg):
    t, x = _logits(31, 700, 128, torch.float32)
    f = ro.route_forward(x, 8)
    ws = gg.route_workspace(700, 128, "cuda")
    r = gg.route(t, 8, counts=True, losses=True, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gg.route(t, 8, idx=r["idx"], prob=r["prob"], counts=r["counts"], losses=r["losses"], ws=ws)
    for n in r:
        r[n].zero_()
    g.replay()
    torch.cuda.synchronize()
    np.testing.assert_array_equal(r["idx"].cpu().numpy(), f["idx"])
    np.testing.assert_array_equal(r["counts"].cpu().numpy(), f["counts"])
    np.testing.assert_allclose(r["prob"].cpu().numpy(), f["prob"], rtol=REL)


@pytest.mark.parametrize("E", [8, 32, 33, 200, 257, 1024])
def test_losses_repeat_over_many_calls(gg, E):
    # the balance loss is put together from the shares of a cluster's blocks, some of which have
    # no column to sum: every call gives the same bits, behind other work or an empty queue
    t, x = _logits(41, 900, E, torch.float32)
    f = ro.route_forward(x, 4)
    ws = gg.route_workspace(900, E, "cuda")
    first = gg.route(t, 4, losses=True, counts=True, ws=ws)
    np.testing.assert_allclose(first["losses"].cpu().numpy(), f["losses"], rtol=REL)
    got = []
    for i in range(200):
        got.append(gg.route(t, 4, losses=True, counts=True, ws=ws))
        if i % 10 == 0:
            torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r["losses"], first["losses"]) and torch.equal(r["counts"],
                                                                         first["counts"])


@pytest.mark.parametrize("sig", [0, 1])
@pytest.mark.parametrize("E,k", [(6, 2), (60, 4), (200, 8), (400, 8), (600, 8), (70, 20)])
def test_a_nan_logit_makes_both_losses_nan(gg, E, k, sig):
    # whatever kernel the sizes choose
    for dtype in (torch.float32, torch.bfloat16):
        t, _ = _logits(51, 40, E, dtype)
        assert torch.isfinite(gg.route(t, k, sig, losses=True)["losses"]).all()
        t[17, E // 2] = float("nan")
        assert torch.isnan(gg.route(t, k, sig, losses=True)["losses"]).all()


@pytest.mark.parametrize("ren", [False, True])
@pytest.mark.parametrize("E,k", [(6, 2), (60, 4), (128, 8), (200, 8), (400, 8), (600, 8), (70, 20)])
def test_a_nan_logit_makes_the_rows_gradient_nan(gg, E, k, ren):
    # softmax: every share of the row depends on the NaN, also where the other experts are
    # switched off; the other rows' gradients, and a row with none left, stay as they are
    for dtype in (torch.float32, torch.bfloat16):
        t, _ = _logits(52, 40, E, dtype, dead=0.1)
        t[9] = float("-inf")
        t[9, E // 3] = float("nan")
        t[17, E - 1] = float("nan")
        t[23] = float("nan")
        t[31] = float("-inf")
        bad = torch.zeros(40, dtype=torch.bool, device="cuda")
        bad[[9, 17, 23]] = True
        r = gg.route(t, k, 0, ren)
        dprob = torch.randn(40, k, generator=torch.Generator().manual_seed(3)).cuda()
        assert torch.isnan(r["prob"][bad]).all()
        d = gg.route_bwd(t, r["idx"], dprob, 0, ren, z_coef=0.1)
        assert torch.isnan(d[bad]).all() and torch.isfinite(d[~bad]).all()
        assert (d[31] == 0).all()
        assert torch.isnan(gg.route_bwd(t, r["idx"], dprob, 0, ren)[bad]).all()
        # sigmoid scores of other columns do not depend on it: those of the losses do
        r = gg.route(t, k, 1, False)
        d = gg.route_bwd(t, r["idx"], dprob, 1, False)
        assert torch.equal(torch.isnan(d), torch.isnan(t))
        d = gg.route_bwd(t, r["idx"], dprob, 1, False, z_coef=0.1)
        assert torch.isnan(d[bad]).all() and torch.isfinite(d[~bad]).all()


# tokens enough that every block of the forward with and without statistics, and of the gradient,
# takes several turns, the last of them in part
@pytest.mark.parametrize("T,E,k", [(80003, 30, 3), (80003, 60, 4), (40009, 64, 6), (80003, 128, 8),
                                   (40007, 200, 8), (20011, 300, 8), (20011, 1024, 8),
                                   (20011, 90, 20)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sig,ren", [(False, False), (True, True)])
def test_many_turns_match_oracle(gg, T, E, k, dtype, sig, ren):
    t, x = _logits(T + E, T, E, dtype, masked=E // 9, dead=0.03)
    r, f = _check_forward(gg, t, x, k, sig, ren, 1.5)
    assert int(r["counts"].sum()) == T * k
    _check_backward(gg, t, x, r, f, sig, ren, 1.5, 5)
    # into the logits' own buffer: the same bits
    dprob = torch.randn(T, k, generator=torch.Generator().manual_seed(6)).cuda()
    args = dict(counts=r["counts"], aux_coef=0.7, z_coef=0.3)
    d = gg.route_bwd(t, r["idx"], dprob, int(sig), ren, 1.5, **args)
    gg.route_bwd(t, r["idx"], dprob, int(sig), ren, 1.5, dlogits=t, **args)
    assert torch.equal(t, d)

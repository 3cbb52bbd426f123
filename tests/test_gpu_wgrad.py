"""GPU parity of the grouped weight gradient (gg_grouped_wgrad) with float64.

Products of BF16 values are exact in fp32. A sum over n rows is taken as 16-row steps inside the
tensor core (at most 16 between two hand-overs to fp32 registers, each truncating to 2^-23 of the
running sum at worst), one rounded addition per 256 rows and one for the base, so an element is off
by at most 2^-23 (18 + n / 256) of the sum of its terms' magnitudes. A BF16 result is rounded once
more, to 2^-9 of its value (the tests allow 2^-8)."""

import ctypes

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


def _inputs(counts, N, K, spare, seed):
    g = torch.Generator().manual_seed(seed)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    R_cap = int(off[-1]) + spare
    dC = torch.randn(R_cap, N, generator=g).bfloat16().cuda()
    A = torch.randn(R_cap, K, generator=g).bfloat16().cuda()
    return dC, A, torch.from_numpy(off).cuda(), off


def _want(dC, A, off):
    """dB in float64 and, per element, the sum of its terms' magnitudes."""
    d, a = dC.double(), A.double()
    spans = list(zip(off[:-1].tolist(), off[1:].tolist()))
    dB = torch.stack([d[lo:hi].t() @ a[lo:hi] for lo, hi in spans])
    mag = torch.stack([d[lo:hi].abs().t() @ a[lo:hi].abs() for lo, hi in spans])
    return dB, mag


def _check(got, want, mag, off, base=None):
    n = torch.from_numpy(np.diff(off)).double().cuda()[:, None, None]
    if base is not None:
        want = want + base.double()
        mag = mag + base.double().abs()
    tol = 2.0 ** -23 * (18 + n / 256) * mag
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all() and (err <= tol).all(), float((err - tol).max())


CASES = [
    # counts, N, K, rows past the last expert's
    ([1], 64, 64, 0),
    ([0], 64, 64, 5),
    ([16, 0, 1, 0, 47], 64, 128, 0),
    ([63, 64, 65, 15, 17, 0], 128, 320, 70),
    ([300, 1, 500, 0, 129, 255, 256, 257], 320, 192, 3),
    ([5, 900], 768, 576, 0),
    ([31] * 40, 128, 64, 9),
    ([4000, 3], 256, 512, 0),
    ([0, 0, 0], 192, 320, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_base", [False, True])
def test_matches_float64(gg, case, dtype, with_base):
    counts, N, K, spare = CASES[case]
    dC, A, offsets, off = _inputs(counts, N, K, spare, 100 + case)
    base = None
    if with_base:
        base = torch.randn(len(counts), N, K, generator=torch.Generator().manual_seed(1))
        base = base.to(dtype).cuda()
    ws = gg.wgrad_workspace(len(counts), dC.shape[0], N, K, "cuda")
    got = gg.grouped_wgrad(dC, A, offsets, base=base, out_dtype=dtype, ws=ws)
    want, mag = _want(dC, A, off)
    _check(got, want, mag, off, base)
    assert got.dtype == dtype and gg.read_status(ws) == 0
    again = gg.grouped_wgrad(dC, A, offsets, base=base, out_dtype=dtype, ws=ws)
    assert torch.equal(got, again)
    if with_base:  # accumulating in place: the same bits
        gg.grouped_wgrad(dC, A, offsets, base=base, dB=base, ws=ws)
        assert torch.equal(base, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_other_experts_rows_do_not_leak(gg, dtype):
    # infinities and NaN in a neighbour's rows and behind the last expert stay there
    counts = [37, 70, 0, 9]
    dC, A, offsets, off = _inputs(counts, 128, 192, 40, 7)
    want, mag = _want(dC, A, off)
    dC[37:107:3] = float("inf")
    A[40:107:5] = float("nan")
    dC[int(off[-1]):] = float("nan")
    A[int(off[-1]):] = float("inf")
    got = gg.grouped_wgrad(dC, A, offsets, out_dtype=dtype)
    keep = [0, 2, 3]
    _check(got[keep], want[keep], mag[keep], np.concatenate([[0], np.cumsum([37, 0, 9])]))
    assert not torch.isfinite(got[1]).all()


def test_padding_rows_of_zeros_add_nothing(gg):
    counts, P = [5, 0, 33, 16], 16
    dC, A, offsets, off = _inputs([-(-c // P) * P for c in counts], 64, 64, 0, 9)
    for lo, c, hi in zip(off[:-1], counts, off[1:]):
        dC[int(lo) + c:int(hi)] = 0
    got = gg.grouped_wgrad(dC, A, offsets, out_dtype=torch.float32)
    want, mag = _want(dC, A, off)
    _check(got, want, mag, off)


def test_bad_offsets_write_nothing(gg):
    dC, A, offsets, off = _inputs([10, 20], 64, 64, 0, 3)
    for bad in ([0, 20, 10], [1, 10, 30], [0, 10, 31]):
        dB = torch.full((2, 64, 64), 7.0, device="cuda")
        ws = gg.wgrad_workspace(2, 30, 64, 64, "cuda")
        gg.grouped_wgrad(dC, A, torch.tensor(bad, dtype=torch.int32).cuda(), dB=dB, ws=ws)
        assert gg.read_status(ws) == 17 and (dB == 7).all()


def test_no_rows_at_all(gg):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    base = torch.randn(3, 64, 64, device="cuda")
    assert (gg.grouped_wgrad(e, e, off, out_dtype=torch.float32) == 0).all()
    assert torch.equal(gg.grouped_wgrad(e, e, off, base=base), base)


def test_side_stream_and_graph_replay(gg):
    dC, A, offsets, off = _inputs([200, 0, 77], 128, 128, 0, 5)
    want, mag = _want(dC, A, off)
    ws = gg.wgrad_workspace(3, 277, 128, 128, "cuda")
    dB = gg.grouped_wgrad(dC, A, offsets, out_dtype=torch.float32, ws=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        gg.grouped_wgrad(dC, A, offsets, dB=dB, ws=ws)
    dB.zero_()
    g.replay()
    torch.cuda.synchronize()
    _check(dB, want, mag, off)


def test_gradient_against_differences_of_the_forward(gg):
    # The forward is linear in B, so a central difference has no truncation error: what is left is
    # the BF16 rounding of its outputs, 2^-9 of each, weighted by dC: at most 2^-9 sum |dC C| / h
    counts, N, K, h = [40, 0, 25], 64, 128, 0.5
    dC, A, offsets, off = _inputs(counts, N, K, 0, 13)
    B = torch.randn(3, N, K, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    dB = gg.grouped_wgrad(dC, A, offsets, out_dtype=torch.float32).double()
    for e, n, c in ((0, 3, 5), (0, 63, 127), (1, 0, 0), (2, 17, 64)):
        hi, lo = B.clone(), B.clone()
        hi[e, n, c] = (B[e, n, c].float() + h).bfloat16()
        lo[e, n, c] = (B[e, n, c].float() - h).bfloat16()
        step = float(hi[e, n, c].double() - lo[e, n, c].double())
        ch = gg.grouped_fwd(A, hi, offsets).double()[:, n]
        cl = gg.grouped_fwd(A, lo, offsets).double()[:, n]
        d = dC.double()[:, n]
        fd = float((d * (ch - cl)).sum()) / step
        tol = 2.0 ** -8 * float((d.abs() * (ch.abs() + cl.abs())).sum()) / step + 1e-6
        assert abs(fd - float(dB[e, n, c])) <= tol


def test_host_refusals(gg):
    L = gg.LIB
    p, mis, ws = (ctypes.c_void_p(v) for v in (1 << 40, (1 << 40) + 8, 1 << 41))
    n0 = gg.launch_count()

    def call(dC=p, A=p, off=p, E=4, R=128, N=64, K=64, dt=0, base=None, dB=p, w=ws, wb=1 << 30):
        return L.gg_grouped_wgrad(dC, A, off, E, R, N, K, dt, base, dB, w, wb, None)

    assert call(E=0) == 1 and call(R=-1) == 1 and call(N=0) == 1 and call(dt=2) == 1
    assert call(dC=None) == 1 and call(A=None) == 1 and call(off=None) == 1 and call(dB=None) == 1
    assert call(N=96) == 2 and call(K=100) == 2 and call(E=1025) == 2
    assert call(dC=mis) == 3 and call(A=mis) == 3 and call(base=mis) == 3 and call(dB=mis) == 3
    assert call(w=None) == 1 and call(wb=16) == 4
    assert gg.launch_count() == n0
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        gg.grouped_wgrad(x.float(), x, off)
    with pytest.raises(ValueError):
        gg.grouped_wgrad(x, x[:4], off)
    with pytest.raises(TypeError):
        gg.grouped_wgrad(x, x, off, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        gg.grouped_wgrad(x, x, off, base=torch.zeros(1, 64, 64, device="cuda"),
                         dB=torch.zeros(1, 64, 64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        gg.grouped_wgrad(x.t().contiguous().t(), x, off)


@pytest.mark.parametrize("with_base", [False, True])
@pytest.mark.parametrize("counts,N,K", [([65536], 4096, 4352), ([20000, 0, 8192, 8193, 30001], 2048, 2112),
                                        ([1048576], 256, 256)])
def test_long_bf16_sums_of_one_sign(gg, counts, N, K, with_base):
    # Sums of one sign over many rows, where truncations add up. A BF16 result's sums leave the
    # tensor core every 8192 rows, 512 additions that each lose up to 2^-23 of the running sum:
    # 2^-14 in all, next to which fp32 additions do not count; then half a BF16 step, 2^-9 to
    # 2^-8 of the value by its mantissa. The first case has too many blocks for slices, the last
    # cuts one block's rows into slices of more than 8192.
    g = torch.Generator(device="cuda").manual_seed(31)
    R = sum(counts)
    dC, A = ((torch.rand(R, n, generator=g, device="cuda") + 0.5).bfloat16() for n in (N, K))
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    base = None
    if with_base:
        base = (torch.rand(len(counts), N, K, generator=g, device="cuda") * 1e4).bfloat16()
    got = gg.grouped_wgrad(dC, A, torch.from_numpy(off).cuda(), base=base, out_dtype=torch.bfloat16)
    some = torch.randperm(N, generator=g, device="cuda")[:48]  # rows of dB
    a, d = A.double(), dC[:, some].double()
    for e, (lo, hi) in enumerate(zip(off[:-1].tolist(), off[1:].tolist())):
        want = d[lo:hi].t() @ a[lo:hi]
        if with_base:
            want = want + base[e, some].double()
        half = torch.exp2(torch.floor(torch.log2(want.clamp_min(1e-30))) - 8)
        err = (got[e, some].double() - want).abs()
        assert (err <= 2.0 ** -14 * want + half * (1 + 2.0 ** -14)).all(), float((err / half).max())


MIXED = [0, 1, 63, 64, 65, 100, 128, 256, 257, 300, 512, 600]


@pytest.mark.parametrize("N,K", [(576, 320), (320, 576), (64, 1088)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_work_items_of_mixed_sizes(gg, N, K, dtype):
    # several items per pair of SMs, in every order of lengths, experts without rows among them,
    # blocks that are cut off on both sides; with and without a base, and in place
    counts = np.random.default_rng(N + K).choice(MIXED, 90).tolist()
    dC, A, offsets, off = _inputs(counts, N, K, 5, 200 + N)
    want, mag = _want(dC, A, off)
    ws = gg.wgrad_workspace(len(counts), dC.shape[0], N, K, "cuda")
    _check(gg.grouped_wgrad(dC, A, offsets, out_dtype=dtype, ws=ws), want, mag, off)
    base = torch.randn(len(counts), N, K, generator=torch.Generator().manual_seed(1)).to(dtype)
    base = base.cuda()
    got = gg.grouped_wgrad(dC, A, offsets, base=base, ws=ws)
    _check(got, want, mag, off, base)
    gg.grouped_wgrad(dC, A, offsets, base=base, dB=base, ws=ws)
    assert torch.equal(base, got) and gg.read_status(ws) == 0


@pytest.mark.parametrize("counts,N,K", [([3000, 0, 2500, 7, 4000], 320, 320),
                                        ([64, 5000, 1, 5001, 0, 4999, 5063], 64, 448),
                                        ([1] * 30 + [3000, 2999, 0, 2000] + [2] * 9, 64, 64),
                                        ([9000, 8000, 100, 7000], 256, 320)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_several_experts_cut_into_slices(gg, counts, N, K, dtype):
    # experts that are cut next to ones that are not; the word behind the workspace's header
    # says how many steps of 64 rows a slice has
    dC, A, offsets, off = _inputs(counts, N, K, 3, 300 + N)
    want, mag = _want(dC, A, off)
    ws = gg.wgrad_workspace(len(counts), dC.shape[0], N, K, "cuda")
    got = gg.grouped_wgrad(dC, A, offsets, out_dtype=dtype, ws=ws)
    steps = int(ws[256:260].view(torch.int32).item())
    assert steps > 0 and sum(-(-c // 64) > steps for c in counts) >= 3
    _check(got, want, mag, off)
    assert torch.equal(got, gg.grouped_wgrad(dC, A, offsets, out_dtype=dtype, ws=ws))
    base = torch.randn(len(counts), N, K, generator=torch.Generator().manual_seed(1)).to(dtype)
    base = base.cuda()
    got = gg.grouped_wgrad(dC, A, offsets, base=base, ws=ws)
    _check(got, want, mag, off, base)
    gg.grouped_wgrad(dC, A, offsets, base=base, dB=base, ws=ws)
    assert torch.equal(base, got) and gg.read_status(ws) == 0

"""GPU parity of the optimizer step with the oracle: the kernel rounds every operation to fp32 in
the oracle's order, so results are compared bit for bit. The norm is compared with float64: squares
are added up 32 at a time in fp32 (32 roundings of 2^-24 of a sum of positive numbers, half of that
after the root), then in 64 bits, and rounded once: at most 2^-19."""

import math

import numpy as np
import pytest
import torch

from oracle import adamw as oa

pytestmark = pytest.mark.gpu

BETAS, EPS = (0.9, 0.95), 1e-8


@pytest.fixture(scope="module")
def gg():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


def _make(sizes, seed, w_bf16, g_bf16, shift=0):
    """Weights and gradients as views of one buffer each, `shift` elements from its start."""
    r = np.random.default_rng(seed)
    total = sum(sizes)

    def flat(std, bf16):
        x = torch.from_numpy((r.normal(size=total + shift) * std).astype(np.float32))
        return (x.bfloat16() if bf16 else x).cuda()[shift:]

    return list(flat(0.05, w_bf16).split(sizes)), list(flat(1e-2, g_bf16).split(sizes))


def _np(t):
    return t.detach().float().cpu().numpy().reshape(-1)


def _same(got, want, what):
    got, want = np.asarray(got), np.asarray(want)
    assert got.shape == want.shape
    same = (got == want) | (np.isnan(got) & np.isnan(want)) if got.dtype.kind == "f" else \
        got == want
    assert same.all(), f"{what}: {int((~same).sum())} of {same.size} differ"


def _codes(t):
    return t.view(torch.uint8).cpu().numpy().reshape(-1)


class Mirror:
    """The oracle's state of a list of tensors."""

    def __init__(self, weights, bits, w_bf16):
        self.w = [_np(t) for t in weights]
        self.bits, self.w_bf16 = bits, w_bf16
        if bits == 8:
            self.m = [(np.zeros(x.size, np.uint8), np.zeros(-(-x.size // 256), np.float32))
                      for x in self.w]
        else:
            self.m = [np.zeros(x.size, np.float32) for x in self.w]
        self.v = [x if bits == 32 else (x[0].copy(), x[1].copy()) for x in self.m]

    def step(self, grads, lr, t, decay, seed=0, grad_scale=1.0, lr_scale=1.0):
        for i, g in enumerate(grads):
            self.w[i], self.m[i], self.v[i] = oa.step(
                self.w[i], _np(g), self.m[i], self.v[i], lr=lr, t=t, beta1=BETAS[0],
                beta2=BETAS[1], eps=EPS, weight_decay=decay[i] if isinstance(decay, list)
                else decay, lr_scale=lr_scale, seed=seed, position=i, grad_scale=grad_scale,
                bits=self.bits, w_bf16=self.w_bf16)

    def check(self, opt, half=True):
        for i, w in enumerate(self.w):
            _same(_np(opt.weights[i]), w, f"w[{i}]")
            if self.bits == 8:
                for name in ("m", "v"):
                    codes, scale = getattr(self, name)[i]
                    _same(_codes(getattr(opt, name)[i]), codes, f"{name}[{i}] codes")
                    _same(_np(getattr(opt, name + "_scale")[i]), scale, f"{name}[{i}] scales")
            else:
                _same(_np(opt.m[i]), self.m[i], f"m[{i}]")
                _same(_np(opt.v[i]), self.v[i], f"v[{i}]")
            if opt.half is not None:
                _same(_np(opt.half[i]), _np(torch.from_numpy(w).bfloat16()), f"half[{i}]")


SIZES = [
    [1], [255], [256], [257], [2048, 2049], [1, 3, 255, 4097, 100000], [5] * 9,
    [7 + 13 * i for i in range(400)],  # more than one launch's list
    [0, 300, 0, 0, 513],
]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("w_bf16,g_bf16", [(False, False), (False, True), (True, True),
                                           (True, False)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_steps_match_the_oracle(gg, sizes, bits, w_bf16, g_bf16):
    weights, grads = _make(sizes, 1, w_bf16, g_bf16)
    half = None if w_bf16 else [torch.empty(n, dtype=torch.bfloat16, device="cuda")
                                for n in sizes]
    decay = [0.1 * (i % 3) for i in range(len(sizes))]
    opt = gg.AdamW(weights, grads, half=half, state_bits=bits, betas=BETAS, eps=EPS,
                   weight_decay=decay, seed=77)
    want = Mirror(weights, bits, w_bf16)
    for t in range(1, 4):
        opt.step(lr=3e-3)
        want.step(grads, 3e-3, t, decay, seed=77)
    want.check(opt)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 3])
def test_unaligned_arrays_give_the_same_bits(gg, bits, shift):
    sizes = [1000, 3000, 4097]
    weights, grads = _make(sizes, 2, False, True, shift)
    opt = gg.AdamW(weights, grads, state_bits=bits, betas=BETAS, eps=EPS)
    want = Mirror(weights, bits, False)
    opt.step(lr=1e-2)
    want.step(grads, 1e-2, 1, 0.0)
    want.check(opt)


@pytest.mark.parametrize("bits", [32, 8])
def test_extreme_values(gg, bits):
    """Zeros, denormals, huge and tiny magnitudes beside each other."""
    n = 1024
    r = np.random.default_rng(5)
    g = (r.normal(size=n) * 10.0 ** r.uniform(-30, 12, n)).astype(np.float32)
    g[:300] = 0.0
    g[300:310] = 1e-42
    weights, _ = _make([n], 3, False, False)
    grads = [torch.from_numpy(g).cuda()]
    opt = gg.AdamW(weights, grads, state_bits=bits, betas=BETAS, eps=EPS)
    want = Mirror(weights, bits, False)
    for t in (1, 2):
        opt.step(lr=1e-3)
        want.step(grads, 1e-3, t, 0.0)
    want.check(opt)
    assert torch.isfinite(weights[0]).all()


def test_nonfinite_gradient_reaches_its_cell_alone(gg):
    for bad in (math.nan, math.inf, -math.inf):
        weights, grads = _make([1024], 4, False, False)
        grads[0][700] = bad
        opt = gg.AdamW(weights, grads, state_bits=8, betas=BETAS, eps=EPS)
        want = Mirror(weights, 8, False)
        opt.step(lr=1e-3)
        want.step(grads, 1e-3, 1, 0.0)
        want.check(opt)
        fine = torch.isfinite(opt.m_scale[0]).cpu()
        assert fine.tolist() == [True, True, False, True]
        opt32 = gg.AdamW(*_make([1024], 4, False, False), betas=BETAS, eps=EPS)
        opt32.grads[0][700] = bad
        opt32.step(lr=1e-3)
        assert int((~torch.isfinite(opt32.weights[0])).sum()) == 1


def test_bf16_weights_nonfinite(gg):
    weights, grads = _make([512], 6, True, True)
    weights[0][3], weights[0][4] = math.inf, math.nan
    opt = gg.AdamW(weights, grads, betas=BETAS, eps=EPS)
    opt.step(lr=1e-3)
    assert weights[0][3].item() == math.inf and math.isnan(weights[0][4].item())
    assert int((~torch.isfinite(weights[0])).sum()) == 2


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf])
def test_a_scale_that_is_not_finite_skips_the_step(gg, bits, scale):
    weights, grads = _make([5000, 70], 7, False, False)
    half = [torch.zeros(n, dtype=torch.bfloat16, device="cuda") for n in (5000, 70)]
    opt = gg.AdamW(weights, grads, half=half, state_bits=bits)
    before = [t.clone() for t in weights]
    opt.step(lr=1.0, grad_scale=torch.tensor([scale], device="cuda"))
    for x, y in zip(weights, before):
        assert torch.equal(x, y)
    assert all(int(t.view(torch.uint8).sum()) == 0 for t in opt.m + opt.v + half)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_follows_lr_step_and_scale(gg, bits):
    sizes = [3000, 257]
    weights, grads = _make(sizes, 8, True, False)
    opt = gg.AdamW(weights, grads, state_bits=bits, betas=BETAS, eps=EPS, weight_decay=0.1, seed=9)
    want = Mirror(weights, bits, True)
    lr = torch.tensor([0.5], device="cuda")
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = torch.ones(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        opt.step(lr=lr, step=step, grad_scale=scale)
    for t, (rate, s) in enumerate([(0.25, 1.0), (2.0 ** -9, 0.5), (2.0 ** -7, 2.0)], 1):
        lr.fill_(rate)
        scale.fill_(s)
        for g in grads:
            g.mul_(1.5)
        graph.replay()
        want.step(grads, rate, t, 0.1, seed=9, grad_scale=s)
    torch.cuda.synchronize()
    want.check(opt)
    before = weights[0].clone()
    step.fill_(-5)  # counted up to -4: skipped
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(before, weights[0])


def test_runs_on_the_current_stream(gg):
    weights, grads = _make([200000], 10, False, False)
    opt = gg.AdamW(weights, grads, betas=BETAS, eps=EPS)
    want = Mirror(weights, 32, False)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        opt.step(lr=1e-3)
    side.synchronize()
    want.step(grads, 1e-3, 1, 0.0)
    want.check(opt)


def test_elements_beyond_32_bits(gg):
    """A BF16 tensor of more than 2^32 elements: the last cells' bits and offsets."""
    n = (1 << 32) + 700
    w = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-700:] = torch.randn(700, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    g[:256] = 1.0
    opt = gg.AdamW([w], [g], state_bits=8, betas=BETAS, eps=EPS, seed=4)
    opt.step(lr=1e-3)
    for lo, hi in ((0, 512), (n - 700 - 256, n)):  # both start at a cell
        assert lo % 256 == 0
        size = hi - lo
        key_at = lo // 256
        want = _step_at(_np(g[lo:hi]), key_at, size)
        _same(_np(w[lo:hi]), want[0], "w")
        _same(_codes(opt.m[0][lo:hi]), want[1][0], "m")
        _same(_codes(opt.v[0][lo:hi]), want[2][0], "v")
    assert int(torch.count_nonzero(w)) <= 700 + 256


def _step_at(g, first_cell, size):
    """The oracle on a slice of a tensor that starts at a cell."""
    real = oa.noise

    def noise(seed, step, position, n):
        key = oa.mix(oa.mix(oa.mix(seed) + step) + position)
        at = np.arange(n, dtype=np.uint64)
        return oa.mix(oa.mix(np.uint64(key) + np.uint64(first_cell) + at // 256) + at % 256)

    oa.noise = noise
    try:
        zero = (np.zeros(size, np.uint8), np.zeros(-(-size // 256), np.float32))
        return oa.step(np.zeros(size, np.float32), g, zero, zero, lr=1e-3, t=1, beta1=BETAS[0],
                       beta2=BETAS[1], eps=EPS, seed=4, bits=8, w_bf16=True)
    finally:
        oa.noise = real


# ------------------------------------------------------------------ the norm

@pytest.mark.parametrize("g_bf16", [False, True])
@pytest.mark.parametrize("sizes", [[1], [8192], [8193], [1, 3, 255, 4097, 100000], [3000000],
                                   [7 + 13 * i for i in range(1500)], [0, 5, 0],
                                   [8192] * 2, [8192 * 64], [8192 * 64 + 1], [700] * 64, [700] * 65,
                                   [1] + [20000] * 20, [9000] * 20 + [1] * 24],
                         ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("shift", [0, 1])
def test_norm(gg, sizes, g_bf16, shift):
    _, grads = _make(sizes, 11, False, g_bf16, shift)
    for max_norm in (0.0, 1e-3, 1e9):
        got = gg.grad_norm(grads, max_norm).cpu().double().numpy()
        want = oa.grad_norm([_np(t) for t in grads], max_norm)
        assert abs(got[0] - want[0]) <= 2.0 ** -19 * want[0]
        assert abs(got[1] - want[1]) <= 2.0 ** -19 * want[1]


def test_norm_of_nothing_and_of_zeros(gg):
    z = torch.zeros(100, device="cuda")
    assert gg.grad_norm([z], 1.0).tolist() == [0.0, 1.0]
    assert gg.grad_norm([torch.empty(0, device="cuda")], 1.0).tolist() == [0.0, 1.0]
    out = torch.full((2,), 7.0, device="cuda")
    ws = torch.zeros(gg.LIB.gg_grad_norm_workspace_size(0), dtype=torch.uint8, device="cuda")
    assert gg.LIB.gg_grad_norm(None, 0, 0, 1.0, out.data_ptr(), ws.data_ptr(), ws.numel(),
                               torch.cuda.current_stream().cuda_stream) == 0
    assert out.tolist() == [0.0, 1.0]


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("at", [0, 9000, 399999])
def test_norm_that_is_not_finite_skips_the_step(gg, bad, at):
    weights, grads = _make([400000], 12, False, True)
    grads[0][at] = bad
    opt = gg.AdamW(weights, grads)
    before = weights[0].clone()
    norm = gg.grad_norm(grads, 1.0)
    opt.step(lr=1.0, grad_scale=norm[1:])
    assert not math.isfinite(norm[0].item()) and math.isnan(norm[1].item())
    assert torch.equal(before, weights[0])


def test_norm_repeats_bitwise_and_captures(gg):
    _, grads = _make([700001, 33, 90000], 13, False, True)
    plan = gg.GradPlan(grads)
    out = torch.empty(2, device="cuda")
    first = gg.grad_norm(plan, 0.5).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gg.grad_norm(plan, 0.5, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    for g in grads:
        g.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], 2 * first[0])


# ------------------------------------------------------------------ the binding's checks

def test_binding_refuses(gg):
    f = torch.zeros(300, device="cuda")
    h = torch.zeros(300, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(300, device="cuda")
    with pytest.raises(ValueError):
        gg.AdamW([], [])
    with pytest.raises(ValueError):
        gg.AdamW([f], [g[:299]])
    with pytest.raises(ValueError):
        gg.AdamW([f], [g, g])
    with pytest.raises(TypeError):
        gg.AdamW([f], [g.half()])
    with pytest.raises(TypeError):
        gg.AdamW([f, h], [g, g.clone()])
    with pytest.raises(ValueError):
        gg.AdamW([f], [torch.zeros(300)])
    with pytest.raises(ValueError):
        gg.AdamW([torch.zeros(600, device="cuda")[::2]], [g])
    with pytest.raises(ValueError):
        gg.AdamW([f, f], [g, g])
    with pytest.raises(ValueError):
        gg.AdamW([f], [g], state_bits=16)
    with pytest.raises(ValueError):
        gg.AdamW([f], [g], m=[f.clone()])
    with pytest.raises(ValueError):
        gg.AdamW([f], [g], m=[f.to(torch.float8_e4m3fn)], v=[f.to(torch.float8_e4m3fn)])
    with pytest.raises(gg.GGError):
        gg.AdamW([h], [g], half=[h.clone()]).step(lr=1e-3)
    opt = gg.AdamW([f], [g])
    with pytest.raises(gg.GGError):
        opt.step(lr=1e-3, step=0)
    with pytest.raises(ValueError):
        opt.step(lr=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        opt.step(lr=1e-3, step=torch.zeros(1, device="cuda"))
    assert opt.t == 0
    with pytest.raises(ValueError):
        gg.GradPlan([])
    with pytest.raises(TypeError):
        gg.grad_norm([f, h])


@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_that_a_step_would_overwrite_are_refused(gg, bits):
    n, cells = 600, 3
    flat = torch.zeros(4 * n, device="cuda")
    w, g = flat[n:2 * n], flat[2 * n:3 * n]  # neighbours do not overlap
    half = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    opt = gg.AdamW([w, flat[:0]], [g, flat[:0]], half=[half, half[:0]], state_bits=bits)
    opt.set_grads([flat[:n], w[:0]])
    opt.set_grads([g, g[:0]])
    parts = [w, flat[n + 1:2 * n + 1], flat[1:n + 1], flat[2 * n - 1:3 * n - 1]]
    if bits == 32:
        parts += [opt.m[0], opt.v[0]]
    for x in parts:
        with pytest.raises(ValueError):
            opt.set_grads([x, x[:0]])
        assert opt.grads[0] is g and opt.table[0].g == g.data_ptr()
        with pytest.raises(ValueError):
            gg.AdamW([w], [x], **({} if bits == 8 else dict(m=[opt.m[0]], v=[opt.v[0]])))
    with pytest.raises(ValueError):
        opt.set_grads([half, half[:0]])
    if bits == 8:
        small = gg.AdamW([flat[:cells]], [g[:cells]], m=[opt.m[0][:cells]], v=[opt.v[0][:cells]],
                         m_scale=[opt.m_scale[0][:1]], v_scale=[opt.v_scale[0][:1]])
        with pytest.raises(ValueError):  # a gradient that begins with a cell's scale
            small.set_grads([opt.m_scale[0][:cells]])
    two = gg.AdamW([w, flat[:n]], [g, g], state_bits=bits)  # a gradient may serve two weights
    g.fill_(1.0)
    two.step(lr=0.5)
    assert torch.equal(w, flat[:n]) and float(w[0]) < 0


@pytest.mark.parametrize("g_bf16", [False, True])
def test_norm_bits_do_not_depend_on_where_an_array_starts(gg, g_bf16):
    dtype = torch.bfloat16 if g_bf16 else torch.float32
    run = 8 if g_bf16 else 4  # elements of a 16-byte load

    def norms(x):
        got = []
        for shift in (0, 1, run - 1):
            at = torch.zeros(x.numel() + shift, dtype=dtype, device="cuda")[shift:]
            at.copy_(x)
            got.append(gg.grad_norm([at], 1.0))
        return got

    # a 1 and 31 squares of 2^-26 in one thread's sum, where each of them is rounded away; apart
    # from the 1 they add up to two units of the last place of the result
    x = torch.zeros(8192, dtype=dtype, device="cuda")
    for i in range(32 // run):
        x[256 * run * i:256 * run * i + run] = 2.0 ** -13
    x[0] = 1.0
    a, *others = norms(x)
    assert a[0].item() == 1.0 and all(torch.equal(a, b) for b in others)
    r = np.random.default_rng(21)
    for n in [int(v) for v in r.integers(1, 60000, 40)] + [8192 * i for i in (1, 2, 7)] * 10:
        x = torch.from_numpy(r.normal(size=n).astype(np.float32)).to(dtype).cuda()
        a, *others = norms(x)
        assert all(torch.equal(a, b) for b in others), n

"""CPU checks of the optimizer step: the oracle against float64 and torch, the stochastic
rounding, and the refusals of gg_adamw_step and gg_grad_norm, which come before any launch."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import adamw as oa


@pytest.fixture(scope="module")
def gg():
    from moe_expert_grouped_gb300 import build

    build.build()
    import moe_expert_grouped_gb300.gg as mod

    return mod


def _data(n, seed=0):
    r = np.random.default_rng(seed)
    return [x.astype(np.float32) for x in (r.normal(size=n) * 0.05, r.normal(size=n) * 1e-2,
                                           r.normal(size=n) * 1e-3, r.normal(size=n) ** 2 * 1e-5)]


@pytest.mark.parametrize("t", [1, 2, 1000, 100000])
def test_oracle_is_adamw(t):
    """float64: torch's AdamW formula; its eps is added to the corrected root as here."""
    w, g, m, v = (torch.from_numpy(x.astype(np.float64)) for x in _data(1000))
    p = torch.nn.Parameter(w.clone())
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)
    p.grad = g.clone()
    opt.state[p] = dict(step=torch.tensor(float(t - 1)), exp_avg=m.clone(), exp_avg_sq=v.clone())
    opt.step()
    got = oa.step(*(x.numpy() for x in (w, g, m, v)), lr=3e-3, t=t, beta2=0.99, weight_decay=0.1,
                  dtype=np.float64)
    np.testing.assert_allclose(got[0], p.detach().numpy(), rtol=1e-11, atol=1e-15)


def test_oracle_fp32_is_near_float64():
    """Four rounded operations on m, five on v (2^-24 each, and the rounded constants); the
    update has those of m / 2 of v and six of its own."""
    a, b = (oa.step(*_data(4000), lr=1e-3, t=7, weight_decay=0.1, grad_scale=0.5, dtype=d)
            for d in (np.float32, np.float64))
    w, g, m, v = (x.astype(np.float64) for x in _data(4000))
    u = 2.0 ** -24
    assert (np.abs(a[1] - b[1]) <= 6 * u * (np.abs(m) + np.abs(g))).all()
    assert (np.abs(a[2] - b[2]) <= 8 * u * b[2]).all()
    assert (np.abs(a[0] - b[0]) <= 4 * u * np.abs(w) + 16 * u * 1e-3 * 40).all()


def test_codes_match_torch_and_float64():
    """Without random bits a code is cut; codes of exactly representable values stay."""
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(t, oa.E4M3.astype(np.float32))
    y = oa.E4M3[:127].astype(np.float32)
    for bits in (0, 1, 65535):
        b = np.full(127, bits, np.uint64)
        np.testing.assert_array_equal(oa.round_code(y, b), np.arange(127))
        np.testing.assert_array_equal(oa.round_code(y.astype(np.float64), b), np.arange(127))
    y = np.random.default_rng(1).uniform(0, 448, 5000).astype(np.float32)
    y[:2000] *= np.float32(2.0 ** -17)
    b = np.random.default_rng(2).integers(0, 65536, 5000).astype(np.uint64)
    # 16 random bits against 20 bits cut off: the same decision in float64
    np.testing.assert_array_equal(oa.round_code(y, b), oa.round_code(y.astype(np.float64), b))


def test_stochastic_rounding_is_unbiased():
    n = 1 << 18
    for y in (300.0, 1.3, 0.011, 0.0007):
        c = oa.round_code(np.full(n, y, np.float32), oa.noise(5, 1, 0, n) & np.uint64(0xFFFF))
        vals = oa.E4M3[c]
        width = vals.max() - vals.min()
        # the mean of n draws with a spread of at most width / 2, six deviations
        assert abs(vals.mean() - y) <= 6 * width / 2 / math.sqrt(n) + width / 65536


def test_small_moves_are_kept_on_average():
    """v decays by 0.1 % a step: rounding to nearest would never move it."""
    n, steps = 4096, 700
    v = oa.quantize(np.full(n, 0.01, np.float32), oa.noise(1, 0, 0, n) >> np.uint64(16), True)
    m = oa.quantize(np.zeros(n, np.float32), oa.noise(1, 0, 0, n) & np.uint64(0xFFFF), False)
    g = np.zeros(n, np.float32)
    g[::256] = 0.01  # holds each cell's scale
    w = np.zeros(n, np.float32)
    for t in range(1, steps + 1):
        w, m, v = oa.step(w, g, m, v, lr=0.0, t=t, bits=8, seed=3)
    got = np.square(oa.dequantize(*v))[np.arange(n) % 256 != 0].mean()
    want = 1e-4 * 0.999 ** steps
    assert abs(got / want - 1) < 0.1, got / want


class TestRefusals:
    """Every refusal comes before the device is looked at: the pointers are never used."""

    def _call(self, gg, n=1, tensor=None, **opt):
        o = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, w_dtype=0, g_dtype=0,
                 state_bits=32)
        o.update(opt)
        t = dict(w=1024, g=2048, m=4096, v=8192, n=100, lr_scale=1.0, weight_decay=0.0)
        t.update(tensor or {})
        table = (gg.GGAdamwTensor * max(n, 1))(*[gg.GGAdamwTensor(**t)] * max(n, 1))
        return gg.LIB.gg_adamw_step(table, n, ctypes.byref(gg.GGAdamwOptions(**o)), None)

    @pytest.mark.parametrize("opt", [
        dict(step=0), dict(step=-3), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0),
        dict(beta2=math.nan), dict(eps=0.0), dict(eps=-1e-8), dict(eps=math.nan),
        dict(eps=1e-60), dict(lr=math.nan), dict(lr=math.inf), dict(state_bits=16),
        dict(w_dtype=2), dict(g_dtype=-1)])
    def test_options(self, gg, opt):
        assert self._call(gg, **opt) == 1

    @pytest.mark.parametrize("tensor,code", [
        (dict(w=0), 1), (dict(g=0), 1), (dict(m=0), 1), (dict(v=0), 1), (dict(n=-1), 1),
        (dict(m_scale=4096), 1), (dict(weight_decay=math.nan), 1), (dict(lr_scale=math.inf), 1),
        (dict(n=1 << 40), 2), (dict(w=1026), 3), (dict(g=2049), 3), (dict(v=8194), 3),
        (dict(half=4097), 3)])
    def test_tensors(self, gg, tensor, code):
        assert self._call(gg, tensor=tensor) == code

    def test_eight_bits_need_scales(self, gg):
        assert self._call(gg, state_bits=8) == 1
        assert self._call(gg, state_bits=8, tensor=dict(m_scale=4096, v_scale=4098)) == 3

    def test_half_of_bf16_weights(self, gg):
        assert self._call(gg, w_dtype=1, tensor=dict(half=4096)) == 1

    def test_null_lists(self, gg):
        o = gg.GGAdamwOptions(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, state_bits=32)
        assert gg.LIB.gg_adamw_step(None, 1, ctypes.byref(o), None) == 1
        assert gg.LIB.gg_adamw_step(None, -1, ctypes.byref(o), None) == 1
        assert gg.LIB.gg_adamw_step(None, 0, None, None) == 1

    def test_norm(self, gg):
        need = gg.LIB.gg_grad_norm_workspace_size(1)
        t = (gg.GGGradTensor * 1)(gg.GGGradTensor(2048, 10))

        def call(t=t, n=1, dtype=0, max_norm=1.0, out=512, ws=1024, nbytes=need):
            return gg.LIB.gg_grad_norm(t, n, dtype, max_norm, out, ws, nbytes, None)

        assert gg.LIB.gg_grad_norm_workspace_size(-1) == 0
        assert call(n=-1) == call(dtype=3) == call(out=None) == call(t=None) == 1
        assert call(ws=None) == call(max_norm=math.nan) == 1
        assert call(nbytes=need - 1) == 4
        assert call(out=514) == call(ws=1025) == 3
        assert call(t=(gg.GGGradTensor * 1)(gg.GGGradTensor(2049, 10))) == 3
        assert call(t=(gg.GGGradTensor * 1)(gg.GGGradTensor(None, 10))) == 1
        assert call(t=(gg.GGGradTensor * 1)(gg.GGGradTensor(2048, -1))) == 1
        assert call(t=(gg.GGGradTensor * 1)(gg.GGGradTensor(2048, 1 << 40))) == 2

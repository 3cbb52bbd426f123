"""Cases that time the expert products on E4M3 weights scaled in blocks of 128, and the
optimizer step that trains them.

* ``fwd``    grouped linear layer on E4M3 weights with an fp32 scale for each 128 x 128 block;
  the rows are quantised on the way in, a scale for each 128 columns; plain or with a fused
  gated activation, whose input is kept where a backward pass follows;
* ``dgrad``  its input gradient on the same codes and scales, plain or with the gated
  activation's gradient and the row sums of the probabilities' gradient;
* ``adamw``  an AdamW step over many tensors, states in fp32 or in E4M3 with a scale for each
  256 elements, weights in fp32 (with a BF16 copy) or in BF16;
* ``norm``   the norm of all gradients and the factor that clips them.

``run`` computes them in plain torch operations in 32 bits, or, where ``own`` is set, by the
library's entry points.
"""

import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
TOP = 448.0                  # largest E4M3 value
AMAX_FLOOR = 2.0 ** -100     # smallest magnitude that a scale is made for
BLOCK = 128                  # columns, and rows of a weight, that share a scale
CELL = 256                   # elements of an optimizer state that share a scale
BETA1, BETA2, EPS = 0.9, 0.95, 1e-8
M32 = 0xFFFFFFFF


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token being decoded, first linear layer of the balanced 128-expert layer: latency
        dict(name="fwd one token fc1", op="fwd", R=8, E=128, N=1536, K=2048, P=1, gated=True,
             keep=False, skew=0.0, empty=0),
        # 64 sequences being decoded, second linear layer
        dict(name="fwd 64 tokens fc2", op="fwd", R=512, E=128, N=2048, K=768, P=1, gated=False,
             keep=False, skew=0.0, empty=0),
        # a chunk of prompt, skewed, widths that are no multiples of 128 or 256
        dict(name="fwd chunk 9001x2688x1856", op="fwd", R=9001, E=32, N=2688, K=1856, P=1,
             gated=False, keep=False, skew=0.8, empty=0),
        # a training batch of the balanced layer, first linear layer, its output kept
        dict(name="fwd train fc1", op="fwd", R=131072, E=128, N=1536, K=2048, P=1, gated=True,
             keep=True, skew=0.0, empty=0),
        # a toy layer's second linear layer: latency
        dict(name="dgrad small fc2", op="dgrad", R=1000, E=8, N=320, K=384, P=1, gated=True,
             skew=0.0, empty=1),
        # second linear layer on a skewed, padded batch, through the activation
        dict(name="dgrad skewed fc2", op="dgrad", R=32768, E=128, N=2048, K=768, P=256,
             gated=True, skew=1.2, empty=16),
        # a training batch of the balanced layer, first linear layer
        dict(name="dgrad train fc1", op="dgrad", R=131072, E=128, N=1536, K=2048, P=1,
             gated=False, skew=0.0, empty=0),
        # the example's layer: two expert weights and a router, latency
        dict(name="adamw small layer", op="adamw", sizes="1048576,524288,4096", bits=32, w="f32",
             g="f32", half=True, step=40),
        # the balanced layer's expert weights: FP32 masters and states, BF16 gradients and copies
        dict(name="adamw balanced fp32", op="adamw", sizes="402653184,201326592", bits=32,
             w="f32", g="bf16", half=True, step=1000),
        # a model's tensors of odd sizes, everything small: 8-bit states, BF16 weights
        dict(name="adamw odd 8-bit bf16", op="adamw", tensors=150, total=120000007, even=False,
             split=7, bits=8, w="bf16", g="bf16", half=False, step=100),
        # clipping the balanced layer's expert gradients
        dict(name="norm balanced bf16", op="norm", sizes="402653184,201326592", g="bf16"),
        # clipping a small model's tensors of odd sizes, fp32 gradients
        dict(name="norm odd f32", op="norm", tensors=60, total=3000017, even=False, split=3,
             g="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "dgrad", "adamw", "norm"])
    if op in ("adamw", "norm"):
        tensors = _log_int(rng, 1, 200)
        case = dict(op=op, tensors=tensors, total=max(tensors, _log_int(rng, 2000, 250000000)),
                    even=rng.random() < 0.4, split=rng.randrange(1 << 20),
                    g=rng.choice(["f32", "bf16"]))
        if op == "adamw":
            w = rng.choice(["f32", "f32", "bf16"])
            case.update(bits=rng.choice([8, 32]), w=w, half=w == "f32" and rng.random() < 0.7,
                        step=_log_int(rng, 1, 100000))
        return case
    E = _log_int(rng, 2, 128)
    N, K = 64 * _log_int(rng, 1, 64), 64 * _log_int(rng, 1, 64)
    R = _log_int(rng, 1, 131072)
    gated = rng.random() < 0.5
    if op == "fwd" and gated:
        N = (N + 64) // 128 * 128
    # no more products than the largest listed case, nor more weights
    E = max(1, min(E, 128 * 1536 * 2048 // (N * K)))
    R = max(1, min(R, 131072 * 1536 * 2048 // (N * K)))
    case = dict(op=op, R=R, E=E, N=N, K=K, P=rng.choice([1, 1, 16]), gated=gated,
                skew=rng.choice([0.0, 0.7, 1.2]), empty=rng.choice([0, E // 8]))
    if op == "fwd":
        case["keep"] = gated and rng.random() < 0.5
    return case


def _sizes(case):
    if "sizes" in case:
        return [int(n) for n in case["sizes"].split(",")]
    r = random.Random(case["split"])
    share = [r.lognormvariate(0.0, 1.5) for _ in range(case["tensors"])]
    got = [max(1, int(case["total"] * x / sum(share))) for x in share]
    return [-(-n // CELL) * CELL for n in got] if case["even"] else got


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _counts(case, seed):
    """Rows per expert: R pairs dealt at random, evenly or with Zipf-like weights, some experts
    without any."""
    r = random.Random(seed)
    E, R = case["E"], case["R"]
    w = [1.0 / (e + 1) ** case["skew"] for e in range(E)]
    r.shuffle(w)
    for e in r.sample(range(E), min(case["empty"], E - 1)):
        w[e] = 0.0
    c = [0] * E
    for e in r.choices(range(E), weights=w, k=R):
        c[e] += 1
    if case["skew"]:  # a token names an expert at most once: none has more than 1/8 of the pairs
        live = [e for e in range(E) if w[e] > 0]
        top = max(-(-R // 8), -(-R // len(live)))
        over = sum(max(n - top, 0) for n in c)
        c = [min(n, top) for n in c]
        for e in live:
            add = min(over, top - c[e])
            c[e] += add
            over -= add
    return c


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("adamw", "norm"):
        return _prepare_step(case, g)
    counts = _counts(case, seed)
    P, E, N, K = case["P"], case["E"], case["N"], case["K"]
    padded = [-(-n // P) * P for n in counts]
    off = [0]
    for n in padded:
        off.append(off[-1] + n)
    R_cap = case["R"] + E * (P - 1)
    live = [e for e in range(E) if padded[e]]
    s = dict(op=case["op"], E=E, N=N, K=K, R_cap=R_cap, gated=case["gated"],
             spans=list(zip(off[:-1], off[1:])), widest=max(padded),
             live=torch.tensor(live, device="cuda"),
             offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    pad = torch.ones(R_cap, dtype=torch.bool)
    for lo, n in zip(off, counts):
        pad[lo:lo + n] = False
    pad = pad.cuda()
    s["Wq"] = torch.cat([(torch.randn((max(1, E // 16), N, K), generator=g, device="cuda")
                          * 110.0).clamp_(-TOP, TOP).to(E4M3)
                         for _ in range(-(-E // max(1, E // 16)))])[:E].contiguous()
    s["Ws"] = 0.02 / 110 * (0.5 + torch.rand((E, -(-N // BLOCK), -(-K // BLOCK)), generator=g,
                                             device="cuda"))
    width = K if case["op"] == "fwd" else N
    s["x"] = _normal(g, (R_cap, width), 1.0)
    # a few columns are much larger than the rest, as in trained models
    s["x"][:, torch.randint(0, width, (max(1, width // 256),), generator=g, device="cuda")] *= 8
    s["x"][pad] = 0
    s["prob"] = torch.rand(R_cap, generator=g, device="cuda") if case["gated"] else None
    if case["op"] == "fwd":
        s["C"] = torch.zeros((R_cap, N // 2 if case["gated"] else N), dtype=torch.bfloat16,
                             device="cuda")
        s["H1"] = torch.zeros((R_cap, N), dtype=torch.bfloat16, device="cuda") \
            if case["keep"] else None
    else:
        s["H1"] = _normal(g, (R_cap, 2 * K), 1.0) if case["gated"] else None
        s["dA"] = torch.zeros((R_cap, 2 * K if case["gated"] else K), dtype=torch.bfloat16,
                              device="cuda")
        s["rowdot"] = torch.zeros((R_cap, (2 * -(-K // 256) + 7) // 8 * 8), device="cuda") \
            if case["gated"] else None
    return s


def _prepare_step(case, g):
    sizes = _sizes(case)
    total = sum(sizes)
    gtype = torch.float32 if case["g"] == "f32" else torch.bfloat16
    grad = torch.empty(total, dtype=gtype, device="cuda")
    grad.normal_(generator=g).mul_(3e-3)
    s = dict(op=case["op"], sizes=sizes, grad=grad, grads=list(grad.split(sizes)))
    if case["op"] == "norm":
        s["max_norm"] = 1.0
        return s
    wtype = torch.float32 if case["w"] == "f32" else torch.bfloat16
    w = torch.empty(total, dtype=wtype, device="cuda")
    w.normal_(generator=g).mul_(0.02)
    blocks = [-(-n // CELL) for n in sizes]
    count = torch.tensor(blocks, device="cuda")
    # of each block of CELL elements: its tensor and its place there
    tensor_of = torch.repeat_interleave(torch.arange(len(sizes), device="cuda"), count)
    first = torch.cumsum(count, 0) - count
    place = torch.arange(sum(blocks), device="cuda") - first[tensor_of]
    s.update(w=w, ws=list(w.split(sizes)), bits=case["bits"], step=case["step"], lr=1e-3,
             seed=int(torch.randint(0, 1 << 31, (1,), generator=g, device="cuda")),
             # biases and norms are not decayed: here, every third tensor
             decay=[0.0 if i % 3 == 2 else 0.1 for i in range(len(sizes))],
             tensor_of=tensor_of, place=place, cells=None, held=None,
             grad_scale=torch.full((1,), 0.7, device="cuda"),
             half=w.bfloat16() if case["half"] else None)
    s["halves"] = list(s["half"].split(sizes)) if case["half"] else None
    if any(n % CELL for n in sizes):  # elements of each block, and which exist
        n = torch.tensor(sizes, device="cuda")
        at = place[:, None] * CELL + torch.arange(CELL, device="cuda")
        s["held"] = at < n[tensor_of][:, None]
        s["cells"] = (at + (torch.cumsum(n, 0) - n)[tensor_of][:, None]).clamp_(max=total - 1)
    spread = torch.empty(total, device="cuda").normal_(generator=g)
    m = torch.empty(total, device="cuda").normal_(generator=g).mul_(1e-3)
    v = spread.mul_(0.7).exp_().mul_(2e-3).square_()
    if case["bits"] == 32:
        s.update(m=m, v=v, ms=list(m.split(sizes)), vs=list(v.split(sizes)))
    else:
        for name, x in (("m", m), ("v", v.sqrt_())):
            x = _grid(s, x)
            scale = x.abs().amax(1).clamp_min(AMAX_FLOOR) / TOP
            codes = _flat(s, (x / scale[:, None]).clamp_(-TOP, TOP).to(E4M3))
            s.update({name: codes, name + "s": list(codes.split(sizes)), name + "_scale": scale,
                      name + "_scales": list(scale.split(blocks))})
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    return {"fwd": _own_fwd if own else _plain_fwd,
            "dgrad": _own_dgrad if own else _plain_dgrad,
            "adamw": _own_adamw if own else _plain_adamw,
            "norm": _own_norm if own else _plain_norm}[state["op"]](state)


def _kept(s, name, make):
    """What a program keeps beside its buffers, made at the first pass."""
    if name not in s:
        s[name] = make()
    return s[name]


def _own_fwd(s):
    import moe_expert_grouped_gb300.gg as gg

    ws = _kept(s, "ws", lambda: gg.f8_workspace(s["R_cap"], s["K"], "cuda"))
    gg.f8_grouped_fwd(s["x"], s["Wq"], s["Ws"], s["offsets"],
                      gg.GG_EPI_SWIGLU if s["gated"] else gg.GG_EPI_NONE,
                      prob_of_row=s["prob"], C=s["C"], H1_save=s["H1"], ws=ws)
    return dict(C=s["C"], H1=s["H1"])


def _own_dgrad(s):
    import moe_expert_grouped_gb300.gg as gg

    ws = _kept(s, "ws", lambda: gg.f8_workspace(s["R_cap"], s["N"], "cuda"))
    gg.f8_grouped_dgrad(s["x"], s["Wq"], s["Ws"], s["offsets"],
                        gg.GG_EPI_SWIGLU_BWD if s["gated"] else gg.GG_EPI_NONE, H1=s["H1"],
                        prob_of_row=s["prob"], dA=s["dA"], rowdot=s["rowdot"], ws=ws)
    return dict(dA=s["dA"], rowdot=s["rowdot"])


def _own_adamw(s):
    import moe_expert_grouped_gb300.gg as gg

    more = {} if s["bits"] == 32 else dict(m_scale=s["m_scales"], v_scale=s["v_scales"])
    opt = _kept(s, "opt", lambda: gg.AdamW(
        s["ws"], s["grads"], half=s["halves"], m=s["ms"], v=s["vs"], **more,
        betas=(BETA1, BETA2), eps=EPS, weight_decay=s["decay"], seed=s["seed"]))
    opt.step(lr=s["lr"], step=s["step"], grad_scale=s["grad_scale"])
    return _step_outputs(s)


def _own_norm(s):
    import moe_expert_grouped_gb300.gg as gg

    plan = _kept(s, "plan", lambda: gg.GradPlan(s["grads"]))
    return gg.grad_norm(plan, s["max_norm"])


def _step_outputs(s):
    return {k: s[k] for k in ("w", "half", "m", "v", "m_scale", "v_scale")
            if s.get(k) is not None}


def _even(s):
    """Whether the live experts' rows fill most of a block padded to the widest expert's."""
    return s["widest"] * s["live"].numel() <= 3 * s["R_cap"]


def _block(s):
    """Row of each cell of the padded block [live experts][widest], and which cells hold one."""
    lo = s["offsets"][:-1].long()[s["live"]]
    n = s["offsets"][1:].long()[s["live"]] - lo
    at = torch.arange(s["widest"], device=lo.device)
    return (lo[:, None] + at).clamp_(max=s["R_cap"] - 1), at < n[:, None]


def _rows_as_held(x):
    """The values that the rows' codes and scales stand for."""
    x = x.float()
    R, width = x.shape
    more = -width % BLOCK
    if more:
        x = torch.cat([x, x.new_zeros((R, more))], 1)
    x = x.view(R, -1, BLOCK)
    a = x.abs().amax(2, keepdim=True).clamp_min(AMAX_FLOOR)
    return ((x * (TOP / a)).to(E4M3).float() * (a / TOP)).view(R, -1)[:, :width]


def _weight(s, e):
    """The values of the experts e's codes and scales, [n][N][K]."""
    scale = s["Ws"][e].repeat_interleave(BLOCK, 1)[:, :s["N"]]
    return s["Wq"].view(torch.uint8)[e].view(E4M3).float() * \
        scale.repeat_interleave(BLOCK, 2)[:, :, :s["K"]]


def _products(s, transposed):
    """Rows times their expert's weight (transposed: W^T), zero past the last expert's row."""
    x = _rows_as_held(s["x"])
    turn = (lambda w: w.transpose(-1, -2)) if transposed else (lambda w: w)
    y = x.new_zeros((s["R_cap"], s["N"] if transposed else s["K"]))
    if _even(s):
        rows, held = _block(s)
        y[rows[held]] = (x[rows] @ turn(_weight(s, s["live"])))[held]
    else:
        got = [x[lo:hi] @ turn(_weight(s, slice(e, e + 1)))[0]
               for e, (lo, hi) in enumerate(s["spans"]) if hi > lo]
        y[:s["spans"][-1][1]] = torch.cat(got)
    return y


def _plain_fwd(s):
    y = _products(s, True)
    if not s["gated"]:
        return dict(C=y.to(torch.bfloat16), H1=None)
    gate, up = y[:, :s["N"] // 2], y[:, s["N"] // 2:]
    C = gate / (1.0 + torch.exp(-gate)) * up * s["prob"][:, None]
    return dict(C=C.to(torch.bfloat16), H1=y.to(torch.bfloat16) if s["H1"] is not None else None)


def _plain_dgrad(s):
    y = _products(s, False)
    if not s["gated"]:
        return dict(dA=y.to(torch.bfloat16), rowdot=None)
    K = s["K"]
    gate, up = s["H1"][:, :K].float(), s["H1"][:, K:].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    d = y * s["prob"][:, None]
    dA = torch.cat([d * up * (sig * (1.0 + gate * (1.0 - sig))), d * (gate * sig)], 1)
    width = s["rowdot"].shape[1] * BLOCK
    dots = y.new_zeros((s["R_cap"], width))
    dots[:, :K] = y * (gate * sig * up)
    dots[s["spans"][-1][1]:] = 0
    dA[s["spans"][-1][1]:] = 0
    return dict(dA=dA.to(torch.bfloat16), rowdot=dots.view(s["R_cap"], -1, BLOCK).sum(2))


def _grid(s, x):
    """A flat tensor as [blocks][CELL], zeros behind each tensor's last element."""
    if s["cells"] is None:
        return x.view(-1, CELL)
    if x.dtype == E4M3:
        return (x.view(torch.uint8)[s["cells"]] * s["held"]).view(E4M3)
    return x[s["cells"]] * s["held"]


def _flat(s, x):
    if s["cells"] is None:
        return x.reshape(-1)
    return x.view(torch.uint8)[s["held"]].view(E4M3) if x.dtype == E4M3 else x[s["held"]]


def _mix(x):
    """A hash of 32 bits (two multiplications between shifts), on integers or int64 tensors."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def _random_bits(s):
    """32 random bits for each element: a hash of seed, step, tensor and element."""
    run_key = _mix(_mix(s["seed"]) + s["step"] & M32)
    key = _mix((run_key + s["tensor_of"]) & M32)
    key = _mix((key + s["place"]) & M32)
    return _mix((key[:, None] + torch.arange(CELL, device=key.device)) & M32)


def _round_codes(y, bits16):
    """E4M3 codes of y in [0, 448], rounded up with the probability of the part cut off."""
    small = y < 2.0 ** -6
    z = torch.where(small, y + 2.0 ** -6, y)
    t = (z.view(torch.int32) + (bits16 << 4)) >> 20
    return (t - torch.where(small, 968, 960)).clamp_(max=126)


def _plain_adamw(s):
    lr, t = s["lr"], s["step"]
    c1, c2 = lr / (1.0 - BETA1 ** t), 1.0 / math.sqrt(1.0 - BETA2 ** t)
    w = _grid(s, s["w"]).float()
    g = _grid(s, s["grad"]).float() * s["grad_scale"]
    m, v = _grid(s, s["m"]).float(), _grid(s, s["v"]).float()
    if s["bits"] == 8:
        m, v = m * s["m_scale"][:, None], (v * s["v_scale"][:, None]).square()
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + (g * g) * (1.0 - BETA2)
    r = v.sqrt()
    kept = torch.tensor([1.0 - lr * d for d in s["decay"]], device=w.device)
    w = w * kept[s["tensor_of"]][:, None] - (m * c1) / (r * c2 + EPS)
    noise = _random_bits(s) if s["bits"] == 8 or s["w"].dtype != torch.float32 else None
    if s["bits"] == 8:
        for x, name, bits16, least in ((m.abs(), "m", noise & 0xFFFF, 0),
                                       (r, "v", noise >> 16, (r > 0).to(torch.int32))):
            a = x.amax(1, keepdim=True).clamp_min(AMAX_FLOOR)
            code = _round_codes(x * (TOP / a), bits16.to(torch.int32))
            code = torch.maximum(code, torch.as_tensor(least, device=x.device, dtype=code.dtype))
            if name == "m":
                code = torch.where(m < 0, code | 128, code)
            s[name].copy_(_flat(s, code.to(torch.uint8).view(E4M3)))
            s[name + "_scale"].copy_((a / TOP)[:, 0])
    else:
        s["m"].copy_(_flat(s, m))
        s["v"].copy_(_flat(s, v))
    w = _flat(s, w)
    if s["w"].dtype == torch.float32:
        s["w"].copy_(w)
    else:
        up = _flat(s, _mix((noise + 0x9E3779B9) & M32) & 0xFFFF).to(torch.int32)
        s["w"].copy_(((w.view(torch.int32) + up) & ~0xFFFF).view(torch.float32))
    if s["half"] is not None:
        s["half"].copy_(w)
    return _step_outputs(s)


def _plain_norm(s):
    norm = s["grad"].float().square().sum(dtype=torch.float64).sqrt()
    return torch.stack([norm, (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)]).float()


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] in ("adamw", "norm"):
        n = sum(_sizes(case))
        b = n * (4 if case["g"] == "f32" else 2)
        if case["op"] == "norm":
            return {"bytes": b + 8, "flops": 2.0 * n}
        b += n * (8 if case["w"] == "f32" else 4) + n * (16 if case["bits"] == 32 else 4)
        if case["bits"] == 8:
            b += 16 * sum(-(-k // CELL) for k in _sizes(case))
        return {"bytes": b + (2 * n if case["half"] else 0), "flops": 16.0 * n}
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    live = E * (1.0 - (1.0 - 1.0 / E) ** R)  # experts that R pairs are expected to reach
    b = live * N * (K + 4 * -(-K // BLOCK) / BLOCK)
    if case["op"] == "fwd":
        out = (N // 2 if case["gated"] else N) + (N if case["keep"] else 0)
        b += 2 * R * (K + out)
    else:
        b += 2 * R * (N + K) if not case["gated"] else 2 * R * (N + 4 * K) + 4 * R * (K // 128 + 1)
    return {"bytes": b, "flops": 2.0 * R * N * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        norm = float(sum(x.double().square().sum() for x in s["grads"])) ** 0.5
        return torch.tensor([norm, min(1.0, s["max_norm"] / (norm + 1e-6))], dtype=torch.float64)
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_products(s)


def _exact_products(s):
    """Block by block of 128: sums of codes, then both scales."""
    fwd = s["op"] == "fwd"
    N, K = s["N"], s["K"]
    width, out = (K, N) if fwd else (N, K)
    y = torch.zeros((s["R_cap"], out), dtype=torch.float64, device="cuda")
    x32 = s["x"].float()
    spread = torch.arange(out, device="cuda") // BLOCK
    for b in range(0, width, BLOCK):
        part = x32[:, b:b + BLOCK]
        a = part.abs().amax(1).clamp_min(AMAX_FLOOR)  # a 32-bit number, as the codes are 8-bit
        codes = (part * (TOP / a)[:, None]).to(E4M3).double()
        scale = a.double() / TOP
        for e, (lo, hi) in enumerate(s["spans"]):
            if hi == lo:
                continue
            if fwd:
                w = s["Wq"][e][:, b:b + BLOCK].double().t()
                ws = s["Ws"][e][:, b // BLOCK].double()
            else:
                w = s["Wq"][e][b:b + BLOCK].double()
                ws = s["Ws"][e][b // BLOCK].double()
            y[lo:hi] += (codes[lo:hi] @ w) * ws[spread] * scale[lo:hi, None]
    if not s["gated"]:
        return dict(C=y, H1=None) if fwd else dict(dA=y, rowdot=None)
    p = s["prob"].double()[:, None]
    if fwd:
        gate, up = y[:, :N // 2], y[:, N // 2:]
        return dict(C=gate * torch.sigmoid(gate) * up * p, H1=y if s["H1"] is not None else None)
    gate, up = s["H1"].double().split(K, 1)
    sg = torch.sigmoid(gate)
    dA = torch.cat([y * p * up * (sg + gate * sg * (1 - sg)), y * p * gate * sg], 1)
    dot = y * gate * sg * up
    rows = torch.zeros(s["rowdot"].shape, dtype=torch.float64, device="cuda")
    for b in range(0, K, BLOCK):
        rows[:, b // BLOCK] = dot[:, b:b + BLOCK].sum(1)
    return dict(dA=dA, rowdot=rows)


def _exact_adamw(s):
    """Tensor by tensor; a code is a whole number of the steps of its binade."""
    out = {k: [] for k in _step_outputs(s)}
    lr, t = s["lr"], s["step"]
    gs = float(s["grad_scale"])
    for i, n in enumerate(s["sizes"]):
        w, g = s["ws"][i].double(), s["grads"][i].double() * gs
        blocks = -(-n // CELL)
        m, v = s["ms"][i].double(), s["vs"][i].double()
        if s["bits"] == 8:
            m = m * s["m_scales"][i].double().repeat_interleave(CELL)[:n]
            v = (v * s["v_scales"][i].double().repeat_interleave(CELL)[:n]) ** 2
        m = m + (1 - BETA1) * (g - m)
        v = v + (1 - BETA2) * (g * g - v)
        mean, root = m / (1 - BETA1 ** t), torch.sqrt(v / (1 - BETA2 ** t))
        w = w - lr * s["decay"][i] * w - lr * mean / (root + EPS)
        if s["half"] is not None:
            out["half"].append(w)
        if s["bits"] == 8 or s["w"].dtype != torch.float32:
            h = _mix(_mix(s["seed"]) + t & M32)
            at = torch.arange(n, device="cuda")
            h = _mix((_mix(h + i & M32) + at // CELL) & M32)
            h = _mix((h + at % CELL) & M32)
        if s["w"].dtype != torch.float32:
            u = (_mix((h + 0x9E3779B9) & M32) & 0xFFFF).double() / 65536
            w = _binade_floor(w.abs(), 7, -126, u) * torch.sign(w)
        out["w"].append(w)
        if s["bits"] == 32:
            out["m"].append(m)
            out["v"].append(v)
            continue
        for x, name, u in ((m, "m", h & 0xFFFF), (v.sqrt(), "v", h >> 16)):
            cells = torch.zeros(blocks * CELL, dtype=torch.float64, device="cuda")
            cells[:n] = x.abs()
            a = cells.view(-1, CELL).amax(1).clamp_min(AMAX_FLOOR)
            y = x.abs() * (TOP / a).repeat_interleave(CELL)[:n]
            code = _binade_floor(y, 3, -6, u.double() / 65536).clamp(max=TOP)
            if name == "v":
                code = torch.where(x > 0, code.clamp(min=2.0 ** -9), code)
            out[name].append(code * torch.sign(x))
            out[name + "_scale"].append(a / TOP)
    return {k: torch.cat(v) for k, v in out.items()}


def _binade_floor(x, mantissa, least, u):
    """x in whole steps of 2^-mantissa of its binade (`least` the lowest), u of a step added
    before the rest is cut off."""
    e = torch.frexp(x).exponent.double() - 1
    step = torch.exp2(e.clamp(min=least) - mantissa)
    return torch.floor(x / step + u) * step

"""Cases that time the router, the experts' weight gradient and the 8-bit expert products.

Three operators around the grouped expert MLP, each at the sizes it meets:

* ``route``  the router: the k largest of E logits per token, their probabilities, the
  tokens per expert, the balance and z losses and, in training, the gradient of the logits;
* ``wgrad``  the weight gradient of a grouped linear layer, one product per expert
  over that expert's rows;
* ``q8``     grouped linear layer on 8-bit weights with a scale per output channel; the
  rows are quantised per row on the way in; plain or with a fused gated activation.

``run`` computes them in plain torch operations in 32 bits, or, where ``own`` is set,
by the library's entry points.
"""

import math

import numpy as np
import torch

own = False

NEG_INF = float("-inf")
AMAX_FLOOR = 2.0 ** -100  # smallest row magnitude that a quantisation scale is made for
AUX, ZCO = 1e-2, 1e-3     # coefficients of the balance and z losses in a training step


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token being decoded: latency
        dict(name="route one token", op="route", T=1, E=128, k=8, dtype="f32", score="softmax",
             renorm=False, scale=1.0, train=False, masked=0),
        # a training batch of the balanced 128-expert layer, forward and backward
        dict(name="route train 16384x128", op="route", T=16384, E=128, k=8, dtype="f32",
             score="softmax", renorm=False, scale=1.0, train=True, masked=0),
        # a long prefill through a wide sigmoid router with renormalised, scaled probabilities
        dict(name="route prefill 121088x256", op="route", T=121088, E=256, k=8, dtype="bf16",
             score="sigmoid", renorm=True, scale=2.5, train=False, masked=0),
        # odd sizes, some experts switched off and some rows with none left
        dict(name="route train 4097x60 masked", op="route", T=4097, E=60, k=4, dtype="bf16",
             score="softmax", renorm=True, scale=1.0, train=True, masked=7),
        # first linear layer of the balanced 128-expert layer: the training step's largest product
        dict(name="wgrad balanced fc1", op="wgrad", R=131072, E=128, N=1536, K=2048, P=1,
             out="bf16", base=False, skew=0.0, empty=0),
        # second linear layer on a skewed, padded batch, added to FP32 gradients
        dict(name="wgrad skewed fc2 f32 add", op="wgrad", R=32768, E=128, N=2048, K=768, P=256,
             out="f32", base=True, skew=1.2, empty=16),
        # few experts with many rows each: hardly any output, a long reduction
        dict(name="wgrad tall 8 experts", op="wgrad", R=60001, E=8, N=768, K=320, P=1,
             out="f32", base=False, skew=0.7, empty=0),
        # a toy layer: latency
        dict(name="wgrad tiny", op="wgrad", R=512, E=4, N=256, K=64, P=1, out="bf16", base=False,
             skew=0.0, empty=1),
        # one token being decoded, first linear layer with the gated activation
        dict(name="q8 one token fc1", op="q8", R=8, E=128, N=1536, K=2048, gated=True, skew=0.0),
        # 64 sequences being decoded, second linear layer
        dict(name="q8 64 tokens fc2", op="q8", R=512, E=128, N=2048, K=768, gated=False,
             skew=0.0),
        # a skewed chunk of prompt on the wide 32-expert shard, first linear layer
        dict(name="q8 chunk wide fc1", op="q8", R=9001, E=32, N=4096, K=4096, gated=True,
             skew=0.8),
        # a long prefill of the balanced layer, first linear layer
        dict(name="q8 prefill fc1", op="q8", R=131072, E=128, N=1536, K=2048, gated=True,
             skew=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# widths of linear layers, multiples of 64 spread evenly over their logarithm
WIDTHS = (64, 128, 192, 256, 320, 384, 512, 640, 768, 896, 1024, 1280, 1536, 1856, 2048, 2688,
          3584, 4096)


def draw(rng):
    op = rng.choice(["route", "wgrad", "q8"])
    if op == "route":
        E = _log_int(rng, 4, 512)
        k = rng.randint(1, min(E, 10))
        T = min(_log_int(rng, 1, 121088), 121088 * 256 // E)
        return dict(op=op, T=T, E=E, k=k, dtype=rng.choice(["f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), train=rng.random() < 0.6,
                    masked=rng.choice([0, 0, max(0, E // 8)]))
    E = _log_int(rng, 2, 128)
    N, K = rng.choice(WIDTHS), rng.choice(WIDTHS)
    R = _log_int(rng, 8, 131072)
    # no more products than the largest listed case, nor more weights
    E = max(1, min(E, 128 * 1536 * 2048 // (N * K)))
    R = max(8, min(R, 131072 * 1536 * 2048 // (N * K)))
    skew = rng.choice([0.0, 0.7, 1.2])
    if op == "wgrad":
        return dict(op=op, R=R, E=E, N=N, K=K, P=rng.choice([1, 1, 16]),
                    out=rng.choice(["bf16", "f32"]), base=rng.random() < 0.4, skew=skew,
                    empty=rng.choice([0, E // 8]))
    gated = rng.random() < 0.5
    return dict(op=op, R=R, E=E, N=max(128, N // 128 * 128) if gated else N, K=K, gated=gated,
                skew=skew)


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
    r = np.random.default_rng(seed)
    E = case["E"]
    w = 1.0 / np.arange(1, E + 1) ** case["skew"]
    w = w[r.permutation(E)]
    w[r.permutation(E)[:min(case.get("empty", 0), E - 1)]] = 0.0
    c = r.multinomial(case["R"], w / w.sum())
    if case["skew"]:  # a token names an expert at most once: no expert has more than 1/8 of
        top = max(-(-case["R"] // 8), -(-case["R"] // max(1, int((w > 0).sum()))))  # the pairs
        over = int(np.maximum(c - top, 0).sum())
        c = np.minimum(c, top)
        for e in np.nonzero(w)[0]:
            add = min(over, top - int(c[e]))
            c[e] += add
            over -= add
    P = case.get("P", 1)
    padded = -(-c // P) * P
    return c, padded


def _offsets(padded):
    off = np.zeros(len(padded) + 1, np.int64)
    off[1:] = np.cumsum(padded)
    return off


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "route":
        return _prepare_route(case, g)
    c, padded = _counts(case, seed)
    off = _offsets(padded)
    E, N, K, R_cap = case["E"], case["N"], case["K"], case["R"] + case["E"] * (case.get("P", 1) - 1)
    spans = list(zip(off[:-1].tolist(), off[1:].tolist()))
    s = dict(op=case["op"], E=E, N=N, K=K, R_cap=R_cap, spans=spans, widest=int(padded.max()),
             live=torch.from_numpy(np.nonzero(padded)[0]).cuda(),
             offsets=torch.from_numpy(off.astype(np.int32)).cuda())
    if case["op"] == "wgrad":
        s["dC"] = _normal(g, (R_cap, N), 1.0)
        s["A"] = _normal(g, (R_cap, K), 0.5)
        pad = torch.ones(R_cap, dtype=torch.bool)
        for (lo, hi), n in zip(spans, c.tolist()):
            pad[lo:lo + n] = False
        pad[off[-1]:] = False  # rows past the last expert's: whatever the buffer held
        s["dC"][pad.cuda()] = 0
        s["A"][pad.cuda()] = 0
        s["dtype"] = torch.float32 if case["out"] == "f32" else torch.bfloat16
        s["base"] = _normal(g, (E, N, K), 1.0, s["dtype"]) if case["base"] else None
        s["dB"] = torch.empty((E, N, K), dtype=s["dtype"], device="cuda")
    else:
        s["gated"] = case["gated"]
        s["A"] = _normal(g, (R_cap, K), 1.0)
        # a few columns are much larger than the rest, as in trained models
        s["A"][:, torch.randint(0, K, (max(1, K // 256),), generator=g, device="cuda")] *= 8
        s["Wq"] = torch.randint(-127, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
        s["Ws"] = 0.02 / 64 * (0.5 + torch.rand((E, N), generator=g, device="cuda"))
        s["prob"] = torch.rand(R_cap, generator=g, device="cuda") if case["gated"] else None
        s["C"] = torch.empty((R_cap, N // 2 if case["gated"] else N), dtype=torch.bfloat16,
                             device="cuda")
    return s


def _prepare_route(case, g):
    T, E, k = case["T"], case["E"], case["k"]
    dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
    x = torch.randn((T, E), generator=g, device="cuda") * 1.5
    x += torch.randn((1, E), generator=g, device="cuda") * 0.5
    if case["masked"]:
        off = torch.randperm(E, generator=g, device="cuda")[:case["masked"]]
        x[:, off] = NEG_INF
        x[torch.rand(T, generator=g, device="cuda") < 0.02] = NEG_INF  # no expert left at all
    s = dict(op="route", T=T, E=E, k=k, x=x.to(dtype), sigmoid=case["score"] == "sigmoid",
             renorm=case["renorm"], scale=case["scale"], train=case["train"],
             idx=torch.empty((T, k), dtype=torch.int32, device="cuda"),
             prob=torch.empty((T, k), dtype=torch.float32, device="cuda"))
    if case["train"]:
        s["dprob"] = torch.randn((T, k), generator=g, device="cuda") * (1.0 / T)
        s["counts"] = torch.empty((E,), dtype=torch.int32, device="cuda")
        s["losses"] = torch.empty((2,), dtype=torch.float32, device="cuda")
        s["dlogits"] = torch.empty((T, E), dtype=dtype, device="cuda")
    return s


# ------------------------------------------------------------------ the operators

def run(state):
    return {"route": _own_route if own else _plain_route,
            "wgrad": _own_wgrad if own else _plain_wgrad,
            "q8": _own_q8 if own else _plain_q8}[state["op"]](state)


def _workspace(s, make):
    """The workspace a program keeps beside its buffers, made at the first pass."""
    if "ws" not in s:
        s["ws"] = make()
    return s["ws"]


def _own_route(s):
    import moe_expert_grouped_gb300.gg as gg

    score = gg.GG_SCORE_SIGMOID if s["sigmoid"] else gg.GG_SCORE_SOFTMAX
    if not s["train"]:
        gg.route(s["x"], s["k"], score, s["renorm"], s["scale"], idx=s["idx"], prob=s["prob"])
        return dict(idx=s["idx"], prob=s["prob"])
    gg.route(s["x"], s["k"], score, s["renorm"], s["scale"], idx=s["idx"], prob=s["prob"],
             counts=s["counts"], losses=s["losses"],
             ws=_workspace(s, lambda: gg.route_workspace(s["T"], s["E"], "cuda")))
    gg.route_bwd(s["x"], s["idx"], s["dprob"], score, s["renorm"], s["scale"],
                 counts=s["counts"], aux_coef=AUX, z_coef=ZCO, dlogits=s["dlogits"])
    return dict(idx=s["idx"], prob=s["prob"], counts=s["counts"], losses=s["losses"],
                dlogits=s["dlogits"])


def _plain_route(s):
    x, T, E, k = s["x"].float(), s["T"], s["E"], s["k"]
    # NaN-free rows: larger first, equal logits by expert id
    idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    top = x.amax(1, keepdim=True)
    none = top == NEG_INF  # no expert left: probabilities, losses and gradients are zero
    e = torch.where(none, torch.zeros_like(x), torch.exp(x - torch.where(none, 0.0, top)))
    mass = e.sum(1, keepdim=True)
    soft = e / torch.where(none, 1.0, mass)
    sc = 1.0 / (1.0 + torch.exp(-x)) if s["sigmoid"] else soft
    picked = sc.gather(1, idx)
    total = picked.sum(1, keepdim=True)
    share = picked / torch.where(total > 0, total, torch.ones_like(total))
    prob = s["scale"] * (share if s["renorm"] else picked)
    out = dict(idx=idx.to(torch.int32), prob=prob)
    if not s["train"]:
        return out
    counts = torch.zeros(E, dtype=torch.int32, device=x.device)
    counts.scatter_add_(0, idx.reshape(-1), torch.ones(T * k, dtype=torch.int32, device=x.device))
    row = sc.sum(1, keepdim=True)
    pn = sc / torch.where(row > 0, row, torch.ones_like(row))
    load = E * counts.float() / (T * k)
    lse = torch.where(none, 0.0, top + torch.log(torch.where(none, 1.0, mass)))
    losses = torch.stack([(load * pn.mean(0)).sum(), lse.square().mean()])
    # backward
    g = s["dprob"] * s["scale"]
    if s["renorm"]:
        g = (g - (g * share).sum(1, keepdim=True)) / torch.where(total > 0, total, math.inf)
    gs = torch.zeros_like(x).scatter_(1, idx, g)  # of the scores
    ga = (load - (load * pn).sum(1, keepdim=True)) * (AUX / T)
    if s["sigmoid"]:
        gs = gs + ga / torch.where(row > 0, row, math.inf)
        dx = gs * sc * (1.0 - sc)
    else:
        if s["renorm"]:
            dx = gs * soft
        else:
            dx = soft * (gs - (gs * soft).sum(1, keepdim=True))
        dx = dx + soft * ga
    dx = dx + (2.0 * ZCO / T) * lse * soft
    out.update(counts=counts, losses=losses, dlogits=dx.to(s["x"].dtype))
    return out


def _own_wgrad(s):
    import moe_expert_grouped_gb300.gg as gg

    ws = _workspace(s, lambda: gg.wgrad_workspace(s["E"], s["R_cap"], s["N"], s["K"], "cuda"))
    return gg.grouped_wgrad(s["dC"], s["A"], s["offsets"], base=s["base"], dB=s["dB"], ws=ws)


def _own_q8(s):
    import moe_expert_grouped_gb300.gg as gg

    ws = _workspace(s, lambda: gg.q8_workspace(s["R_cap"], s["K"], "cuda"))
    return gg.q8_grouped_fwd(s["A"], s["Wq"], s["Ws"], s["offsets"],
                             gg.GG_EPI_SWIGLU if s["gated"] else gg.GG_EPI_NONE,
                             prob_of_row=s["prob"], C=s["C"], ws=ws)


def _even(s):
    """Whether the live experts' rows fill most of a block padded to the widest expert's."""
    return s["widest"] * s["live"].numel() <= 3 * s["R_cap"]


def _block(s):
    """Row of each cell of the padded block [live experts][widest], and which cells hold one."""
    lo = s["offsets"][:-1].long()[s["live"]]
    n = s["offsets"][1:].long()[s["live"]] - lo
    at = torch.arange(s["widest"], device=lo.device)
    return (lo[:, None] + at).clamp_(max=s["R_cap"] - 1), at < n[:, None]


def _plain_wgrad(s):
    if _even(s):
        rows, held = _block(s)
        a = s["A"].float()[rows] * held[:, :, None]
        d = s["dC"].float()[rows] * held[:, :, None]
        dB = torch.zeros((s["E"], s["N"], s["K"]), device=a.device)
        dB[s["live"]] = d.transpose(1, 2) @ a
    else:
        dB = torch.stack([s["dC"][lo:hi].float().t() @ s["A"][lo:hi].float()
                          for lo, hi in s["spans"]])
    if s["base"] is not None:
        dB = dB + s["base"].float()
    return dB.to(s["dtype"])


def _plain_q8(s):
    a = s["A"].float()
    amax = a.abs().amax(1, keepdim=True).clamp_min(AMAX_FLOOR)
    q = torch.round(a * (127.0 / amax))
    if _even(s):
        rows, held = _block(s)
        y = q[rows] @ s["Wq"][s["live"]].float().transpose(1, 2)
        y = (y * s["Ws"][s["live"]][:, None, :])[held]
    else:
        y = torch.cat([q[lo:hi] @ s["Wq"][e].float().t() * s["Ws"][e]
                       for e, (lo, hi) in enumerate(s["spans"]) if hi > lo])
    y = y * (amax / 127.0)
    if s["gated"]:
        F = s["N"] // 2
        gate, up = y[:, :F], y[:, F:]
        y = gate / (1.0 + torch.exp(-gate)) * up * s["prob"][:, None]
    return y.to(torch.bfloat16)


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "route":
        T, E, k, w = case["T"], case["E"], case["k"], 4 if case["dtype"] == "f32" else 2
        b = T * E * w + 8 * T * k
        if case["train"]:
            b += T * E * w + 4 * T * k + 4 * E + 8
        return {"bytes": b, "flops": 8.0 * T * E * (3 if case["train"] else 1)}
    R, E, N, K = case["R"], case["E"], case["N"], case["K"]
    flops = 2.0 * R * N * K
    if case["op"] == "wgrad":
        w = 4 if case["out"] == "f32" else 2
        return {"bytes": 2 * R * (N + K) + E * N * K * w * (2 if case["base"] else 1),
                "flops": flops}
    live = E * (1.0 - (1.0 - 1.0 / E) ** R)  # experts that R pairs are expected to reach
    out = N // 2 if case["gated"] else N
    return {"bytes": 2 * R * K + live * N * (K + 4) + 2 * R * out, "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "wgrad": _exact_wgrad, "q8": _exact_q8}[case["op"]](s)


def _exact_route(s):
    """Row statistics and gradients from the Jacobians of softmax, sigmoid and the shares."""
    x = s["x"].double().cpu().numpy()
    T, E, k = s["T"], s["E"], s["k"]
    idx = np.argsort(-x, axis=1, kind="stable")[:, :k]
    dead = np.isneginf(x).all(1)
    xs = np.where(dead[:, None], 0.0, x)
    m = xs.max(1, keepdims=True)
    lse = np.log(np.exp(xs - m).sum(1, keepdims=True)) + m
    p = np.exp(xs - lse)
    p[dead] = 0.0
    lse[dead] = 0.0
    score = 1.0 / (1.0 + np.exp(-x)) if s["sigmoid"] else p
    sel = np.take_along_axis(score, idx, 1)
    tot = sel.sum(1, keepdims=True)
    safe = np.where(tot > 0, tot, 1.0)
    prob = s["scale"] * (sel / safe if s["renorm"] else sel)
    out = dict(idx=idx.astype(np.int32), prob=prob)
    if not s["train"]:
        return out
    counts = np.bincount(idx.reshape(-1), minlength=E)
    norm = score.sum(1, keepdims=True)
    norm_safe = np.where(norm > 0, norm, 1.0)
    dist = score / norm_safe
    c = E * counts / (T * k)
    losses = np.array([np.dot(c, dist.sum(0)) / T, (lse ** 2).sum() / T])
    dscore = np.zeros_like(x)
    up = s["dprob"].double().cpu().numpy() * s["scale"]
    if s["renorm"]:
        dsel = up / safe - (up * sel).sum(1, keepdims=True) / safe ** 2
        dsel = np.where(tot > 0, dsel, 0.0)
    else:
        dsel = up
    np.put_along_axis(dscore, idx, dsel, 1)
    # dist_e = score_e / norm
    ddist = np.broadcast_to(AUX * c / T, x.shape)
    dscore = dscore + np.where(norm > 0, ddist / norm_safe
                               - (ddist * score).sum(1, keepdims=True) / norm_safe ** 2, 0.0)
    if s["sigmoid"]:
        dx = dscore * score * (1.0 - score)
    else:
        dx = p * dscore - p * (p * dscore).sum(1, keepdims=True)
    dx = dx + ZCO / T * 2.0 * lse * p
    out.update(counts=counts.astype(np.int32), losses=losses, dlogits=dx)
    return out


def _exact_wgrad(s):
    dB = torch.zeros((s["E"], s["N"], s["K"]), dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(s["spans"]):
        torch.matmul(s["dC"][lo:hi].double().t(), s["A"][lo:hi].double(), out=dB[e])
        if s["base"] is not None:
            dB[e] += s["base"][e].double()
    return dB


def _exact_q8(s):
    a = s["A"].double()
    # the scale is a 32-bit number, as the codes are 8-bit ones
    amax = a.abs().amax(1).clamp_min(AMAX_FLOOR).float()
    codes = torch.round((a.float() * (127.0 / amax)[:, None])).double()
    y = torch.zeros((s["R_cap"], s["N"]), dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(s["spans"]):
        if hi > lo:
            y[lo:hi] = (codes[lo:hi] @ s["Wq"][e].double().t()) * s["Ws"][e].double()
    y *= (amax.double() / 127.0)[:, None]
    if s["gated"]:
        F = s["N"] // 2
        y = y[:, :F] * torch.sigmoid(y[:, :F]) * y[:, F:] * s["prob"].double()[:, None]
    return y

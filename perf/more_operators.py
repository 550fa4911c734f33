"""Experts on quantised tokens, as cases that can be timed.

Four operators around the MXFP4 routed experts:

  route     scores of the experts (softmax or sigmoid), a bias that only steers
            the choice, groups of experts, top K, normalised weights;
  quantize  tokens to MXFP4 (E2M1 codes, one power-of-two scale per 32 values)
            and the values they stand for, read back;
  linear    the product of MXFP4 tokens and MXFP4 weights;
  experts   the routed expert linear on MXFP4 tokens.

An MXFP4 group of 32 values with largest magnitude a has the scale byte
s = clamp(floor(log2 a) - 2 + 127, 0, 254) and holds x 2^(127 - s) rounded to
the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, larger
magnitudes to 6), with x's sign.

``own`` selects who computes: False, the plain form below (elementary torch
operations in float32, the router's choice in float64, rounded once); True,
the library's kernels.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # The decode batch of 8 tokens: softmax over 32 experts, bf16 logits
        # (equal logits happen), nothing but latency.
        dict(name="route 8x32", op="route", T=8, E=32, K=4, dtype="bf16", score="softmax",
             bias=False, groups=1, top_groups=1, best=2, normalize=True, scaling=1.0),
        # A prompt batch: sigmoid scores, a balancing bias, 4 of 8 groups of
        # 32 experts, float32 logits.
        dict(name="route 4096x256 groups", op="route", T=4096, E=256, K=8, dtype="fp32",
             score="sigmoid", bias=True, groups=8, top_groups=4, best=2, normalize=True,
             scaling=2.5),
        # The skewed prefill's router at four times its tokens (a step of
        # several prompts): 384 experts.
        dict(name="route 32768x384", op="route", T=32768, E=384, K=8, dtype="fp32",
             score="sigmoid", bias=True, groups=1, top_groups=1, best=2, normalize=True,
             scaling=1.0),
        # The decode batch's tokens.
        dict(name="quantize 8x2880", op="quantize", T=8, I=2880, dtype="bf16", pad=0),
        # The largest prompt batch's tokens, hidden width 7168.
        dict(name="quantize 8192x7168", op="quantize", T=8192, I=7168, dtype="bf16", pad=0),
        # float32 activations, an odd number of tokens, rows that are slices
        # of a wider matrix.
        dict(name="quantize fp32 1021x2912", op="quantize", T=1021, I=2912, dtype="fp32", pad=32),
        # One token through one projection of the decode workload's sizes.
        dict(name="linear 1x2880x5760", op="linear", T=1, I=2880, O=5760, dtype="bf16"),
        # The largest prompt batch through a dense projection.
        dict(name="linear 8192x7168x4096", op="linear", T=8192, I=7168, O=4096, dtype="bf16"),
        # The decode batch: 8 tokens, 4 of 128 experts.
        dict(name="experts decode 8", op="experts", T=8, E=128, K=4, I=2880, O=5760, dtype="bf16",
             zipf=0.0),
        # The wide decode batch: 16 tokens, 8 of 384 experts.
        dict(name="experts decode 16 wide", op="experts", T=16, E=384, K=8, I=7168, O=4096,
             dtype="bf16", zipf=0.0),
        # A small ragged chunk with odd sizes, float32 shared output.
        dict(name="experts fp32 333", op="experts", T=333, E=24, K=3, I=1056, O=1001, dtype="fp32",
             zipf=0.7),
        # The skewed prefill: 8192 tokens, 8 of 384 experts by Zipf's law.
        dict(name="experts prefill 8192", op="experts", T=8192, E=384, K=8, I=7168, O=4096,
             dtype="bf16", zipf=1.2),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "quantize", "linear", "experts", "experts"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    if op == "route":
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 512 // groups)
        top = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 32768), E=E,
                    K=rng.randint(1, min(16, top * (E // groups))), dtype=dtype,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6,
                    groups=groups, top_groups=top, best=rng.choice([1, 2]),
                    normalize=rng.random() < 0.7, scaling=rng.choice([1.0, 2.5]))
    I = 32 * _log(rng, 1, 256)
    if op == "quantize":
        return dict(op=op, T=_log(rng, 1, 8192), I=I, dtype=dtype, pad=rng.choice([0, 0, 32, 160]))
    T, O = _log(rng, 1, 8192), _log(rng, 1, 8192)
    if op == "linear":
        return dict(op=op, T=T, I=I, O=O, dtype=dtype)
    E = _log(rng, 1, min(384, max(1, (1 << 32) // (I * O))))
    K = rng.randint(1, min(8, E))
    return dict(op=op, T=T, E=E, K=K, I=I, O=O, dtype=dtype, zipf=rng.choice([0.0, 0.7, 1.2]))


def _touched(case):
    """Experts with at least one token, on average over the picks' law."""
    T, E, K = case["T"], case["E"], case["K"]
    w = [(r + 1.0) ** -case["zipf"] for r in range(E)]
    top = sum(w)
    return sum(1.0 - max(0.0, 1.0 - min(1.0, K * v / top)) ** T for v in w)


def work(case):
    T, size = case["T"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "route":
        E = case["E"]
        return {"bytes": T * E * size + (E * 4 if case["bias"] else 0) + T * case["K"] * 8,
                "flops": 8 * T * E}
    I = case["I"]
    packed = I // 32 * 17
    if case["op"] == "quantize":          # codes written and read back
        return {"bytes": 2 * T * I * size + 2 * T * packed, "flops": 4 * T * I}
    O = case["O"]
    if case["op"] == "linear":
        return {"bytes": (T + O) * packed + T * O * size, "flops": 2 * T * I * O}
    K = case["K"]
    return {"bytes": int(_touched(case) * O) * packed + T * packed + 2 * T * O * size + T * K * 8,
            "flops": 2 * T * K * I * O}


# ----------------------------------------------------------------- inputs ----
def _quantize(x):
    """(codes as (..., G, 16) bytes, scale bytes (..., G)) of x (..., I)."""
    g = x.float().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1)
    _, e = torch.frexp(top)                   # top = m 2^e, 0.5 <= m < 1
    s = torch.where(top > 0, e - 3 + 127, 0).clamp(0, 254)
    y = g * ((254 - s) << 23).int().view(torch.float32)[..., None]     # x 2^(127 - s)
    a = y.abs()
    # Ties go to the even code: below 0.25 and at it to 0, at 0.75 to 1, ...
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0))
    code = code + 8 * torch.signbit(y)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), s.to(torch.uint8)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    T = case["T"]
    s = {"case": dict(case)}

    def normal(*shape, by=1.0):
        return torch.randn(*shape, generator=g, device=dev).mul_(by)

    if case["op"] == "route":
        s["logits"] = normal(T, case["E"], by=1.5).to(DTYPES[case["dtype"]])
        s["bias"] = normal(case["E"], by=0.05) if case["bias"] else None
        return s
    I = case["I"]
    if case["op"] == "quantize":
        # Activations: normal values, tokens of different size, a few channels
        # far above the others.
        x = normal(T, I + case["pad"]) * torch.exp(normal(T, 1))
        x[:, torch.rand(I + case["pad"], generator=g, device=dev) < 0.01] *= 20
        s["x"] = x.to(DTYPES[case["dtype"]])[:, case["pad"]:]
        return s
    x = normal(T, I) * torch.exp(normal(T, 1, by=0.5))
    s["x_packed"], s["x_scales"] = _quantize(x)
    rows = (case["E"], case["O"]) if case["op"] == "experts" else (case["O"],)
    s["packed"] = torch.randint(0, 256, rows + (I // 32, 16), generator=g, device=dev,
                                dtype=torch.uint8)
    s["scales"] = torch.randint(116, 122, rows + (I // 32,), generator=g, device=dev,
                                dtype=torch.uint8)
    if case["op"] == "experts":
        E, K = case["E"], case["K"]
        rank = torch.randperm(E, generator=g, device=dev).float() + 1
        u = torch.rand(T, E, generator=g, device=dev).clamp_(1e-7, 1 - 1e-7)
        key = -case["zipf"] * rank.log() - torch.log(-torch.log(u))
        s["sel"] = key.topk(K, 1).indices.to(torch.int32)
        s["p"] = torch.softmax(normal(T, K), 1)
        s["shared"] = normal(T, case["O"]).to(DTYPES[case["dtype"]])
    return s


def run(state):
    case = state["case"]
    if not own:
        return globals()["_plain_" + case["op"]](state)
    import mxfp4_routed_expert_route_gb300 as lib
    if case["op"] == "route":
        return list(lib.route_experts(
            state["logits"], case["K"], score=case["score"], bias=state["bias"],
            groups=case["groups"], top_groups=case["top_groups"], group_best=case["best"],
            normalize=case["normalize"], scaling=case["scaling"]))
    if case["op"] == "quantize":
        packed, scales = lib.quantize_mxfp4(state["x"])
        return lib.dequantize_mxfp4(packed, scales, DTYPES[case["dtype"]])
    if case["op"] == "linear":
        return lib.mxfp4_linear(state["x_packed"], state["x_scales"], state["packed"],
                                state["scales"], dtype=DTYPES[case["dtype"]])
    return lib.mxfp4_expert_linear_quantized(
        state["x_packed"], state["x_scales"], state["packed"], state["scales"], state["sel"],
        state["p"], state["shared"])


# --------------------------------------------------------------- plain form --
def _plain_route(s):
    c = s["case"]
    x = s["logits"].double()
    T, E = x.shape
    if c["score"] == "softmax":
        z = (x - x.amax(1, keepdim=True)).exp()
        score = z / z.sum(1, keepdim=True)
    else:
        score = 1 / (1 + (-x).exp())
    choice = score if s["bias"] is None else score + s["bias"].double()
    order = x if s["bias"] is None else choice    # the same order, without rounding
    if c["groups"] > 1:
        n = E // c["groups"]
        best = choice.view(T, c["groups"], n).sort(dim=2, descending=True).values
        best = best[..., :min(c["best"], n)].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        seen = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        order = order.masked_fill(~seen.repeat_interleave(n, 1), -math.inf)
    sel = order.sort(dim=1, descending=True, stable=True).indices[:, :c["K"]]
    p = score.gather(1, sel)
    if c["normalize"]:
        p = p / (p.sum(1, keepdim=True) + 1e-20)
    return [sel.int(), (p * c["scaling"]).float()]


def _plain_values(packed, scales):
    """The float32 values of codes (..., G, 16) and scale bytes (..., G)."""
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).int()
    e, m = (code >> 1) & 3, (code & 1).float()
    mag = torch.where(e > 0, (1 + 0.5 * m) * (1 << e) * 0.5, 0.5 * m)
    mag = torch.where(code >= 8, -mag, mag)
    return (mag * (scales.int() << 23).view(torch.float32)[..., None]).flatten(-2)


def _plain_quantize(s):
    packed, scales = _quantize(s["x"])
    return _plain_values(packed, scales).to(s["x"].dtype)


def _plain_linear(s):
    x, w = _plain_values(s["x_packed"], s["x_scales"]), _plain_values(s["packed"], s["scales"])
    return (x @ w.T).to(DTYPES[s["case"]["dtype"]])


def _plain_experts(s):
    c = s["case"]
    x = _plain_values(s["x_packed"], s["x_scales"])
    pairs = s["sel"].long().flatten()
    order = pairs.sort(stable=True).indices
    counts = pairs.bincount(minlength=c["E"]).tolist()
    part = torch.empty(pairs.numel(), c["O"], device=x.device)
    at = 0
    for e, n in enumerate(counts):
        if n:
            own_pairs = order[at:at + n]
            w = _plain_values(s["packed"][e], s["scales"][e])
            part[own_pairs] = x[own_pairs // c["K"]] @ w.T
            at += n
    part = part.view(c["T"], c["K"], c["O"]).mul_(s["p"][..., None])
    return part.sum(1).add_(s["shared"].float()).to(s["shared"].dtype)


# ------------------------------------------------------------- 64 bits -------
_TABLE = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _table_values(packed, scales):
    table = torch.tensor(_TABLE + [-v for v in _TABLE], dtype=torch.float64, device=packed.device)
    out = torch.empty(*packed.shape[:-1], 32, dtype=torch.float64, device=packed.device)
    out[..., 0::2] = table[(packed % 16).long()]
    out[..., 1::2] = table[(packed // 16).long()]
    return (out * torch.exp2(scales.double() - 127)[..., None]).flatten(-2)


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    T = case["T"]
    if case["op"] == "route":
        x = s["logits"].double()
        score = torch.softmax(x, 1) if case["score"] == "softmax" else torch.sigmoid(x)
        bias = 0.0 if s["bias"] is None else s["bias"].double()
        choice = score + bias
        key = choice if case["bias"] else x
        left = torch.ones_like(x, dtype=torch.bool)
        rows = torch.arange(T, device=x.device)

        def best(v):                      # the first of the largest of each row
            top = v.amax(1, keepdim=True)
            return (v == top).int().argmax(1) if v.shape[1] else None

        if case["groups"] > 1:
            n = case["E"] // case["groups"]
            group = choice.view(T, case["groups"], n).topk(min(case["best"], n), 2).values.sum(2)
            keep = torch.zeros_like(group, dtype=torch.bool)
            for _ in range(case["top_groups"]):
                keep[rows, best(group.masked_fill(keep, -math.inf))] = True
            left = keep[:, :, None].expand(T, case["groups"], n).reshape(T, -1).clone()
        sel = []
        for _ in range(case["K"]):
            sel.append(best(key.masked_fill(~left, -math.inf)))
            left[rows, sel[-1]] = False
        sel = torch.stack(sel, 1)
        p = score.gather(1, sel)
        if case["normalize"]:
            p = p / p.sum(1, keepdim=True)
        return [sel.int(), p * case["scaling"]]
    if case["op"] == "quantize":
        g = s["x"].double().unflatten(-1, (-1, 32))
        top = g.abs().amax(-1, keepdim=True)
        # 2^floor(log2 top) is the power of two that a double's exponent field holds.
        power = (top.view(torch.int64) >> 52 << 52).view(torch.float64)
        scale = power.clamp_min(2.0 ** -125) / 4
        grid = torch.tensor(_TABLE, dtype=torch.float64, device=g.device)
        a = (g.abs() / scale).clamp_max(6.0)
        hi = torch.searchsorted(grid, a).clamp_max(7)             # grid[hi] >= a
        lo = (hi - 1).clamp_min(0)
        down, up = a - grid[lo], grid[hi] - a
        code = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
        return (torch.sign(g) * grid[code] * scale).flatten(-2)
    pairs = T * case.get("K", 1)
    if 2.0 * pairs * case["I"] * case["O"] > 4e12:
        return None
    x = _table_values(s["x_packed"], s["x_scales"])
    if case["op"] == "linear":
        return x @ _table_values(s["packed"], s["scales"]).T
    out = s["shared"].double()
    for e in s["sel"].unique().tolist():
        t, k = (s["sel"] == e).nonzero(as_tuple=True)
        y = x[t] @ _table_values(s["packed"][e], s["scales"][e]).T
        out.index_add_(0, t, y * s["p"][t, k].double()[:, None])
    return out

"""Plain 64-bit forms of the operators on quantised tokens.

MXFP4 values and the quantiser are exact, so the tests ask for equal bits.
The router's choice is made in float64 here as in the library; its weights are
float32 there: a score is one exponential (2 ulp; the softmax's difference of
logits is carried in two terms, exactly), an addition and a division
(half an ulp each, at most 3.5 ulp of 2^-23 together, with the sum of a softmax
adding log2(1024) = 10 roundings of half an ulp of the larger operand at most
when it is summed as a tree of 32 lanes over up to 32 terms each: 37 half ulps),
then one sum of up to 32 picks (31 half ulps), a division and a product: under
64 half ulps of 2^-23 in all, 64 * 2^-24 = 2^-18 relative.
"""
import math

import torch

WEIGHT_RTOL = 2.0 ** -18
GRID = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def quantize(x):
    """(packed, scales) of x (..., I) on the CPU, by trying every code."""
    g = x.double().cpu().unflatten(-1, (-1, 32))
    finite = g.isfinite().all(-1)
    top = torch.where(finite, g.abs().amax(-1), 0.0)
    s = torch.where(top > 0, (torch.frexp(top)[1] - 1 - 2 + 127), 0).clamp(0, 252)
    y = torch.where(finite[..., None], g, 0.0) * torch.exp2(127.0 - s.double())[..., None]
    dist = (y.abs()[..., None].clamp(max=6.0) - GRID).abs()
    # The nearest; of two as near the even code: order the codes 0, 2, 4, 6, 1, ...
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])
    code = order[dist[..., order].argmin(-1)]
    code = torch.where(torch.signbit(y) & finite[..., None], code + 8, code)
    packed = code[..., 0::2] + 16 * code[..., 1::2]
    return packed.to(torch.uint8), torch.where(finite, s, 255).to(torch.uint8)


def values(packed, scales):
    """The float64 values of MXFP4 rows, on their device; 255 is NaN."""
    grid = torch.cat([GRID, -GRID]).to(packed.device)
    code = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).long()
    by = torch.exp2(scales.double() - 127)
    by = torch.where(scales == 255, math.nan, by)
    return (grid[code] * by[..., None]).flatten(-2)


def route(logits, K, score="softmax", bias=None, groups=1, top_groups=None, group_best=2,
          normalize=True, scaling=1.0):
    """(ids, weights) as lists of Python numbers, token by token."""
    top_groups = groups if top_groups is None else top_groups
    ids, weights = [], []
    b = [0.0] * logits.shape[1] if bias is None else bias.double().tolist()
    for row in logits.double().tolist():
        E = len(row)
        if score == "softmax":
            top = max((v for v in row if v == v), default=0.0)
            z = [1.0 if v == top else math.exp(v - top) if v < top else 0.0 for v in row]
            s = [v / (sum(z) or 1.0) for v in z]
        else:
            s = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in row]
        choice = [math.nan if row[e] != row[e] else s[e] + b[e] for e in range(E)]
        n, kept = E // groups, set(range(groups))
        if groups > 1:
            rank = []
            for g in range(groups):
                c = sorted((v for v in choice[g * n:(g + 1) * n] if v == v), reverse=True)
                v = sum(c[:group_best])
                if c and v == v:
                    rank.append((-v, g))
            kept = {g for _, g in sorted(rank)[:top_groups]}
        key = row if bias is None else choice
        left = [e for e in range(E) if choice[e] == choice[e] and e // n in kept]
        pick = sorted(left, key=lambda e: (-key[e], e))[:K]
        w = [s[e] for e in pick]
        if normalize:
            total = sum(w) + 1e-20
            w = [v / total for v in w]
        ids.append(pick + [-1] * (K - len(pick)))
        weights.append([v * scaling for v in w] + [0.0] * (K - len(pick)))
    return (torch.tensor(ids, dtype=torch.int32).view(-1, K),
            torch.tensor(weights, dtype=torch.float64).view(-1, K))


def product_bound(x, w, I, dtype, more=0):
    """How far a product of the float64 values x (T, I) and w (O, I) may be off,
    before `more` roundings of half an ulp of the sums' size and the result's
    own rounding: products are exact, and each of the I/64 steps of the tensor
    core adds 64 of them and the running sum in float32, aligned to the largest
    and cut, not rounded, which loses at most an ulp (2^-23 of the sum of
    magnitudes) for each of two operands' groups."""
    terms = x.abs() @ w.abs().T
    return (I / 64 + 1 + more) * 2.0 ** -22 * terms

"""Plain 64-bit forms of the attention operators, and the error bounds of the
GPU results against them.

Both are written from the definitions in include/mxfp4el_attention.h, one
sequence and one head at a time, and run on whatever device the inputs are on.

Bound of the attention. Let A = sum_j w_j |v_j| with the softmax weights w.
A score is a float32 sum of D products (each addition within 2^-23 of the sum
of magnitudes: tensor-core sums need not round to nearest), scaled in float32:

    |ds_j| <= ((D + 4) 2^-23 + 2^-22) scale |q| . |k_j|

e^s then has the relative error 2 max|ds| (score and running maximum) + 2^-20
(the power's argument and value), and the weight that multiplies v another u_P
where it is rounded to the token dtype for the second product (bf16: 2^-8).
Numerator and denominator both carry it, and their float32 sums over n keys
(tiles of 32 to 128 keys, then the tiles) add (160 + n / 32) 2^-23 each:

    |out - exact| <= 2 A (2 max|ds| + 2^-20 + u_P + (160 + n / 32) 2^-23) + u |out|

with u the rounding to the token dtype (2^-8 bf16, 2^-24 float32).

Bound of the append. The mean square, its root, the two weights and the
rotation are about 20 float32 roundings (the sum of D squares in pairs adds
log2 D): 40 2^-24 (|a c| + |b s|) + u |y| covers them.
"""
from __future__ import annotations

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
U_P = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


def gather(pages, table_row, head, n):
    """The first n rows of a head of one sequence, in float64."""
    size = pages.shape[2]
    ids = table_row[:-(-n // size)].long()
    return pages[ids, head].reshape(-1, pages.shape[3])[:n].double()


def attention(q, k_pages, v_pages, table, lens, offsets, *, scale=None, window=0, sinks=0,
              sink_logits=None):
    """(out, bound), both float64. lens and offsets are lists."""
    T, heads, D = q.shape
    dtype = q.dtype
    kv_heads = k_pages.shape[1]
    group = heads // kv_heads
    scale = D ** -0.5 if scale is None else scale
    out = torch.zeros(T, heads, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b, n in enumerate(lens):
        r0, r1 = offsets[b], offsets[b + 1]
        m = r1 - r0
        if m == 0 or n == 0:
            continue
        pos = torch.arange(n - m, n, device=q.device)[:, None]
        key = torch.arange(n, device=q.device)[None]
        seen = key <= pos
        if window:
            seen = seen & ((pos - key < window) | (key < sinks))
        for c in range(kv_heads):
            k, v = gather(k_pages, table[b], c, n), gather(v_pages, table[b], c, n)
            for h in range(c * group, (c + 1) * group):
                x = q[r0:r1, h].double()
                s = torch.where(seen, x @ k.T * scale, -math.inf)
                ds = ((D + 4) * 2.0 ** -23 + 2.0 ** -22) * abs(scale) * (x.abs() @ k.abs().T)
                ds = torch.where(seen, ds, 0.0).amax(1, keepdim=True)
                top = s.amax(1, keepdim=True)
                if sink_logits is not None:
                    top = top.clamp(min=float(sink_logits[h]))
                top = torch.where(top == -math.inf, 0.0, top)
                p = torch.where(seen, (s - top).exp(), 0.0)
                total = p.sum(1, keepdim=True)
                if sink_logits is not None:
                    total = total + (sink_logits[h].double() - top).exp()
                w = torch.where(total > 0, p / total, 0.0)
                # A key that a row does not see takes no part, whatever it holds.
                clean = torch.where(torch.isfinite(v), v, 0.0)
                y = w @ clean
                bad = ~torch.isfinite(v)
                for j, d in bad.nonzero().tolist():
                    y[:, d] = torch.where(seen[:, j], y[:, d] + w[:, j] * v[j, d], y[:, d])
                out[r0:r1, h] = y
                e = 2 * ds + 2.0 ** -20 + U_P[dtype] + (160 + n / 32) * 2.0 ** -23
                bound[r0:r1, h] = 2 * e * (w @ clean.abs()) + U[dtype] * y.abs() + 1e-30
    return out, bound


def turn(x, norm, eps, cos, sin, interleaved):
    """(y, magnitude): one row set (tokens, heads, D) normed and turned in
    float64; magnitude is |a c| + |b s| per element."""
    x = x.double()
    if norm is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * norm.double()
    y, mag = x.clone(), x.abs()
    half = cos.shape[-1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        c, s = cos[:, None, i], sin[:, None, i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def append(q, k, v, k_pages, v_pages, table, lens, offsets, *, cos_sin=None, interleaved=False,
           q_norm=None, k_norm=None, eps=1e-6):
    """((q_out, bound), (k_pages, bound), v_pages) in float64 after the append."""
    D, size = q.shape[2], k_pages.shape[2]
    u = U[q.dtype]
    pos = torch.zeros(q.shape[0], dtype=torch.long, device=q.device)
    for b, n in enumerate(lens):
        r0, r1 = offsets[b], offsets[b + 1]
        pos[r0:r1] = torch.arange(n - (r1 - r0), n, device=q.device)
    half = 0 if cos_sin is None else cos_sin.shape[1] // 2
    if cos_sin is None:
        cos = sin = torch.zeros(q.shape[0], 0, dtype=torch.float64, device=q.device)
    else:
        cos, sin = cos_sin[pos, :half].double(), cos_sin[pos, half:].double()

    def bounded(x, norm):
        y, mag = turn(x, norm, eps, cos, sin, interleaved)
        return y, 40 * 2.0 ** -24 * mag + u * y.abs() + 1e-30

    q_out, q_bound = bounded(q, q_norm)
    k_out, k_bound = bounded(k, k_norm)
    kp, vp = k_pages.double(), v_pages.double()
    kb = torch.zeros_like(kp)
    for b, n in enumerate(lens):
        for t in range(offsets[b], offsets[b + 1]):
            p = int(pos[t])
            if p < 0:        # no such position: nothing is appended
                continue
            page, slot = int(table[b, p // size]), p % size
            kp[page, :, slot] = k_out[t]
            kb[page, :, slot] = k_bound[t]
            vp[page, :, slot] = v[t].double()
    return (q_out, q_bound), (kp, kb), vp

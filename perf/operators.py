"""The attention half of a decoder layer, as cases that can be timed.

Three operators that a serving program runs next to the routed experts:

  append   norms of the query and key heads, the position rotation, and the
           write of the new keys and values into a paged cache, in one pass;
  decode   attention of one new token of each sequence over the paged cache;
  prefill  attention of prompts (or chunks of prompts, with a history in the
           cache) over the paged cache.

With n keys in a sequence after the append and m new tokens, new token i has
position n - m + i. A query at position a sees key j when j <= a and, with a
window w > 0, when a - j < w or j < sinks. A head may also carry a learned
logit that joins the softmax's sum without a value of its own. A query that
sees no key gives zeros.

``own`` selects who computes: False, the plain form below (elementary torch
operations in float32, rounded once); True, the library's kernels.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6
ROTARY_BASE = 10000.0


def listed():
    return [
        # One decode step of 8 sequences (the linear's decode batch), heads of
        # 64 at hidden width 2880's layer: a few hundred KB, all launch latency.
        dict(name="append decode 8", op="append", dtype="bf16", heads=64, kv_heads=8, head_dim=64,
             page=16, seqs=8, ctx_min=1, ctx_max=2000, new_min=1, new_max=1, rotary=64,
             interleaved=False, norm=False, ragged=1),
        # The largest prompt batch (8192 tokens, as the linear's skewed
        # prefill): normed heads of 128, five ragged prompts.
        dict(name="append prompts 8192", op="append", dtype="bf16", heads=64, kv_heads=8,
             head_dim=128, page=64, seqs=5, ctx_min=0, ctx_max=0, new_min=300, new_max=2503,
             rotary=128, interleaved=False, norm=True, ragged=2, tokens=8192),
        # float32 tokens, a partial interleaved rotation, odd lengths behind
        # histories that end inside a page.
        dict(name="append fp32 partial", op="append", dtype="fp32", heads=12, kv_heads=4,
             head_dim=64, page=32, seqs=7, ctx_min=3, ctx_max=500, new_min=1, new_max=601,
             rotary=32, interleaved=True, norm=True, ragged=3),
        # A single short chat turn: one sequence, a few hundred keys.
        dict(name="decode 1x333", op="decode", dtype="bf16", heads=32, kv_heads=8, head_dim=128,
             page=16, seqs=1, ctx_min=333, ctx_max=333, window=0, sinks=0, logits=False, ragged=4),
        # The wide decode batch (16 sequences) in a layer with a short window,
        # first tokens that stay visible and learned logits.
        dict(name="decode window 16", op="decode", dtype="bf16", heads=64, kv_heads=8, head_dim=64,
             page=64, seqs=16, ctx_min=40, ctx_max=32768, window=128, sinks=4, logits=True,
             ragged=5),
        # Two very long sequences, seven queries to a key head: the work has
        # to be split over the cache's length.
        dict(name="decode 2x131072", op="decode", dtype="bf16", heads=56, kv_heads=8, head_dim=128,
             page=64, seqs=2, ctx_min=100003, ctx_max=131072, window=0, sinks=0, logits=False,
             ragged=6),
        # A full serving batch of ragged lengths: gigabytes of cache.
        dict(name="decode 128 ragged", op="decode", dtype="bf16", heads=64, kv_heads=8,
             head_dim=128, page=32, seqs=128, ctx_min=1, ctx_max=16384, window=0, sinks=0,
             logits=False, ragged=7),
        # The same in float32, a middle-sized batch.
        dict(name="decode fp32 24", op="decode", dtype="fp32", heads=16, kv_heads=4, head_dim=128,
             page=16, seqs=24, ctx_min=17, ctx_max=3001, window=0, sinks=0, logits=False,
             ragged=8),
        # Three short float32 prompts.
        dict(name="prefill fp32 3 short", op="prefill", dtype="fp32", heads=16, kv_heads=4,
             head_dim=64, page=16, seqs=3, ctx_min=0, ctx_max=0, new_min=1, new_max=301, window=0,
             sinks=0, logits=False, ragged=9),
        # The prefill batch (4096 tokens) in a layer with a short window and
        # learned logits, heads of 64.
        dict(name="prefill window 4096", op="prefill", dtype="bf16", heads=64, kv_heads=8,
             head_dim=64, page=16, seqs=2, ctx_min=0, ctx_max=0, new_min=1500, new_max=2596,
             window=128, sinks=0, logits=True, ragged=10, tokens=4096),
        # Chunks of six ragged prompts behind histories of up to 16k keys.
        dict(name="prefill chunks 6", op="prefill", dtype="bf16", heads=56, kv_heads=8,
             head_dim=128, page=32, seqs=6, ctx_min=100, ctx_max=16384, new_min=1, new_max=1024,
             window=0, sinks=0, logits=False, ragged=11),
        # One prompt of 8192 tokens, full causal attention: the most work.
        dict(name="prefill 8192", op="prefill", dtype="bf16", heads=64, kv_heads=8, head_dim=128,
             page=64, seqs=1, ctx_min=0, ctx_max=0, new_min=8192, new_max=8192, window=0, sinks=0,
             logits=False, ragged=12),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    kv = rng.choice([1, 2, 4, 8])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "bf16", "fp32"]),
                heads=kv * rng.choice([1, 2, 3, 4, 5, 7, 8]), kv_heads=kv,
                head_dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
                ragged=rng.randrange(1 << 30))
    if op == "append":
        case["seqs"] = _log(rng, 1, 64)
        case["new_min"], case["new_max"] = 1, _log(rng, 1, max(1, 8192 // case["seqs"]))
        case["ctx_min"], case["ctx_max"] = 0, _log(rng, 1, 2000)
        case["rotary"] = rng.choice([case["head_dim"], case["head_dim"], 32])
        case["interleaved"], case["norm"] = rng.random() < 0.3, rng.random() < 0.6
        return case
    case["window"] = rng.choice([0, 0, 128, _log(rng, 1, 4096)])
    case["sinks"] = rng.choice([0, 4, _log(rng, 1, 200)]) if case["window"] else 0
    case["logits"] = rng.random() < 0.3
    if op == "decode":
        case["seqs"] = _log(rng, 1, 160)
        case["ctx_min"] = 1
        case["ctx_max"] = _log(rng, 2, min(131072, 1600000 // (kv * case["seqs"])))
    else:
        # (sequences, heads, new, keys) stays under half of the largest listed
        # case's (query, key) pairs, and lower still in float32.
        most = 1 << 30
        if case["dtype"] == "fp32":
            most >>= 3
        case["seqs"] = _log(rng, 1, 12)
        case["new_min"], case["new_max"] = 1, _log(rng, 1, 4096)
        most //= case["seqs"] * case["heads"]
        case["new_max"] = min(case["new_max"], max(1, int(math.sqrt(most) / 1.1)))
        case["ctx_min"] = 0
        left = most // case["new_max"] - case["new_max"]
        case["ctx_max"] = _log(rng, 1, max(1, min(32768, left)))
    return case


def _lengths(case):
    """(history, new) token counts of each sequence: a fixed draw per case."""
    r = random.Random(case["ragged"])
    hist, new = [], []
    for i in range(case["seqs"]):
        hi, lo = case["ctx_max"], case["ctx_min"]
        if case["op"] == "decode":  # the new token is among the keys
            n = hi if i == 0 else r.randint(lo, hi)
            hist.append(n - 1)
            new.append(1)
        else:
            hist.append(hi if i == 0 else r.randint(lo, hi))
            new.append(case["new_max"] if i == 0 else r.randint(case["new_min"], case["new_max"]))
    if "tokens" in case:  # the last prompt makes up the stated total
        new[-1] += case["tokens"] - sum(new)
        if new[-1] < 1:
            new = [case["tokens"] // case["seqs"]] * case["seqs"]
            new[-1] += case["tokens"] - sum(new)
    return hist, new


def _visible(case):
    """Keys that some new token of each sequence sees, and (query, key) pairs."""
    hist, new = _lengths(case)
    w, s = case.get("window", 0), case.get("sinks", 0)
    keys = pairs = 0
    for h, m in zip(hist, new):
        n = h + m
        lo = max(0, h - w + 1) if w else 0     # first key in the first query's window
        keys += n - lo + min(s if w else 0, lo)
        if not w:
            pairs += m * h + m * (m + 1) // 2
        else:
            for a in range(h, n):
                first = max(0, a - w + 1)
                pairs += a + 1 - first + min(s, first)
    return keys, pairs


def work(case):
    hist, new = _lengths(case)
    hq, hk, d = case["heads"], case["kv_heads"], case["head_dim"]
    size = 2 if case["dtype"] == "bf16" else 4
    tokens = sum(new)
    if case["op"] == "append":
        values = tokens * (hq + 2 * hk) * d
        table = tokens * case["rotary"] * 4
        return {"bytes": 2 * values * size + table, "flops": 8 * values}
    keys, pairs = _visible(case)
    moved = 2 * keys * hk * d * size + 2 * tokens * hq * d * size
    return {"bytes": moved, "flops": 4 * pairs * hq * d}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    hist, new = _lengths(case)
    dtype, d, hk, page = DTYPES[case["dtype"]], case["head_dim"], case["kv_heads"], case["page"]
    hq, tokens = case["heads"], sum(new)
    lens = [h + m for h, m in zip(hist, new)]
    used = [-(-n // page) for n in lens]
    pages = sum(used) + 1

    def normal(*shape, by=1.0):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).mul_(by).to(dtype)

    s = {"case": dict(case), "max_new": max(new), "tokens": tokens}
    s["k_pages"] = torch.empty(pages, hk, page, d, device=dev, dtype=dtype).normal_(0.0, 1.0, generator=g)
    s["v_pages"] = torch.empty(pages, hk, page, d, device=dev, dtype=dtype).normal_(0.0, 1.0, generator=g)
    # Pages in any order; table entries that no key uses hold -1.
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int32)
    table = torch.full((len(lens), max(used) + 1), -1, device=dev, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    s["page_table"] = table
    s["seq_lens"] = torch.tensor(lens, device=dev, dtype=torch.int32)
    offsets = [0]
    for m in new:
        offsets.append(offsets[-1] + m)
    s["q_offsets"] = torch.tensor(offsets, device=dev, dtype=torch.int32)
    if case["op"] == "append":
        # One fused projection's output: the heads' rows are strided views.
        qkv = normal(tokens, hq + 2 * hk, d, by=2.0)
        s["q"], s["k"], s["v"] = qkv.split([hq, hk, hk], dim=1)
        r = case["rotary"]
        inv = ROTARY_BASE ** (-torch.arange(0, r, 2, device=dev, dtype=torch.float64) / r)
        angle = torch.arange(max(lens) + 1, device=dev, dtype=torch.float64)[:, None] * inv
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], dim=1).float()
        s["q_norm"] = (1 + 0.2 * normal(d).float()).to(dtype) if case["norm"] else None
        s["k_norm"] = (1 + 0.2 * normal(d).float()).to(dtype) if case["norm"] else None
    else:
        s["q"] = normal(tokens, hq, d, by=1.5)
        s["sink_logits"] = torch.randn(hq, generator=g, device=dev) if case["logits"] else None
    if own:
        import mxfp4_routed_expert_route_gb300 as lib
        s["cache"] = lib.PagedKVCache(s["k_pages"], s["v_pages"])
        s["seqs"] = lib.PagedSequences(s["page_table"], s["seq_lens"],
                                       None if case["op"] == "decode" else s["q_offsets"])
    return s


def run(state):
    case = state["case"]
    if not own:
        return (_plain_append if case["op"] == "append" else _plain_attention)(state)
    import mxfp4_routed_expert_route_gb300 as lib
    if case["op"] == "append":
        q = lib.append_kv(state["q"], state["k"], state["v"], state["cache"], state["seqs"],
                          cos_sin=state["cos_sin"], interleaved=case["interleaved"],
                          q_norm=state["q_norm"], k_norm=state["k_norm"], eps=EPS)
        return [q, state["k_pages"], state["v_pages"]]
    attention = lib.paged_attention_decode if case["op"] == "decode" else lib.paged_attention_prefill
    return attention(state["q"], state["cache"], state["seqs"], window=case["window"],
                     sinks=case["sinks"], sink_logits=state["sink_logits"])


# --------------------------------------------------------------- plain form --
def _rows(s):
    """Sequence, index among its new tokens and position of every token."""
    off, lens = s["q_offsets"].long(), s["seq_lens"].long()
    t = torch.arange(s["tokens"], device=off.device)
    b = torch.searchsorted(off, t, right=True) - 1
    i = t - off[b]
    return b, i, lens[b] - (off[b + 1] - off[b]) + i


def _plain_turn(x, norm, cos, sin, interleaved):
    x = x.float()
    if norm is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * norm.float()
    half = cos.shape[-1]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
    else:
        a, b = turned[..., :half], turned[..., half:]
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([turned, rest], -1)


def _plain_append(s):
    case, dtype = s["case"], s["q"].dtype
    b, _, pos = _rows(s)
    cos, sin = s["cos_sin"][pos][:, None].chunk(2, dim=-1)
    page = s["page_table"].long()[b, pos // case["page"]]
    slot = pos % case["page"]
    q = _plain_turn(s["q"], s["q_norm"], cos, sin, case["interleaved"]).to(dtype)
    s["k_pages"][page, :, slot] = _plain_turn(s["k"], s["k_norm"], cos, sin,
                                              case["interleaved"]).to(dtype)
    s["v_pages"][page, :, slot] = s["v"]
    return [q, s["k_pages"], s["v_pages"]]


def _plain_attention(s):
    case, q = s["case"], s["q"]
    hk, d, most = case["kv_heads"], case["head_dim"], s["max_new"]
    group = case["heads"] // hk
    seqs, dev = case["seqs"], q.device
    # Queries padded to (sequence, key head, group, new, width).
    off, lens = s["q_offsets"].long(), s["seq_lens"].long()
    i = torch.arange(most, device=dev)
    at = (off[:-1, None] + i).clamp(max=s["tokens"] - 1)
    x = q[at].float().view(seqs, most, hk, group, d).permute(0, 2, 3, 1, 4)
    pos = (lens - (off[1:] - off[:-1]))[:, None] + i
    # Keys and values gathered to (sequence, key head, key, width).
    table = s["page_table"].long().clamp(min=0)
    key = torch.arange(table.shape[1] * case["page"], device=dev)
    k, v = (p[table].float().transpose(1, 2).reshape(seqs, hk, -1, d)
            for p in (s["k_pages"], s["v_pages"]))
    k, v = (torch.where((key < lens[:, None])[:, None, :, None], p, 0.0) for p in (k, v))
    score = torch.matmul(x.reshape(seqs, hk, -1, d), k.transpose(-1, -2))
    score = score.view(seqs, hk, group, most, -1).mul_(1.0 / math.sqrt(d))
    seen = (key <= pos[..., None]) & (key < lens[:, None, None])
    if case["window"]:
        seen = seen & ((pos[..., None] - key < case["window"]) | (key < case["sinks"]))
    score.masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if s["sink_logits"] is not None:
        logit = s["sink_logits"].view(1, hk, group, 1, 1)
        top = torch.maximum(top, logit)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    if s["sink_logits"] is not None:
        total = total + (logit - top).exp()
    y = torch.matmul(p.view(seqs, hk, -1, key.numel()), v).view(seqs, hk, group, most, d)
    y = torch.where(total > 0, y / total, 0.0)
    b, i, _ = _rows(s)
    return y.permute(0, 3, 1, 2, 4).reshape(seqs, most, case["heads"], d)[b, i].to(q.dtype)


# ------------------------------------------------------------- 64 bits -------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    hist, new = _lengths(case)
    page, d = case["page"], case["head_dim"]
    if case["op"] == "append":
        q_out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
        k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
        half = case["rotary"] // 2
        n = 0
        for b, (h, m) in enumerate(zip(hist, new)):
            pos = torch.arange(h, h + m, device="cuda")
            phase = torch.complex(s["cos_sin"][pos, :half].double(), s["cos_sin"][pos, half:].double())
            where = s["page_table"][b, pos // page].long()
            for src, w, out in ((s["q"], s["q_norm"], "q"), (s["k"], s["k_norm"], "k")):
                x = src[n:n + m].double()
                if w is not None:
                    x = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w.double()
                pair = x[..., :2 * half].unflatten(-1, (half, 2) if case["interleaved"] else (2, half))
                if not case["interleaved"]:
                    pair = pair.transpose(-1, -2)
                z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * phase[:, None])
                if not case["interleaved"]:
                    z = z.transpose(-1, -2)
                x = torch.cat([z.flatten(-2), x[..., 2 * half:]], -1)
                if out == "q":
                    q_out[n:n + m] = x
                else:
                    k_pages[where, :, pos % page] = x
            v_pages[where, :, pos % page] = s["v"][n:n + m].double()
            n += m
        return [q_out, k_pages, v_pages]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group = case["heads"] // case["kv_heads"]
    n = 0
    for b, (h, m) in enumerate(zip(hist, new)):
        pages = s["page_table"][b, :-(-(h + m) // page)].long()
        key = torch.arange(h + m, device="cuda")[None]
        at = torch.arange(h, h + m, device="cuda")[:, None]
        hidden = key > at
        if case["window"]:
            hidden |= (key <= at - case["window"]) & (key >= case["sinks"])
        for c in range(case["kv_heads"]):
            k, v = (p[pages, c].reshape(-1, d)[:h + m].double() for p in (s["k_pages"], s["v_pages"]))
            for e in range(c * group, (c + 1) * group):
                z = s["q"][n:n + m, e].double() @ k.T / math.sqrt(d)
                z[hidden] = -math.inf
                if s["sink_logits"] is not None:  # one more column, without a value
                    z = torch.cat([z, s["sink_logits"][e].double().expand(m, 1)], 1)
                z = torch.softmax(z, -1)
                out[n:n + m, e] = z[:, :h + m] @ v
        n += m
    return out

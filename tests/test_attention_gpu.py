"""The attention operators against plain 64-bit forms (attention_ref.py, with
the derivation of the bounds): paged append, decode and prefill."""
import math

import pytest
import torch

import attention_ref as ref
import mxfp4_routed_expert_route_gb300 as lib

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(lens, new, *, heads=8, kv_heads=2, dim=64, page=16, dtype=BF16, seed=0, fused=False,
         slot_major=False, spare=3, fill=0.0):
    """Inputs of one call: pages in a random order, table entries and slots
    that no key uses filled with ids out of range and with `fill`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    used = [-(-n // page) for n in lens]
    pages = sum(used) + spare
    shape = (pages, page, kv_heads, dim) if slot_major else (pages, kv_heads, page, dim)

    def cache():
        x = torch.randn(shape, generator=g, device="cuda").to(dtype)
        return x.transpose(1, 2) if slot_major else x

    kp, vp = cache(), cache()
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((len(lens), max(used, default=0) + 2), 1 << 30, dtype=torch.int32,
                       device="cuda")
    at = 0
    live = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        for i in range(u):
            live[int(order[at + i]), :min(page, lens[b] - i * page)] = True
        at += u
    if fill:
        for p in (kp, vp):
            p.masked_fill_(~live[:, None, :, None], fill)
    offsets = [0]
    for m in new:
        offsets.append(offsets[-1] + m)
    T = offsets[-1]
    if fused:
        q = torch.randn(T, heads + 2 * kv_heads, dim, generator=g, device="cuda").to(dtype)[:, :heads]
    else:
        q = torch.randn(T, heads, dim, generator=g, device="cuda").to(dtype)
    d = dict(q=q, kp=kp, vp=vp, table=table, lens=list(lens), offsets=offsets)
    d["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    d["q_offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    d["cache"] = lib.PagedKVCache(kp, vp)
    d["logits"] = torch.randn(heads, generator=g, device="cuda")
    return d


def call(d, decode, logits=False, **kw):
    seqs = lib.PagedSequences(d["table"], d["seq_lens"], None if decode else d["q_offsets"])
    f = lib.paged_attention_decode if decode else lib.paged_attention_prefill
    return f(d["q"], d["cache"], seqs, sink_logits=d["logits"] if logits else None, **kw)


def check(d, decode, logits=False, **kw):
    lib.page_errors()
    got = call(d, decode, logits, **kw)
    want, bound = ref.attention(d["q"], d["kp"], d["vp"], d["table"], d["lens"], d["offsets"],
                                sink_logits=d["logits"] if logits else None,
                                **{k: v for k, v in kw.items() if k in ("scale", "window", "sinks")})
    err = (got.double() - want).abs()
    same = (got.double() == want) | (torch.isnan(want) & torch.isnan(got))
    ratio = torch.where(same, 0.0, err / bound)
    assert not torch.isnan(ratio).any(), "NaN in the result"
    worst = float(ratio.max()) if ratio.numel() else 0.0
    assert worst <= 1.0, f"max err/bound {worst:.3g}"
    fine = torch.isfinite(want)
    norm = float(want[fine].norm())
    if norm:
        rms = float(err[fine].norm()) / norm
        # Rounding the weights and the result to the token dtype each adds a
        # relative error spread over [-u, u], u / sqrt(3) of root mean square.
        assert rms <= (5e-3 if got.dtype == BF16 else 5e-6), f"relative error {rms:.3g}"
    assert lib.page_errors() == 0 and lib.wait_timeouts() == 0
    return got


LENS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 513, 1000]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (6, 2), (7, 1), (16, 2), (17, 1), (40, 2)])
def test_decode_lengths_and_groups(dtype, dim, heads, kv_heads):
    d = make(LENS, [1] * len(LENS), heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
             fill=math.nan)
    check(d, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 1024])
def test_decode_pages(dtype, page):
    check(make(LENS, [1] * len(LENS), page=page, dtype=dtype, dim=128, fill=math.inf), True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (64, 0), (100, 70), (128, 4),
                                          (129, 500), (5000, 9)])
@pytest.mark.parametrize("logits", [False, True])
def test_decode_window(dtype, window, sinks, logits):
    check(make(LENS, [1] * len(LENS), dtype=dtype, fill=math.nan), True, logits, window=window,
          sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,heads,kv_heads,lens", [
    (128, 8, 1, [20011]), (64, 8, 2, [9001, 3, 12345]), (128, 7, 1, [1, 15000, 2, 0, 8192]),
    (64, 64, 1, [5000, 77])])
def test_decode_long_sequences_are_split_and_joined(dtype, dim, heads, kv_heads, lens):
    d = make(lens, [1] * len(lens), heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=32,
             fill=math.nan)
    first = check(d, True, logits=True)
    for _ in range(3):     # the workspace is left as it was found; the sums have a fixed order
        assert torch.equal(call(d, True, True), first)


def test_decode_many_sequences():
    lens = [(37 * i) % 301 for i in range(700)]
    check(make(lens, [1] * len(lens), heads=4, kv_heads=2, fill=math.nan), True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (6, 2), (7, 1), (16, 2), (80, 2)])
def test_prefill_ragged(dtype, dim, heads, kv_heads):
    # Prompts, chunks behind histories that end inside a page, single tokens,
    # a sequence without new tokens and an empty one.
    lens = [1, 130, 16, 0, 77, 300, 40, 129]
    new = [1, 130, 16, 0, 0, 33, 1, 128]
    check(make(lens, new, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, fill=math.nan),
          False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [8, 32, 64, 128, 1024])
def test_prefill_pages(dtype, page):
    check(make([200, 515, 64], [200, 100, 1], page=page, dtype=dtype, dim=128, fill=math.inf), False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 3), (64, 0), (100, 150), (128, 4),
                                          (5000, 9)])
@pytest.mark.parametrize("logits", [False, True])
def test_prefill_window(dtype, window, sinks, logits):
    check(make([700, 333, 900], [700, 20, 257], dtype=dtype, fill=math.nan), False, logits,
          window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128])
def test_prefill_long(dtype, dim):
    check(make([2500, 1111], [2500, 700], heads=4, kv_heads=2, dim=dim, dtype=dtype), False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_few_rows_behind_a_long_history(dtype):
    d = make([20000, 9000], [5, 3], heads=8, kv_heads=1, dim=128, dtype=dtype, page=64,
             fill=math.nan)
    first = check(d, False, logits=True)
    assert torch.equal(call(d, False, True), first)
    check(d, False, window=6000, sinks=100)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_of_single_tokens_is_decode(dtype):
    lens = [5, 100, 1, 257]
    d = make(lens, [1] * 4, dtype=dtype)
    check(d, True)
    check(d, False)
    seqs = lib.PagedSequences(d["table"], d["seq_lens"])       # no offsets
    a = lib.paged_attention_prefill(d["q"], d["cache"], seqs)
    assert torch.equal(a, call(d, False))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_more_new_tokens_than_keys_leaves_rows_empty(dtype):
    # The first rows have negative positions: they see nothing.
    d = make([3, 40], [10, 60], dtype=dtype, fill=math.nan)
    out = check(d, False)
    assert not out[:7].any() and not out[10:30].any() and out[7:10].any()
    check(d, False, logits=True)


def test_rows_past_the_last_sequence_are_zeros():
    d = make([50, 20], [50, 20])
    seqs = lib.PagedSequences(d["table"], d["seq_lens"], d["q_offsets"])
    q = torch.randn(333, 8, 64, device="cuda", dtype=BF16)
    q[:70] = d["q"]
    out = torch.full_like(q, 7.0)
    lib.paged_attention_prefill(q, d["cache"], seqs, out=out)
    assert torch.equal(out[:70], call(d, False)) and not out[70:].any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
def test_strides(dtype, decode):
    # Queries sliced from a fused projection, pages with the slots before the
    # heads, keys and values of one tensor.
    lens, new = [100, 37, 260], [1, 1, 1] if decode else [100, 3, 90]
    d = make(lens, new, dtype=dtype, dim=128, fused=True, slot_major=True, fill=math.nan)
    check(d, decode)
    both = torch.stack([d["kp"], d["vp"]], 1)
    d["kp"], d["vp"] = both[:, 0], both[:, 1]
    d["cache"] = lib.PagedKVCache(d["kp"], d["vp"])
    check(d, decode, logits=True, window=50, sinks=2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_prefill_keys_not_seen_do_not_reach_a_row(dtype, value):
    # A value or key that later rows see must not touch the earlier ones.
    lens, new = [200, 300], [200, 150]
    d = make(lens, new, dtype=dtype)
    clean = call(d, False, window=90, sinks=2)
    for b, j in ((0, 120), (1, 170)):
        page, slot = int(d["table"][b, j // 16]), j % 16
        d["vp"][page, :, slot, 5] = value
    got = check(d, False, window=90, sinks=2)
    assert torch.equal(got[:120], clean[:120]) and torch.equal(got[200:220], clean[200:220])
    assert torch.equal(got[310:350, :, :], clean[310:350])     # past the window of key 170
    page, slot = int(d["table"][0, 120 // 16]), 120 % 16
    d["kp"][page, :, slot, 3] = value
    got = call(d, False, window=90, sinks=2)
    assert torch.equal(got[:120], clean[:120]) and torch.equal(got[200:220], clean[200:220])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_that_are_seen_keep_their_infinities(dtype):
    d = make([70], [1], dtype=dtype)
    page, slot = int(d["table"][0, 33 // 16]), 33 % 16
    d["vp"][page, :, slot, 7] = math.inf
    out = call(d, True)
    assert torch.isinf(out[:, :, 7]).all() and torch.isfinite(out[:, :, :7]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
def test_large_scores(dtype, decode):
    # Scores of hundreds, of both signs: the softmax keeps its maximum.
    lens, new = [300, 90], [1, 1] if decode else [300, 50]
    d = make(lens, new, dtype=dtype)
    d["q"].mul_(40)
    got, (want, _) = call(d, decode), ref.attention(
        d["q"], d["kp"], d["vp"], d["table"], d["lens"], d["offsets"])
    err = (got.double() - want).norm() / want.norm()
    assert err <= (1e-2 if dtype == BF16 else 1e-4)
    check(d, decode, scale=0.001)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
def test_page_ids_out_of_range_read_as_zeros_and_are_counted(dtype, decode):
    lens, new = [64, 40], [1, 1] if decode else [30, 40]
    d = make(lens, new, dtype=dtype)
    bad = d["table"].clone()
    bad[0, 1], bad[1, 0] = d["kp"].shape[0], -3
    zero = torch.cat([d["kp"], torch.zeros_like(d["kp"][:1])]), \
        torch.cat([d["vp"], torch.zeros_like(d["vp"][:1])])
    fixed = bad.clone()
    fixed[0, 1] = fixed[1, 0] = d["kp"].shape[0]
    want = call(dict(d, cache=lib.PagedKVCache(*zero), table=fixed), decode)
    assert lib.page_errors() == 0
    assert torch.equal(call(dict(d, table=bad), decode), want)
    assert lib.page_errors() > 0


@pytest.mark.parametrize("decode", [True, False])
def test_lengths_beyond_the_table_are_cut_and_counted(decode):
    d = make([48, 31], [1, 1] if decode else [5, 31])
    d["table"] = d["table"][:, :3].contiguous()      # room for 48 keys
    want = call(d, decode)
    assert lib.page_errors() == 0
    d["seq_lens"] = torch.tensor([1000, 31], dtype=torch.int32, device="cuda")
    assert torch.equal(call(d, decode), want)
    assert lib.page_errors() > 0


@pytest.mark.parametrize("decode", [True, False])
def test_other_streams_and_graphs(decode):
    lens, new = [400, 77, 3000], [1, 1, 1] if decode else [100, 77, 9]
    d = make(lens, new, dim=128, heads=16)
    want = call(d, decode)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call(d, decode)
    s.synchronize()
    assert torch.equal(got, want)
    ws = lib.attention_workspace("cuda")
    g = torch.cuda.CUDAGraph()
    out = torch.empty_like(d["q"])
    with torch.cuda.graph(g):
        call(d, decode, out=out, workspace=ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    # Lengths are read when the graph runs.
    d["seq_lens"].copy_(torch.tensor([399, 77, 2001], dtype=torch.int32))
    d["lens"] = [399, 77, 2001]
    g.replay()
    assert torch.equal(out, check(d, decode))


@pytest.mark.parametrize("decode", [True, False])
def test_offsets_beyond_32_bits(decode):
    # More than 2^31 elements of keys: pages at the far end.
    page, kv_heads, dim = 1024, 8, 128
    pages = (1 << 31) // (page * kv_heads * dim) + 9
    kp = torch.empty(pages, kv_heads, page, dim, dtype=BF16, device="cuda")
    vp = torch.empty_like(kp)
    d = make([1500], [1] if decode else [200], heads=8, kv_heads=kv_heads, dim=dim, page=page)
    ids = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    for i in range(2):
        kp[pages - 1 - 2 * i] = d["kp"][int(d["table"][0, i])]
        vp[pages - 1 - 2 * i] = d["vp"][int(d["table"][0, i])]
    want = call(d, decode)
    got = call(dict(d, cache=lib.PagedKVCache(kp, vp), table=ids), decode)
    assert torch.equal(got, want)


def test_nothing_to_do():
    d = make([], [])
    d["table"] = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    assert call(d, True).shape == (0, 8, 64)
    assert call(d, False).shape == (0, 8, 64)
    d = make([0, 0], [0, 0])
    assert call(d, False).shape == (0, 8, 64)
    assert not call(make([0, 0], [1, 1]), True).any()


def test_gradient_free_paths_leave_their_inputs():
    d = make([100, 60], [40, 60])
    before = [t.clone() for t in (d["q"], d["kp"], d["vp"], d["table"], d["seq_lens"])]
    call(d, False)
    call(make([100, 60], [1, 1]), True)
    for t, b in zip((d["q"], d["kp"], d["vp"], d["table"], d["seq_lens"]), before):
        assert torch.equal(t, b)


# ------------------------------------------------------------------ append --
def rope_table(positions, rotary):
    inv = 10000.0 ** (-torch.arange(0, rotary, 2, device="cuda", dtype=torch.float64) / rotary)
    angle = torch.arange(positions, device="cuda", dtype=torch.float64)[:, None] * inv
    return torch.cat([angle.cos(), angle.sin()], 1).float()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,rotary", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 32),
                                        (128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norms", ["both", "none", "query"])
def test_append(dtype, dim, rotary, interleaved, norms):
    lens, new = [5, 16, 33, 0, 90, 21], [5, 1, 17, 0, 40, 0]
    d = make(lens, new, heads=6, kv_heads=3, dim=dim, dtype=dtype, slot_major=norms == "query")
    g = torch.Generator(device="cuda").manual_seed(7)
    T = d["offsets"][-1]
    qkv = torch.randn(T, 12, dim, generator=g, device="cuda").mul_(3).to(dtype)
    q, k, v = qkv.split([6, 3, 3], 1)
    w = [(1 + 0.3 * torch.randn(dim, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    kw = dict(cos_sin=rope_table(95, rotary) if rotary else None, interleaved=interleaved,
              q_norm=w[0] if norms != "none" else None, k_norm=w[1] if norms == "both" else None,
              eps=1e-5)
    (qw, qb), (kw_, kb), vw = ref.append(q, k, v, d["kp"], d["vp"], d["table"], lens, d["offsets"],
                                         **kw)
    lib.page_errors()
    seqs = lib.PagedSequences(d["table"], d["seq_lens"], d["q_offsets"])
    got = lib.append_kv(q, k, v, d["cache"], seqs, **kw)
    assert lib.page_errors() == 0
    assert ((got.double() - qw).abs() <= qb).all()
    assert ((d["kp"].double() - kw_).abs() <= kb).all()      # untouched slots: equal
    assert torch.equal(d["vp"].double(), vw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("seqs", [1, 3, 100, 1100])
def test_append_one_token_each(dtype, seqs):
    lens = [1 + (i * 13) % 70 for i in range(seqs)]
    d = make(lens, [1] * seqs, heads=5, kv_heads=1, dim=64, dtype=dtype, page=8)
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = (torch.randn(seqs, n, 64, generator=g, device="cuda").to(dtype) for n in (5, 1, 1))
    cs = rope_table(71, 64)
    (qw, qb), (kw_, kb), vw = ref.append(q, k, v, d["kp"], d["vp"], d["table"], lens, d["offsets"],
                                         cos_sin=cs)
    kp, vp = d["kp"].clone(), d["vp"].clone()
    got = lib.append_kv(q, k, v, d["cache"], lib.PagedSequences(d["table"], d["seq_lens"]),
                        cos_sin=cs)
    assert ((got.double() - qw).abs() <= qb).all()
    assert ((d["kp"].double() - kw_).abs() <= kb).all()
    assert torch.equal(d["vp"].double(), vw)
    # The same through offsets, bit for bit.
    seqs_off = lib.PagedSequences(d["table"], d["seq_lens"], d["q_offsets"])
    assert torch.equal(got, lib.append_kv(q, k, v, lib.PagedKVCache(kp, vp), seqs_off, cos_sin=cs))
    assert torch.equal(kp, d["kp"]) and torch.equal(vp, d["vp"])


def test_append_drops_and_counts_what_is_out_of_range():
    d = make([20, 20, 2, 40], [3, 2, 5, 2], heads=2, kv_heads=1)
    T = d["offsets"][-1]
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(T + 4, n, 64, generator=g, device="cuda").to(BF16) for n in (2, 1, 1))
    cs = rope_table(39, 64)          # position 39 has no row
    bad = d["table"].clone()
    bad[0, 1] = -1                   # positions 17 .. 19 of sequence 0
    (qw, qb), (kw_, kb), vw = ref.append(
        q[:T], k[:T], v[:T], d["kp"], d["vp"], d["table"], [20, 20, 2, 40], d["offsets"],
        cos_sin=torch.cat([cs, cs[:1]]))
    kp0, vp0 = d["kp"].clone(), d["vp"].clone()
    lib.page_errors()
    got = lib.append_kv(q, k, v, d["cache"],
                        lib.PagedSequences(bad, d["seq_lens"], d["q_offsets"]), cos_sin=cs)
    # 3 tokens without a page, 3 with negative positions, 1 past the table of angles
    assert lib.page_errors() == 7
    live = [0, 1, 2, 3, 4, 8, 9, 10]
    assert ((got[live].double() - qw[live]).abs() <= qb[live]).all()
    assert not got[[5, 6, 7, 11, 12, 13, 14, 15]].any()
    # Only sequence 1, the last two tokens of sequence 2 and position 38 were written.
    changed = (d["kp"] != kp0).any(-1).any(1).nonzero().tolist()
    want = sorted([[int(d["table"][b, p // 16]), p % 16]
                   for b, p in ((1, 18), (1, 19), (2, 0), (2, 1), (3, 38))])
    assert sorted(changed) == want
    for page, slot in want:
        assert ((d["kp"][page, :, slot].double() - kw_[page, :, slot]).abs()
                <= kb[page, :, slot]).all()
        assert torch.equal(d["vp"][page, :, slot].double(), vw[page, :, slot])


def test_append_offsets_beyond_32_bits():
    page, kv_heads, dim = 1024, 8, 128
    pages = (1 << 31) // (page * kv_heads * dim) + 5
    kp = torch.empty(pages, kv_heads, page, dim, dtype=BF16, device="cuda")
    vp = torch.empty_like(kp)
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1000], dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(1, n, dim, device="cuda").to(BF16) for n in (8, 8, 8))
    out = lib.append_kv(q, k, v, lib.PagedKVCache(kp, vp), lib.PagedSequences(table, lens))
    assert torch.equal(out, q)
    assert torch.equal(kp[-1, :, 999], k[0]) and torch.equal(vp[-1, :, 999], v[0])


# --------------------------------------------------------------- refusals --
def test_refusals():
    d = make([40, 20], [40, 20])
    one = lib.PagedSequences(d["table"], d["seq_lens"])
    many = lib.PagedSequences(d["table"], d["seq_lens"], d["q_offsets"])
    q, cache = d["q"], d["cache"]
    with pytest.raises(ValueError):
        lib.paged_attention_decode(q[:2], cache, many)              # offsets in a decode call
    with pytest.raises(ValueError):
        lib.paged_attention_decode(q[:3], cache, one)               # a row too many
    with pytest.raises(ValueError):
        lib.paged_attention_prefill(q[:3], cache, one)
    with pytest.raises(ValueError):
        lib.paged_attention_prefill(q[:, :7], cache, many)          # 7 heads over 2
    with pytest.raises(TypeError):
        lib.paged_attention_prefill(q.float(), cache, many)
    with pytest.raises(TypeError):
        lib.paged_attention_prefill(q.half(), cache, many)
    with pytest.raises(ValueError):
        lib.paged_attention_prefill(q[..., :32], cache, many)
    with pytest.raises(ValueError):
        lib.paged_attention_prefill(q, cache, many, window=-1)
    with pytest.raises(ValueError):
        lib.paged_attention_prefill(q, cache, many, sinks=-1, window=4)
    with pytest.raises(ValueError):
        lib.paged_attention_prefill(q, cache, many, sink_logits=d["logits"][:3])
    with pytest.raises(ValueError):
        lib.paged_attention_prefill(q, cache, many, out=q[:3])
    with pytest.raises(ValueError):
        lib.paged_attention_prefill(q.cpu(), cache, many)
    with pytest.raises(lib.MXFP4Error):
        lib.paged_attention_prefill(q, cache, many, out=q)          # overlaps an input
    with pytest.raises(lib.MXFP4Error):
        lib.paged_attention_prefill(q, cache, many, scale=math.inf)
    with pytest.raises(lib.MXFP4Error):
        lib.paged_attention_prefill(q, cache, many,
                                    workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    wide = torch.zeros(60, 8, 65, device="cuda", dtype=BF16)[..., :64]     # 130-byte rows
    with pytest.raises(lib.MXFP4Error):
        lib.paged_attention_prefill(wide, cache, many)
    k = torch.zeros(60, 2, 64, device="cuda", dtype=BF16)
    with pytest.raises(ValueError):
        lib.append_kv(q, k[:5], k, cache, many)
    with pytest.raises(ValueError):
        lib.append_kv(q, k, k, cache, many, cos_sin=torch.zeros(50, 24, device="cuda"))
    with pytest.raises(ValueError):
        lib.append_kv(q, k, k, cache, many, q_norm=torch.zeros(64, device="cuda"))
    with pytest.raises(lib.MXFP4Error):
        lib.append_kv(q, k, k, cache, many, eps=-1.0)
    with pytest.raises(lib.MXFP4Error):
        lib.append_kv(q, k, k, cache, many, q_out=q)
    with pytest.raises(ValueError):
        lib.PagedKVCache(torch.zeros(4, 2, 12, 64, device="cuda"),
                         torch.zeros(4, 2, 12, 64, device="cuda"))          # page size 12
    with pytest.raises(ValueError):
        lib.PagedKVCache(torch.zeros(4, 2, 16, 80, device="cuda"),
                         torch.zeros(4, 2, 16, 80, device="cuda"))          # head_dim 80
    with pytest.raises(TypeError):
        lib.PagedKVCache(torch.zeros(4, 2, 16, 64, device="cuda"),
                         torch.zeros(4, 2, 16, 64, device="cuda", dtype=BF16))
    with pytest.raises(TypeError):
        lib.PagedSequences(d["table"].long(), d["seq_lens"])
    with pytest.raises(ValueError):
        lib.PagedSequences(d["table"], d["seq_lens"][:1])


# ------------------------------------------------------- many sequences ----
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("seqs", [30, 31, 100, 700])
def test_prefill_many_sequences(dtype, seqs):
    # Prompts and chunks of 0 to 40 new tokens behind histories of 0 to 60.
    new = [(13 * i) % 41 for i in range(seqs)]
    lens = [n + (29 * i) % 61 for i, n in enumerate(new)]
    d = make(lens, new, heads=4, kv_heads=2, dtype=dtype, fill=math.nan)
    check(d, False)
    check(d, False, logits=True, window=20, sinks=3)


def test_prefill_many_sequences_of_one_token():
    lens = [1 + (37 * i) % 301 for i in range(90)]
    d = make(lens, [1] * 90, heads=6, kv_heads=2, fill=math.nan)
    want = check(d, False)
    seqs = lib.PagedSequences(d["table"], d["seq_lens"])
    assert torch.equal(lib.paged_attention_prefill(d["q"], d["cache"], seqs), want)


def test_decode_more_sequences_than_a_launch_takes():
    lens = [(41 * i) % 97 for i in range(2500)]
    d = make(lens, [1] * 2500, heads=2, kv_heads=1, page=32, spare=1)
    got = call(d, True)
    for b0 in (0, 1000, 2400):      # the 64-bit form of a few stretches
        part = dict(d, q=d["q"][b0:b0 + 100], table=d["table"][b0:b0 + 100],
                    lens=lens[b0:b0 + 100], offsets=list(range(101)))
        want, bound = ref.attention(part["q"], d["kp"], d["vp"], part["table"], part["lens"],
                                    part["offsets"])
        assert ((got[b0:b0 + 100].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
def test_calls_in_a_row_do_not_disturb_each_other(dtype, decode):
    # Different inputs through one workspace, nothing waited for between.
    cases = [make([900 + 300 * i, 40, 2000 - 100 * i], [1] * 3 if decode else [30 + i, 40, 9],
                  dim=64 if i % 2 else 128, dtype=dtype, seed=i, fill=math.nan) for i in range(4)]
    kw = dict(window=150, sinks=5)
    want = [(call(d, decode), call(d, decode, **kw)) for d in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(25):
        got.append([(call(d, decode), call(d, decode, **kw)) for d in cases])
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert lib.wait_timeouts() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (6, 2), (100, 1)])
def test_prefill_split_over_the_keys(dtype, dim, heads, kv_heads):
    # Few rows behind histories long and short: units in many parts, in few
    # and whole, rows that see nothing, a part that only the later row tile
    # reaches.
    lens, new = [6000, 1025, 130, 3, 0, 2048], [70, 3, 130, 5, 0, 300]
    d = make(lens, new, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype, page=32,
             fill=math.nan)
    first = check(d, False, logits=True)
    for _ in range(3):
        assert torch.equal(call(d, False, True), first)
    check(d, False, window=1500, sinks=200)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_not_finite_in_a_split_unit(dtype):
    lens, new = [5000], [40]
    d = make(lens, new, heads=4, kv_heads=1, dtype=dtype)
    clean = call(d, False, window=4000, sinks=50)
    for j in (4975, 970, 20):        # seen by the last rows, by the first, by all
        page, slot = int(d["table"][0, j // 16]), j % 16
        d["vp"][page, :, slot, 9] = math.inf
        got = check(d, False, window=4000, sinks=50)
        if j == 4975:
            assert torch.equal(got[:15, :, :9], clean[:15, :, :9])


@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv_heads", [(100, 1), (128, 1), (66, 2)])
def test_many_heads_to_a_key_head(decode, dtype, heads, kv_heads):
    lens = [70, 1, 333, 0]
    new = [1] * 4 if decode else [70, 1, 5, 0]
    check(make(lens, new, heads=heads, kv_heads=kv_heads, dtype=dtype, fill=math.nan), decode,
          logits=True)

"""Arguments and values at the edge of what the attention operators accept,
against the 64-bit forms of attention_ref.py."""
import math
import random

import pytest
import torch

import mxfp4_routed_expert_route_gb300 as lib
from mxfp4_routed_expert_route_gb300 import attention
from test_attention_gpu import BF16, F32, call, check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("sinks", [1 << 30, (1 << 31) - 64, (1 << 31) - 1, 1 << 40])
def test_every_first_token_stays_visible(dtype, dim, decode, sinks):
    # More first tokens than any length: the window hides nothing.
    lens = [100, 1550, 3000, 40, 1]
    d = make(lens, [1] * 5 if decode else [70, 33, 5, 40, 1], dim=dim, dtype=dtype, fill=math.nan)
    check(d, decode, window=50, sinks=sinks)
    check(d, decode, window=2000, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("window", [(1 << 30) - 1, 1 << 30, (1 << 31) - 2, (1 << 31) - 1, 1 << 40])
def test_windows_past_every_length_hide_nothing(dtype, decode, window):
    # Rows with negative positions among them: they still see nothing.
    d = make([3, 40, 700], [1] * 3 if decode else [10, 60, 300], dtype=dtype, fill=math.nan)
    got = check(d, decode, window=window, sinks=4)
    assert torch.equal(got, call(d, decode))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
def test_lengths_near_the_end_of_32_bits_are_cut(dtype, decode):
    d = make([48, 31], [1, 1] if decode else [5, 31], dtype=dtype)
    d["table"] = d["table"][:, :3].contiguous()      # room for 48 keys
    want = call(d, decode, window=20, sinks=2)
    d["seq_lens"] = torch.tensor([(1 << 31) - 1, 31], dtype=torch.int32, device="cuda")
    lib.page_errors()
    assert torch.equal(call(d, decode, window=20, sinks=2), want)
    assert lib.page_errors() > 0


# ------------------------------------------- values that are not finite ----
def plant(d, keys):
    """Values that are not finite: (sequence, key, column, value) of every
    key head."""
    size = d["vp"].shape[2]
    for b, j, col, value in keys:
        d["vp"][int(d["table"][b, j // size]), :, j % size, col] = value


def expected(clean, d, keys, window=0, sinks=0):
    """`clean`, the result without them, with what they do to it: a weight is
    positive, so a row that sees one has its value in that column (their sum,
    if it sees several), whatever the weight, and nothing else changes."""
    bad = torch.zeros(clean.shape, device="cuda")
    for b, j, col, value in keys:
        r0, r1 = d["offsets"][b], d["offsets"][b + 1]
        pos = torch.arange(d["lens"][b] - (r1 - r0), d["lens"][b], device="cuda")
        seen = j <= pos
        if window:
            seen &= (pos - j < window) | (j < sinks)
        bad[r0:r1, :, col] += torch.where(seen, value, 0.0)[:, None]
    return torch.where(bad == 0, clean, bad.to(clean.dtype))


def same(a, b):
    return bool(((a == b) | (torch.isnan(a) & torch.isnan(b))).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 64), (6, 2, 128), (8, 1, 64), (8, 1, 128)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (17, 3), (100, 0), (128, 4), (300, 150)])
def test_values_that_are_not_finite_change_what_sees_them_only(dtype, heads, kv_heads, dim, window,
                                                               sinks):
    # Keys in every place: seen by all rows of a unit, by its first or its last
    # ones, by rows of one of its row tiles; several to a row, of all kinds.
    lens, new = [900, 500, 64], [700, 500, 1]
    d = make(lens, new, heads=heads, kv_heads=kv_heads, dim=dim, dtype=dtype)
    clean = call(d, False, window=window, sinks=sinks)
    rng = random.Random(window * 10 + heads)
    keys = [(b, rng.randrange(n), rng.randrange(dim), rng.choice([math.inf, -math.inf, math.nan]))
            for b, n in enumerate(lens) for _ in range(40)]
    keys += [(0, 10, 5, math.inf), (0, 300, 6, math.inf), (1, 0, 7, math.nan), (1, 499, 8, -math.inf)]
    plant(d, keys)
    want = expected(clean, d, keys, window, sinks)
    for _ in range(10):      # whoever gets to a tile first, the bits are the same
        assert same(call(d, False, window=window, sinks=sinks), want)
    assert lib.wait_timeouts() == 0


@pytest.mark.parametrize("seqs", [20, 40])
def test_values_that_are_not_finite_in_many_sequences(seqs):
    new = [1 + (31 * i) % 150 for i in range(seqs)]
    lens = [n + (67 * i) % 201 for i, n in enumerate(new)]
    d = make(lens, new, heads=8, kv_heads=2, dim=128)
    clean = call(d, False, window=60)
    keys = [(b, n - 1 - (7 * b) % min(n, 40), b % 128, math.inf) for b, n in enumerate(lens)]
    plant(d, keys)
    assert same(call(d, False, window=60), expected(clean, d, keys, 60))


def test_values_that_are_not_finite_behind_a_long_history():
    # Units after one another in a CTA, 256 rows each behind 65000 keys: the
    # rows of the next units and of the other sequence are as without them.
    lens, new = [70000, 40000], [5000, 300]
    d = make(lens, new, heads=8, kv_heads=8, dim=64, page=64)
    clean = call(d, False)
    keys = [(0, 65000 + 250 * i, i, math.inf) for i in range(20)] + [(0, 69999, 40, math.nan)]
    plant(d, keys)
    assert same(call(d, False), expected(clean, d, keys))
    window = 30000
    plant(d, [(0, 35000 + 211 * i, 30, -math.inf) for i in range(20)])
    got = call(d, False, window=window)
    d["vp"].nan_to_num_(0.0, 0.0, 0.0)
    keys += [(0, 35000 + 211 * i, 30, -math.inf) for i in range(20)]
    assert same(got, expected(call(d, False, window=window), d, keys, window))
    assert lib.wait_timeouts() == 0


@pytest.mark.parametrize("heads,kv_heads", [(2, 2), (8, 1)])
def test_values_that_are_not_finite_in_units_split_over_the_keys(heads, kv_heads):
    lens, new = [30000, 9000], [40, 7]
    d = make(lens, new, heads=heads, kv_heads=kv_heads, dim=128, page=64)
    for window, sinks in ((0, 0), (20000, 100)):
        clean = call(d, False, window=window, sinks=sinks)
        keys = [(0, 29990, 3, math.inf), (0, 29965, 4, math.nan), (0, 9970, 5, math.inf),
                (0, 50, 6, -math.inf), (0, 15000, 7, math.inf), (1, 8994, 8, math.inf)]
        plant(d, keys)
        assert same(call(d, False, window=window, sinks=sinks),
                    expected(clean, d, keys, window, sinks))
        plant(d, [(b, j, col, 0.5) for b, j, col, _ in keys])


def test_nothing_but_nan_values():
    # What a model that has diverged leaves in its cache.
    d = make([4096, 700], [4096, 100], heads=16, kv_heads=2, dim=128, page=64)
    d["vp"].fill_(math.nan)
    assert torch.isnan(call(d, False)).all()
    assert torch.isnan(call(d, False, window=200, sinks=4)).all()
    assert lib.wait_timeouts() == 0


# ----------------------------------------------------------- workspaces ----
@pytest.mark.parametrize("decode", [True, False])
def test_a_captured_call_brings_its_workspace(decode):
    # The stream's kept one would be shared by the graph, wherever it runs, and
    # the stream's later calls.
    d = make([400, 3000], [1, 1] if decode else [100, 9], dim=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = call(d, decode)
    out = torch.empty_like(d["q"])
    g = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="workspace"):
        with torch.cuda.graph(g, stream=s):
            out.zero_()
            call(d, decode, out=out)
    # Two graphs of one stream, replayed side by side on others.
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for _ in range(2):
        ws = lib.attention_workspace()
        outs.append(torch.empty_like(d["q"]))
        graphs.append((torch.cuda.CUDAGraph(), ws))
        with torch.cuda.graph(graphs[-1][0], stream=s):
            for _ in range(20):
                call(d, decode, out=outs[-1], workspace=ws)
    torch.cuda.synchronize()
    for (g, _), t in zip(graphs, streams):
        with torch.cuda.stream(t):
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)


@pytest.mark.parametrize("decode", [True, False])
def test_the_workspace_is_looked_at(decode):
    d = make([40, 20], [1, 1] if decode else [30, 20])
    want = call(d, decode)
    ws = lib.attention_workspace()
    with pytest.raises(ValueError, match="workspace"):
        call(d, decode, workspace=ws.cpu())
    with pytest.raises(ValueError, match="workspace"):
        call(d, decode, workspace=torch.zeros(2, ws.numel(), dtype=torch.uint8, device="cuda").t())
    with pytest.raises(lib.MXFP4Error):
        call(d, decode, workspace=ws[256:])                  # too short
    with pytest.raises(lib.MXFP4Error):
        call(d, decode, workspace=torch.zeros(ws.numel() + 16, dtype=torch.uint8,
                                              device="cuda")[16:])          # not aligned
    # What counts is its bytes.
    assert torch.equal(call(d, decode, workspace=ws.view(torch.float32)), want)


def test_kept_workspaces_are_given_up_after_a_wait_that_gave_up(monkeypatch):
    # The count comes from a stand-in for the library's call.
    d = make([3000, 9000], [1, 1], dim=128)
    want = call(d, True)
    kept = attention._workspaces
    assert any(k[0] == 0 for k in kept)
    native = lib._native.load()
    old = next(t for k, t in kept.items() if k[0] == 0)

    class Library:
        count = 3

        def mxfp4el_wait_timeouts(self, stream, n):
            n._obj.value = self.count
            return 0

        def __getattr__(self, name):
            return getattr(native, name)

    monkeypatch.setattr(lib._native, "load", Library)
    assert lib.wait_timeouts() == 3 and not any(k[0] == 0 for k in kept)
    old[:4096].fill_(1)               # what a call that gave up might leave
    assert torch.equal(call(d, True), want)
    Library.count = 0
    assert lib.wait_timeouts() == 0 and any(k[0] == 0 for k in kept)
    assert torch.equal(call(d, True), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("decode", [True, False])
@pytest.mark.parametrize("window,sinks,bad", [(50, 0, 1), (37, 0, 1), (37, 2, 0), (1, 0, 3), (0, 0, 0)])
def test_every_page_id_out_of_range_is_counted(dtype, decode, window, sinks, bad):
    # 100 keys in pages of 32: windows that begin inside a page, first tokens.
    d = make([100], [1], dtype=dtype, page=32)
    d["table"][0, bad] = -7
    lib.page_errors()
    call(d, decode, window=window, sinks=sinks)
    assert lib.page_errors() > 0
    if window == 37 and sinks == 0:      # a page that nothing sees is not looked up
        d["table"][0, 0], d["table"][0, 1] = -7, 0
        call(d, decode, window=window)
        assert lib.page_errors() == 0


@pytest.mark.parametrize("decode", [True, False])
def test_a_table_of_one_page_each_in_any_layout(decode):
    # A column of page ids: its inner stride counts for nothing.
    d = make([9, 16, 3], [1, 1, 1] if decode else [5, 16, 1])
    want = call(d, decode)
    ids = d["table"][:, 0].clone()
    for table in (ids[None].t(), ids.view(3, 1), torch.stack([ids, ids], 1)[:, 1:]):
        assert torch.equal(call(dict(d, table=table), decode), want)
    with pytest.raises(ValueError):
        lib.PagedSequences(d["table"].t().contiguous().t(), d["seq_lens"])

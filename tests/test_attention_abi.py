"""Argument checks of the attention operators' C entry points: everything here
returns before any GPU work, so it runs without a GPU."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from mxfp4_routed_expert_route_gb300 import _native, build
    build.build()
    return _native.load()


def _cache(n, **kw):
    f = dict(k=1 << 32, v=1 << 33, num_pages=10, num_kv_heads=2, page_size=16, head_dim=64,
             k_page_stride=2 * 16 * 64, k_head_stride=16 * 64, k_slot_stride=64,
             v_page_stride=2 * 16 * 64, v_head_stride=16 * 64, v_slot_stride=64,
             dtype=n.DTYPE_BF16)
    f.update(kw)
    return n.KvCache(**f)


def _seqs(n, **kw):
    f = dict(page_table=1 << 24, seq_lens=1 << 25, q_offsets=1 << 26, num_seqs=3, max_pages=4,
             table_stride=4)
    f.update(kw)
    return n.Sequences(**f)


def _prefill(lib, cache, seqs, q=1 << 36, qt=512, qh=64, scale=0.1, window=0, sinks=0, logits=None,
             out=1 << 37, T=9, heads=8, ws=1 << 38, wsb=None):
    wsb = lib.mxfp4el_attention_workspace_size() if wsb is None else wsb
    return lib.mxfp4el_attention_prefill(
        q, qt, qh, ctypes.addressof(cache) if cache else None,
        ctypes.addressof(seqs) if seqs else None, scale, window, sinks, logits, out, T, heads, ws,
        wsb, None)


def _append(lib, cache, seqs, q=1 << 36, qt=512, qh=64, k=1 << 37, kt=128, kh=64, v=1 << 38,
            qn=None, kn=None, eps=1e-6, cs=1 << 39, pos=100, rot=64, out=1 << 40, T=9, heads=8):
    return lib.mxfp4el_append_kv(q, qt, qh, k, kt, kh, v, kt, kh, qn, kn, eps, cs, pos, rot, 0,
                                 ctypes.addressof(cache), ctypes.addressof(seqs), out, T, heads,
                                 None)


def test_cache_checks(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n
    s = _seqs(n)
    bad, big, dt = n.ERR_INVALID_ARGUMENT, n.ERR_TOO_LARGE, n.ERR_UNSUPPORTED_DTYPE
    for code, kw in ((dt, dict(dtype=7)), (bad, dict(head_dim=80)), (bad, dict(head_dim=256)),
                     (bad, dict(page_size=12)), (bad, dict(page_size=4)),
                     (bad, dict(page_size=2048)), (bad, dict(num_kv_heads=0)),
                     (bad, dict(num_pages=-1)), (bad, dict(k=None)), (bad, dict(v=(1 << 33) + 8)),
                     (bad, dict(k_slot_stride=68)), (bad, dict(v_slot_stride=32)),
                     (bad, dict(k_page_stride=-64)), (big, dict(num_pages=1 << 31)),
                     (big, dict(v_page_stride=1 << 50))):
        assert _prefill(lib, _cache(n, **kw), s) == code, kw
        assert _append(lib, _cache(n, **kw), s) == code, kw
    assert _prefill(lib, None, s) == bad


def test_attention_checks(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n
    c = _cache(n)
    s = _seqs(n)
    bad, big = n.ERR_INVALID_ARGUMENT, n.ERR_TOO_LARGE
    inf, nan = float("inf"), float("nan")
    for code, kw in ((bad, dict(T=-1)), (bad, dict(heads=0)), (bad, dict(heads=9)),
                     (bad, dict(window=-1)), (bad, dict(sinks=-2)), (bad, dict(scale=inf)),
                     (bad, dict(scale=nan)), (bad, dict(q=None)), (bad, dict(q=(1 << 36) + 2)),
                     (bad, dict(qt=65)), (bad, dict(qh=-64)), (bad, dict(out=None)),
                     (bad, dict(out=(1 << 37) + 8)), (big, dict(T=1 << 40)),
                     (big, dict(heads=2 * 129)), (n.ERR_ALIAS, dict(out=(1 << 36) + 16)),
                     (n.ERR_ALIAS, dict(out=(1 << 32) + 256)),
                     (n.ERR_ALIAS, dict(logits=(1 << 37) + 32)),
                     (n.ERR_WORKSPACE, dict(ws=None)), (n.ERR_WORKSPACE, dict(wsb=0)),
                     (n.ERR_WORKSPACE, dict(ws=(1 << 38) + 16)), (n.OK, dict(T=0))):
        assert _prefill(lib, c, s, **kw) == code, kw
    assert _prefill(lib, c, None) == bad
    for kw in (dict(seq_lens=None), dict(page_table=None), dict(num_seqs=-1), dict(max_pages=-1),
               dict(q_offsets=None)):          # 9 tokens of 3 sequences need offsets
        assert _prefill(lib, c, _seqs(n, **kw)) == bad, kw
    # decode takes no offsets
    f = lib.mxfp4el_attention_decode
    args = (1 << 36, 512, 64, ctypes.addressof(c), ctypes.addressof(s), 0.1, 0, 0, None, 1 << 37, 8,
            1 << 38, lib.mxfp4el_attention_workspace_size(), None)
    assert f(*args) == bad


def test_append_checks(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n
    c, s = _cache(n), _seqs(n)
    bad, big = n.ERR_INVALID_ARGUMENT, n.ERR_TOO_LARGE
    for code, kw in ((bad, dict(T=-1)), (bad, dict(heads=0)), (bad, dict(rot=24)),
                     (bad, dict(rot=80)), (bad, dict(rot=-16)), (bad, dict(pos=-1)),
                     (bad, dict(eps=-1.0)), (bad, dict(eps=float("nan"))), (bad, dict(cs=None)),
                     (bad, dict(cs=(1 << 39) + 4)), (bad, dict(qn=(1 << 41) + 2)),
                     (bad, dict(k=None)), (bad, dict(kt=65)), (bad, dict(out=None)),
                     (big, dict(T=1 << 40)), (n.ERR_ALIAS, dict(out=1 << 36)),
                     (n.ERR_ALIAS, dict(k=(1 << 32) + 64)), (n.ERR_ALIAS, dict(out=1 << 33)),
                     (n.OK, dict(T=0))):
        assert _append(lib, c, s, **kw) == code, kw


def test_page_errors_needs_somewhere_to_write(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n
    assert lib.mxfp4el_page_errors(None, None) == n.ERR_INVALID_ARGUMENT


def test_scale_is_positive(lib):
    from mxfp4_routed_expert_route_gb300 import _native as n
    for scale in (0.0, -0.125):
        assert _prefill(lib, _cache(n), _seqs(n), scale=scale) == n.ERR_INVALID_ARGUMENT

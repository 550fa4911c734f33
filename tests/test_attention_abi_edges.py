"""Sizes and addresses at the edge of what the attention operators' C entry
points accept: everything here returns before any GPU work."""
from test_attention_abi import _append, _cache, _prefill, _seqs, lib  # noqa: F401


def test_strides_past_the_address_space(lib):  # noqa: F811
    from mxfp4_routed_expert_route_gb300 import _native as n
    big, s = n.ERR_TOO_LARGE, _seqs(n)
    # Rows times stride past 64 bits: the span was taken for a short one.
    for kw in (dict(T=1 << 30, qt=1 << 34), dict(T=1 << 30, qt=1 << 39), dict(heads=8, qh=1 << 39),
               dict(T=9, qt=1 << 62)):
        assert _prefill(lib, _cache(n), s, **kw) == big, kw
        assert _append(lib, _cache(n), s, **kw) == big, kw
    assert _append(lib, _cache(n), s, T=1 << 30, kt=1 << 34) == big
    for kw in (dict(num_pages=(1 << 31) - 1, k_page_stride=1 << 38), dict(v_slot_stride=1 << 60),
               dict(k_head_stride=1 << 39)):
        assert _prefill(lib, _cache(n, **kw), s) == big, kw
        assert _append(lib, _cache(n, **kw), s) == big, kw
    # A tensor map takes byte strides below 2^40, whatever the type.
    f32 = dict(dtype=n.DTYPE_F32, k_page_stride=1 << 38)
    assert _prefill(lib, _cache(n, **f32), s) == big


def test_addresses_between_elements(lib):  # noqa: F811
    from mxfp4_routed_expert_route_gb300 import _native as n
    bad, c = n.ERR_INVALID_ARGUMENT, _cache(n)
    for kw in (dict(page_table=(1 << 24) + 2), dict(seq_lens=(1 << 25) + 1),
               dict(q_offsets=(1 << 26) + 3)):
        assert _prefill(lib, c, _seqs(n, **kw)) == bad, kw
        assert _append(lib, c, _seqs(n, **kw)) == bad, kw
    assert _prefill(lib, c, _seqs(n), logits=(1 << 39) + 2) == bad

"""The attention half of a decoder layer: appending keys and values to a
paged cache (with head norms and the position rotation on the way), attention
of single new tokens, and attention of prompts.

Like the rest of the package this is the thin Python face of the C library
(header ``include/mxfp4el_attention.h``): it checks and marshals arguments;
the work is done by the library's CUDA kernels on the current stream.

A program keeps two handles: a :class:`PagedKVCache` for each layer's cache
and a :class:`PagedSequences` for the sequences of a step. Both hold tensors
that the program fills and updates in place; neither copies anything.
"""
from __future__ import annotations

import ctypes

import torch

from . import _native

__all__ = ["PagedKVCache", "PagedSequences", "append_kv", "paged_attention_decode",
           "paged_attention_prefill", "attention_workspace", "page_errors"]

_DTYPES = {torch.float32: _native.DTYPE_F32, torch.bfloat16: _native.DTYPE_BF16}


# The current stream's handle of a device by index: the tuple-free form of
# torch.cuda.current_stream(device).cuda_stream, which costs 2 us a call.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice
_capturing = torch._C._cuda_isCurrentStreamCapturing


class PagedKVCache:
    """A paged cache of keys and values.

    ``k_pages`` and ``v_pages`` are (num_pages, num_kv_heads, page_size,
    head_dim) CUDA tensors, float32 or bfloat16, with contiguous rows of
    head_dim (64 or 128) elements and strides of 16-byte multiples, so a
    transposed view of a (num_pages, page_size, num_kv_heads, head_dim) tensor
    fits too. page_size is a power of two from 8 to 1024.
    """

    def __init__(self, k_pages: torch.Tensor, v_pages: torch.Tensor):
        if not k_pages.is_cuda or v_pages.device != k_pages.device:
            raise ValueError("k_pages and v_pages must be on one CUDA device")
        if k_pages.dtype not in _DTYPES or v_pages.dtype != k_pages.dtype:
            raise TypeError("k_pages and v_pages must share a supported dtype")
        if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
            raise ValueError("expected k_pages and v_pages of one shape "
                             "(num_pages, num_kv_heads, page_size, head_dim)")
        if k_pages.stride(3) != 1 or v_pages.stride(3) != 1:
            raise ValueError("the rows of k_pages and v_pages must be contiguous")
        pages, heads, page, dim = k_pages.shape
        if dim not in (64, 128):
            raise ValueError("head_dim must be 64 or 128")
        if not 8 <= page <= 1024 or page & (page - 1):
            raise ValueError("page_size must be a power of two from 8 to 1024")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.device, self.dtype = k_pages.device, k_pages.dtype
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self._c = _native.KvCache(
            k_pages.data_ptr(), v_pages.data_ptr(), pages, heads, page, dim,
            *k_pages.stride()[:3], *v_pages.stride()[:3], _DTYPES[k_pages.dtype])
        self._address = ctypes.addressof(self._c)
        self._index = k_pages.device.index

    @classmethod
    def empty(cls, num_pages: int, num_kv_heads: int, page_size: int, head_dim: int,
              dtype: torch.dtype = torch.bfloat16, device="cuda") -> "PagedKVCache":
        """A cache of uninitialised pages."""
        shape = (num_pages, num_kv_heads, page_size, head_dim)
        return cls(torch.empty(shape, dtype=dtype, device=device),
                   torch.empty(shape, dtype=dtype, device=device))


class PagedSequences:
    """The sequences of a step.

    ``page_table`` (num_seqs, max_pages) int32 holds each sequence's pages in
    order, ``seq_lens`` (num_seqs) int32 its tokens, new ones included, and
    ``q_offsets`` (num_seqs + 1) int32 the rows of its new tokens (rows
    q_offsets[b] to q_offsets[b + 1] - 1); None means one new token per
    sequence. All on one CUDA device.
    """

    def __init__(self, page_table: torch.Tensor, seq_lens: torch.Tensor,
                 q_offsets: torch.Tensor | None = None):
        if not page_table.is_cuda:
            raise ValueError("page_table must be a CUDA tensor")
        for name, t, dim in (("page_table", page_table, 2), ("seq_lens", seq_lens, 1),
                             ("q_offsets", q_offsets, 1)):
            if t is None:
                continue
            if t.device != page_table.device:
                raise ValueError(f"{name} is on {t.device}, page_table on {page_table.device}")
            if t.dtype != torch.int32:
                raise TypeError(f"{name} must be int32")
            if t.dim() != dim or (t.shape[-1] > 1 and t.stride(-1) != 1):
                raise ValueError(f"{name} must have {dim} dimension(s) and contiguous rows")
        n = page_table.shape[0]
        if seq_lens.shape[0] != n or (q_offsets is not None and q_offsets.shape[0] != n + 1):
            raise ValueError("page_table, seq_lens and q_offsets do not match")
        self.page_table, self.seq_lens, self.q_offsets = page_table, seq_lens, q_offsets
        self.device, self.num_seqs = page_table.device, n
        self._index = page_table.device.index
        self._c = _native.Sequences(
            page_table.data_ptr(), seq_lens.data_ptr(),
            q_offsets.data_ptr() if q_offsets is not None else None,
            n, page_table.shape[1], page_table.stride(0))
        self._address = ctypes.addressof(self._c)


# The calls below are short next to what Python spends on them, so their
# checks are written out in one place each, and what they refuse is worked out
# only then.
def _refuse_rows(name: str, t: torch.Tensor, cache: PagedKVCache, heads: int | None = None):
    if t.dtype != cache.dtype:
        raise TypeError(f"{name} must have the cache's dtype {cache.dtype}")
    if t.device != cache.device:
        raise ValueError(f"{name} is on {t.device}, the cache on {cache.device}")
    if t.dim() != 3 or t.shape[2] != cache.head_dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be (tokens, heads, {cache.head_dim})")
    raise ValueError(f"the rows of {name} must be contiguous")


def _check_out(name: str, out: torch.Tensor, q: torch.Tensor) -> None:
    if out.shape != q.shape or out.dtype != q.dtype or out.device != q.device \
            or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of q's shape, dtype and device")


def _call(f, name: str, cache: PagedKVCache, args: tuple) -> None:
    """One library call on the cache's device, the current stream last."""
    index = cache._index
    if _current_device() == index:
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = f(*args, _raw_stream(index))
    if rc:
        _native.check(rc, name)


def append_kv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cache: PagedKVCache,
              seqs: PagedSequences, *, cos_sin: torch.Tensor | None = None,
              interleaved: bool = False, q_norm: torch.Tensor | None = None,
              k_norm: torch.Tensor | None = None, eps: float = 1e-6,
              q_out: torch.Tensor | None = None) -> torch.Tensor:
    """Norm and turn the new tokens' queries and keys, write keys and values
    to the cache, and return the queries, (tokens, num_heads, head_dim).

    q is (tokens, num_heads, head_dim), k and v (tokens, num_kv_heads,
    head_dim) in the cache's dtype, strided views allowed. ``cos_sin``
    (max_positions, rotary_dim) float32 holds each position's cosines, then
    its sines; None leaves the rows unturned. ``q_norm`` and ``k_norm``
    (head_dim) in the cache's dtype weigh an RMS norm of each head's row.
    See mxfp4el_append_kv in the C header.
    """
    dtype, index, dim, kv_heads = cache.dtype, cache._index, cache.head_dim, cache.num_kv_heads
    qs, ks, vs = q.stride(), k.stride(), v.stride()
    shape, kshape = q.shape, k.shape
    if q.dtype is not dtype or q.get_device() != index or len(shape) != 3 or shape[2] != dim \
            or qs[2] != 1:
        _refuse_rows("q", q, cache)
    if k.dtype is not dtype or k.get_device() != index or len(kshape) != 3 \
            or kshape[1] != kv_heads or kshape[2] != dim or ks[2] != 1:
        _refuse_rows("k", k, cache, kv_heads)
    T = shape[0]
    if kshape[0] != T or v.shape[0] != T:
        raise ValueError("q, k and v must have the same number of tokens")
    if v.dtype is not dtype or v.get_device() != index or v.shape != kshape or vs[2] != 1:
        _refuse_rows("v", v, cache, kv_heads)
    if seqs._index != index:
        raise ValueError(f"the sequences are on {seqs.device}, the cache on {cache.device}")
    if seqs.q_offsets is None and seqs.num_seqs != T:
        raise ValueError("without q_offsets there is one token per sequence")
    for w in (q_norm, k_norm):
        if w is not None and (w.dtype is not dtype or w.get_device() != index
                              or w.shape != (dim,) or not w.is_contiguous()):
            raise ValueError(f"q_norm and k_norm must be ({dim},) in the cache's dtype, on its device")
    positions = rotary = 0
    if cos_sin is not None:
        if cos_sin.dtype is not torch.float32 or cos_sin.get_device() != index \
                or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin must be a contiguous (max_positions, rotary_dim) float32 "
                             "tensor on the cache's device")
        positions, rotary = cos_sin.shape
        if rotary % 16 or not 0 < rotary <= dim:
            raise ValueError("rotary_dim must be a multiple of 16 up to head_dim")
    if q_out is not None:
        _check_out("q_out", q_out, q)
    else:
        q_out = torch.empty(shape, dtype=dtype, device=cache.device)
    if T:
        _call(_native.load().mxfp4el_append_kv, "append_kv", cache, (
            q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
            None if q_norm is None else q_norm.data_ptr(),
            None if k_norm is None else k_norm.data_ptr(), eps,
            None if cos_sin is None else cos_sin.data_ptr(), positions, rotary,
            1 if interleaved else 0, cache._address, seqs._address, q_out.data_ptr(), T, shape[1]))
    return q_out


def attention_workspace(device=None) -> torch.Tensor:
    """A zeroed workspace for the attention calls, to be kept and passed as
    ``workspace``. Calls that may run at the same time (on different streams,
    or in different graphs) need one each. After :func:`wait_timeouts` has
    reported a wait that gave up, it has to be zeroed."""
    dev = torch.device("cuda" if device is None else device)
    return torch.zeros(_native.load().mxfp4el_attention_workspace_size(), dtype=torch.uint8,
                       device=dev)


# The workspace of calls that bring none: one per device and stream, so that
# calls on different streams do not share one.
_workspaces: dict[tuple[int, int], torch.Tensor] = {}


def _drop_workspaces(index: int) -> None:
    """A call that gave up may leave a workspace's counters as they should not
    be: the next calls on the device get new ones."""
    for key in [k for k in _workspaces if k[0] == index]:
        del _workspaces[key]


def _kept_workspace(cache: PagedKVCache) -> torch.Tensor:
    index = cache._index
    if _current_device() != index:
        with torch.cuda.device(index):
            return _kept_workspace(cache)
    # A graph may run on any stream, beside the calls of this one.
    if _capturing():
        raise RuntimeError("pass a workspace of its own (attention_workspace) to a call that "
                           "is captured in a graph")
    key = (index, _raw_stream(index))
    ws = _workspaces.get(key)
    if ws is None:
        ws = _workspaces[key] = attention_workspace(cache.device)
    return ws


def _attention(decode, q, cache, seqs, scale, window, sinks, sink_logits, out, workspace):
    shape, stride, index = q.shape, q.stride(), cache._index
    if q.dtype is not cache.dtype or q.get_device() != index or len(shape) != 3 \
            or shape[2] != cache.head_dim or stride[2] != 1:
        _refuse_rows("q", q, cache)
    T, heads, dim = shape
    if heads == 0 or heads % cache.num_kv_heads:
        raise ValueError("the number of query heads must be a multiple of the cache's heads")
    if seqs._index != index:
        raise ValueError(f"the sequences are on {seqs.device}, the cache on {cache.device}")
    if seqs.q_offsets is None and seqs.num_seqs != T:
        raise ValueError("without q_offsets there is one token per sequence")
    window = 0 if window is None else window
    if window < 0 or sinks < 0:
        raise ValueError("window and sinks must not be negative")
    if sink_logits is not None and (
            sink_logits.dtype is not torch.float32 or sink_logits.get_device() != index
            or sink_logits.shape != (heads,) or not sink_logits.is_contiguous()):
        raise ValueError("sink_logits must be a (heads,) float32 tensor on the cache's device")
    if out is not None:
        _check_out("out", out, q)
    elif stride[1] == dim and stride[0] == heads * dim:
        out = torch.empty_like(q)
    else:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
    if T:
        if workspace is None:
            workspace = _kept_workspace(cache)
        elif workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the cache's device")
        args = (q.data_ptr(), stride[0], stride[1], cache._address, seqs._address,
                dim ** -0.5 if scale is None else scale, window, sinks,
                None if sink_logits is None else sink_logits.data_ptr(), out.data_ptr())
        lib = _native.load()
        if decode:
            _call(lib.mxfp4el_attention_decode, "paged_attention_decode", cache,
                  args + (heads, workspace.data_ptr(), workspace.nbytes))
        else:
            _call(lib.mxfp4el_attention_prefill, "paged_attention_prefill", cache,
                  args + (T, heads, workspace.data_ptr(), workspace.nbytes))
    return out


def paged_attention_decode(q: torch.Tensor, cache: PagedKVCache, seqs: PagedSequences, *,
                           scale: float | None = None, window: int | None = None,
                           sinks: int = 0, sink_logits: torch.Tensor | None = None,
                           out: torch.Tensor | None = None,
                           workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of one new token of each sequence over the cache.

    Row b of q (num_seqs, num_heads, head_dim) is the last token of sequence
    b, whose own key and value are already in the cache. ``scale`` defaults to
    head_dim ** -0.5. With a ``window`` w the token sees the last w keys (its
    own among them) and the first ``sinks``. ``sink_logits`` (num_heads)
    float32 adds exp(logit) to each head's softmax sum. A sequence without
    keys gives zeros. ``workspace`` is an :func:`attention_workspace`; by
    default one per stream is kept. A call that is captured in a graph has to
    bring one, since the graph may run beside the stream's other calls. Sums
    are float32; bfloat16 calls round the softmax's weights to bfloat16 where
    they multiply the values. See mxfp4el_attention_decode in the C header.
    """
    if seqs.q_offsets is not None:
        raise ValueError("decode takes one token per sequence: leave q_offsets out, or use "
                         "paged_attention_prefill")
    return _attention(True, q, cache, seqs, scale, window, sinks, sink_logits,
                      out, workspace)


def paged_attention_prefill(q: torch.Tensor, cache: PagedKVCache, seqs: PagedSequences, *,
                            scale: float | None = None, window: int | None = None,
                            sinks: int = 0, sink_logits: torch.Tensor | None = None,
                            out: torch.Tensor | None = None,
                            workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of each sequence's new tokens over the cache, causal.

    q is (tokens, num_heads, head_dim), the sequences' new tokens one after
    another as ``seqs.q_offsets`` says; their keys and values are already in
    the cache, behind any history. Arguments otherwise as
    :func:`paged_attention_decode`.
    """
    return _attention(False, q, cache, seqs, scale, window, sinks,
                      sink_logits, out, workspace)


def page_errors(device=None) -> int:
    """Page ids, lengths and positions out of range that the attention calls
    met since the last query (syncs)."""
    dev = torch.device(device) if device is not None else torch.device(
        "cuda", torch.cuda.current_device())
    n = ctypes.c_int64(0)
    with torch.cuda.device(dev):
        stream = torch.cuda.current_stream(dev).cuda_stream
        _native.check(_native.load().mxfp4el_page_errors(stream, ctypes.byref(n)),
                      "mxfp4el_page_errors")
    return int(n.value)

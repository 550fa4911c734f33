// attn_api.cu -- the C ABI of the attention operators
// (include/mxfp4el_attention.h): argument checks and launches.
#include <cmath>
#include <limits>

#include "../../include/mxfp4_expert_linear.h"
#include "../../include/mxfp4el_attention.h"
#include "attn.h"

namespace mxfp4el {
namespace {

constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxTokens = kMaxKeys;
constexpr int64_t kMaxStrideBytes = ((int64_t)1 << 40) - 1;   // as a tensor map has it
constexpr int64_t kMaxSpanBytes = (int64_t)1 << 56;
constexpr int64_t kMaxHeads = 1 << 15;
constexpr int64_t kMaxGroup = 128;                   // query heads to a key head

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

struct Span {
  uintptr_t lo, hi;   // bytes [lo, hi); empty when equal
};
bool overlaps(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
Span span_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, p == nullptr || bytes <= 0 ? lo : lo + (uintptr_t)bytes};
}

// A (n0, n1, width) array with element strides s0, s1: whether it can be
// read in 16-byte pieces, and the bytes it spans.
int check_rows(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t width,
               int64_t esize, Span* span) {
  if (p == nullptr || !aligned16(p)) return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (s0 < 0 || s1 < 0 || s0 % (16 / esize) != 0 || s1 % (16 / esize) != 0)
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (s0 > kMaxStrideBytes / esize || s1 > kMaxStrideBytes / esize) return MXFP4EL_ERR_TOO_LARGE;
  const __int128 bytes = ((__int128)(n0 - 1) * s0 + (__int128)(n1 - 1) * s1 + width) * esize;
  if (bytes > kMaxSpanBytes) return MXFP4EL_ERR_TOO_LARGE;
  *span = span_of(p, (int64_t)bytes);
  return MXFP4EL_OK;
}

int check_cache(const mxfp4el_kv_cache* c, KvCacheView* v, Span* k_span, Span* v_span) {
  if (c == nullptr) return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (c->dtype != MXFP4EL_DTYPE_F32 && c->dtype != MXFP4EL_DTYPE_BF16)
    return MXFP4EL_ERR_UNSUPPORTED_DTYPE;
  if (c->num_pages <= 0 || c->num_kv_heads <= 0 || (c->head_dim != 64 && c->head_dim != 128) ||
      c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (c->num_pages > kMaxDim || c->num_kv_heads > kMaxHeads) return MXFP4EL_ERR_TOO_LARGE;
  const int64_t es = c->dtype == MXFP4EL_DTYPE_BF16 ? 2 : 4;
  *k_span = *v_span = Span{0, 0};
  const void* base[2] = {c->k, c->v};
  const int64_t st[2][3] = {{c->k_page_stride, c->k_head_stride, c->k_slot_stride},
                            {c->v_page_stride, c->v_head_stride, c->v_slot_stride}};
  for (int i = 0; i < 2; ++i) {
    // Slots of a page must not fall together: the append writes them.
    if (st[i][2] < c->head_dim) return MXFP4EL_ERR_INVALID_ARGUMENT;
    if (st[i][2] % (16 / es) != 0) return MXFP4EL_ERR_INVALID_ARGUMENT;
    if (st[i][2] > kMaxStrideBytes / es) return MXFP4EL_ERR_TOO_LARGE;
    Span* s = i == 0 ? k_span : v_span;
    const int rc = check_rows(base[i], c->num_pages, st[i][0], c->num_kv_heads, st[i][1],
                              (c->page_size - 1) * st[i][2] + c->head_dim, es, s);
    if (rc != MXFP4EL_OK) return rc;
  }
  v->k = c->k;
  v->v = c->v;
  v->num_pages = c->num_pages;
  v->k_page = c->k_page_stride;
  v->k_head = c->k_head_stride;
  v->k_slot = c->k_slot_stride;
  v->v_page = c->v_page_stride;
  v->v_head = c->v_head_stride;
  v->v_slot = c->v_slot_stride;
  v->page_size = (int)c->page_size;
  v->page_shift = 0;
  while ((1 << v->page_shift) < v->page_size) ++v->page_shift;
  v->kv_heads = (int)c->num_kv_heads;
  v->head_dim = (int)c->head_dim;
  v->token_dtype = c->dtype == MXFP4EL_DTYPE_BF16 ? kTokenBF16 : kTokenF32;
  return MXFP4EL_OK;
}

int check_sequences(const mxfp4el_sequences* s, int64_t T, SequencesView* v) {
  if (s == nullptr || s->num_seqs < 0 || s->max_pages < 0) return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (s->num_seqs > kMaxTokens || s->max_pages > kMaxDim) return MXFP4EL_ERR_TOO_LARGE;
  if (s->num_seqs > 0 && (s->seq_lens == nullptr ||
                          (s->max_pages > 0 && (s->page_table == nullptr ||
                                                (s->num_seqs > 1 && s->table_stride < 0)))))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (!aligned4(s->page_table) || !aligned4(s->seq_lens) || !aligned4(s->q_offsets))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (s->q_offsets == nullptr && s->num_seqs != T) return MXFP4EL_ERR_INVALID_ARGUMENT;
  v->page_table = s->page_table;
  v->seq_lens = s->seq_lens;
  v->q_offsets = s->q_offsets;
  v->table_stride = s->table_stride;
  v->num_seqs = (int)s->num_seqs;
  v->max_pages = (int)s->max_pages;
  return MXFP4EL_OK;
}

// Checks of the two attention calls, in the order the header documents.
// *nothing: the call is valid and has no rows.
int check_attention(const void* q, int64_t q_token, int64_t q_head, const mxfp4el_kv_cache* cache,
                    const mxfp4el_sequences* seqs, float scale, int64_t window, int64_t sinks,
                    const float* sink_logits, void* out, int64_t T, int64_t heads,
                    const void* workspace, size_t workspace_bytes, AttnArgs* a, bool* nothing) {
  *nothing = false;
  Span ks, vs, qs;
  int rc = check_cache(cache, &a->cache, &ks, &vs);
  if (rc != MXFP4EL_OK) return rc;
  if (T < 0 || heads <= 0 || heads % a->cache.kv_heads != 0 || window < 0 || sinks < 0 ||
      !(scale > 0.f) || !std::isfinite(scale))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (T > kMaxTokens || heads > kMaxHeads || heads / a->cache.kv_heads > kMaxGroup)
    return MXFP4EL_ERR_TOO_LARGE;
  rc = check_sequences(seqs, T, &a->seqs);
  if (rc != MXFP4EL_OK) return rc;
  // The prefill kernels count (query tile, key head) units in 31 bits, with
  // room for the grid past the last.
  if ((T + seqs->num_seqs + 1) * a->cache.kv_heads > kMaxDim - (1 << 20)) return MXFP4EL_ERR_TOO_LARGE;
  if (T == 0) {
    *nothing = true;
    return MXFP4EL_OK;
  }
  const int64_t es = a->cache.token_dtype == kTokenBF16 ? 2 : 4, D = a->cache.head_dim;
  rc = check_rows(q, T, q_token, heads, q_head, D, es, &qs);
  if (rc != MXFP4EL_OK) return rc;
  if (out == nullptr || !aligned16(out) || !aligned4(sink_logits))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  const Span os = span_of(out, T * heads * D * es);
  const Span others[] = {qs, ks, vs, span_of(sink_logits, heads * 4),
                         span_of(workspace, (int64_t)workspace_bytes),
                         span_of(seqs->seq_lens, seqs->num_seqs * 4),
                         span_of(seqs->q_offsets, (seqs->num_seqs + 1) * 4)};
  for (const Span& s : others)
    if (overlaps(os, s)) return MXFP4EL_ERR_ALIAS;
  if (workspace == nullptr || workspace_bytes < mxfp4el_attention_workspace_size() ||
      reinterpret_cast<uintptr_t>(workspace) % 256 != 0)
    return MXFP4EL_ERR_WORKSPACE;
  a->q = q;
  a->q_token = q_token;
  a->q_head = q_head;
  a->out = out;
  a->sink_logits = sink_logits;
  a->scale = scale;
  a->T = (int)T;
  a->heads = (int)heads;
  a->group = (int)(heads / a->cache.kv_heads);
  // A window that no length reaches is no window; first tokens past every
  // length show no more.
  a->window = window >= kMaxKeys ? 0 : (int)window;
  a->sinks = a->window == 0 ? 0 : (int)(sinks > kMaxKeys ? kMaxKeys : sinks);
  a->status = device_status_words();
  return a->status == nullptr ? MXFP4EL_ERR_CUDA : MXFP4EL_OK;
}

}  // namespace
}  // namespace mxfp4el

using namespace mxfp4el;

extern "C" int mxfp4el_append_kv(const void* q, int64_t q_token_stride, int64_t q_head_stride,
                                 const void* k, int64_t k_token_stride, int64_t k_head_stride,
                                 const void* v, int64_t v_token_stride, int64_t v_head_stride,
                                 const void* q_norm, const void* k_norm, float eps,
                                 const float* cos_sin, int64_t max_positions, int64_t rotary_dim,
                                 int interleaved, const mxfp4el_kv_cache* cache,
                                 const mxfp4el_sequences* seqs, void* q_out, int64_t T,
                                 int64_t num_heads, void* stream) {
  AppendArgs a = {};
  Span ks, vs, in[3];
  int rc = check_cache(cache, &a.cache, &ks, &vs);
  if (rc != MXFP4EL_OK) return rc;
  if (T < 0 || num_heads <= 0 || rotary_dim < 0 || rotary_dim > a.cache.head_dim ||
      rotary_dim % 16 != 0 || max_positions < 0 || !(eps >= 0.f))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (T > kMaxTokens || num_heads > kMaxHeads) return MXFP4EL_ERR_TOO_LARGE;
  rc = check_sequences(seqs, T, &a.seqs);
  if (rc != MXFP4EL_OK) return rc;
  if (T == 0) return MXFP4EL_OK;
  const int64_t es = a.cache.token_dtype == kTokenBF16 ? 2 : 4, D = a.cache.head_dim;
  const int64_t hk = a.cache.kv_heads;
  if ((rc = check_rows(q, T, q_token_stride, num_heads, q_head_stride, D, es, &in[0])) ||
      (rc = check_rows(k, T, k_token_stride, hk, k_head_stride, D, es, &in[1])) ||
      (rc = check_rows(v, T, v_token_stride, hk, v_head_stride, D, es, &in[2])))
    return rc;
  if (q_out == nullptr || !aligned16(q_out) || !aligned16(q_norm) || !aligned16(k_norm) ||
      (rotary_dim > 0 && (cos_sin == nullptr || !aligned16(cos_sin))))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  const Span table = span_of(cos_sin, rotary_dim > 0 ? max_positions * rotary_dim * 4 : 0);
  const Span outs[] = {span_of(q_out, T * num_heads * D * es), ks, vs};
  const Span ins[] = {in[0], in[1], in[2], table, span_of(q_norm, D * es), span_of(k_norm, D * es),
                      span_of(seqs->seq_lens, seqs->num_seqs * 4),
                      span_of(seqs->q_offsets, (seqs->num_seqs + 1) * 4)};
  for (const Span& o : outs)
    for (const Span& i : ins)
      if (overlaps(o, i)) return MXFP4EL_ERR_ALIAS;
  if (overlaps(outs[0], ks) || overlaps(outs[0], vs)) return MXFP4EL_ERR_ALIAS;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_token = q_token_stride;
  a.q_head = q_head_stride;
  a.k_token = k_token_stride;
  a.k_head = k_head_stride;
  a.v_token = v_token_stride;
  a.v_head = v_head_stride;
  a.q_norm = q_norm;
  a.k_norm = k_norm;
  a.cos_sin = cos_sin;
  a.max_positions = max_positions;
  a.eps = eps;
  a.rotary_dim = (int)rotary_dim;
  a.T = (int)T;
  a.heads = (int)num_heads;
  a.q_out = q_out;
  a.status = device_status_words();
  if (a.status == nullptr) return MXFP4EL_ERR_CUDA;
  return launch_append_kv(a, interleaved != 0, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MXFP4EL_OK
             : MXFP4EL_ERR_CUDA;
}

extern "C" size_t mxfp4el_attention_workspace_size(void) { return kAttentionWorkspaceBytes; }

extern "C" int mxfp4el_attention_decode(const void* q, int64_t q_token_stride,
                                        int64_t q_head_stride, const mxfp4el_kv_cache* cache,
                                        const mxfp4el_sequences* seqs, float scale,
                                        int64_t window, int64_t sinks, const float* sink_logits,
                                        void* out, int64_t num_heads, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  if (seqs == nullptr || seqs->q_offsets != nullptr) return MXFP4EL_ERR_INVALID_ARGUMENT;
  AttnArgs a = {};
  bool nothing;
  const int rc = check_attention(q, q_token_stride, q_head_stride, cache, seqs, scale, window,
                                 sinks, sink_logits, out, seqs->num_seqs, num_heads, workspace,
                                 workspace_bytes, &a, &nothing);
  if (rc != MXFP4EL_OK || nothing) return rc;
  return launch_attention_decode(a, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MXFP4EL_OK
             : MXFP4EL_ERR_CUDA;
}

extern "C" int mxfp4el_attention_prefill(const void* q, int64_t q_token_stride,
                                         int64_t q_head_stride, const mxfp4el_kv_cache* cache,
                                         const mxfp4el_sequences* seqs, float scale,
                                         int64_t window, int64_t sinks, const float* sink_logits,
                                         void* out, int64_t T, int64_t num_heads, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  AttnArgs a = {};
  bool nothing;
  const int rc =
      check_attention(q, q_token_stride, q_head_stride, cache, seqs, scale, window, sinks,
                      sink_logits, out, T, num_heads, workspace, workspace_bytes, &a, &nothing);
  if (rc != MXFP4EL_OK || nothing) return rc;
  // The tensor cores take no float32 operands.
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t err = a.cache.token_dtype == kTokenBF16
                              ? launch_attention_prefill(a, workspace, s)
                              : launch_attention_simt(a, workspace, s);
  return err == cudaSuccess ? MXFP4EL_OK : MXFP4EL_ERR_CUDA;
}

extern "C" int mxfp4el_page_errors(void* stream, int64_t* count) {
  if (count == nullptr) return MXFP4EL_ERR_INVALID_ARGUMENT;
  return read_and_reset_status(static_cast<cudaStream_t>(stream), kStatusBadPages, count) ==
                 cudaSuccess
             ? MXFP4EL_OK
             : MXFP4EL_ERR_CUDA;
}

// attn.h -- declarations shared by the attention operators' translation
// units (include/mxfp4el_attention.h).
#pragma once

#include <cuda.h>

#include "internal.h"

namespace mxfp4el {

// Lengths, windows and first tokens are cut to this many keys (no cache holds
// as many), and a call has no more tokens than that, so that positions (-2^30
// at least), their differences and sums with tile sizes stay in 32 bits.
constexpr int kMaxKeys = 1 << 30;

// Keys and values of one sequence are found through its page table; strides
// are in elements.
struct KvCacheView {
  void* k;
  void* v;
  int64_t num_pages;
  int64_t k_page, k_head, k_slot;
  int64_t v_page, v_head, v_slot;
  int page_size, page_shift;
  int kv_heads, head_dim;
  int token_dtype;
};

struct SequencesView {
  const int* page_table;
  const int* seq_lens;
  const int* q_offsets;      // null: one new token per sequence
  int64_t table_stride;
  int num_seqs;
  int max_pages;
};

struct AppendArgs {
  const void *q, *k, *v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  const void *q_norm, *k_norm;
  const float* cos_sin;
  int64_t max_positions;
  float eps;
  int rotary_dim;
  int T, heads;
  void* q_out;
  KvCacheView cache;
  SequencesView seqs;
  unsigned long long* status;
};
cudaError_t launch_append_kv(const AppendArgs& a, bool interleaved, cudaStream_t stream);

struct AttnArgs {
  const void* q;
  int64_t q_token, q_head;
  void* out;                 // (T, heads, head_dim), dense
  const float* sink_logits;  // (heads) or null
  float scale;
  int T, heads, group;       // group: query heads per key head
  int window;                // 0: none
  int sinks;                 // 0 without a window
  KvCacheView cache;
  SequencesView seqs;
  unsigned long long* status;
};

// One new token of each sequence, split over the cache's length and joined
// through the workspace (attn_decode.cu).
cudaError_t launch_attention_decode(const AttnArgs& a, void* workspace, cudaStream_t stream);

// The workspace of an attention call: the decode kernel's counters, the
// prefill kernels' (all zero between calls), and the pieces of split work.
constexpr int kDecodeCounters = 256, kPrefillCounters = 768;
constexpr size_t kPiecesBytes = (size_t)36 << 20;
inline unsigned int* decode_counters(void* ws) { return static_cast<unsigned int*>(ws); }
inline unsigned int* prefill_counters(void* ws) { return decode_counters(ws) + kDecodeCounters; }
inline void* workspace_pieces(void* ws) { return prefill_counters(ws) + kPrefillCounters; }
constexpr size_t kAttentionWorkspaceBytes = (kDecodeCounters + kPrefillCounters) * 4 + kPiecesBytes;

// bf16 prompts on the tensor cores (attn_prefill.cu).
cudaError_t launch_attention_prefill(const AttnArgs& a, void* workspace, cudaStream_t stream);

bool kv_tensor_map(const KvCacheView& c, bool values, int box_rows, int box_subs,
                   CUtensorMap* map);
int attention_num_sms();

// float32 prompts, on the CUDA cores (attn_simt.cu).
cudaError_t launch_attention_simt(const AttnArgs& a, void* workspace, cudaStream_t stream);

}  // namespace mxfp4el

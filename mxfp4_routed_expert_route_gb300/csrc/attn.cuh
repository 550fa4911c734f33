// attn.cuh -- device helpers shared by the attention operators: the rows of
// a sequence, its page table, and the mask.
#pragma once

#include "attn.h"
#include "common.cuh"

namespace mxfp4el {

// The new tokens of one sequence and its keys.
struct SeqRows {
  int first;    // row of the first new token
  int count;    // new tokens
  int len;      // keys, the new tokens' own included
  int pos0;     // position of the first new token (negative rows see nothing)
};

// The last i in [0, count) where holds(i), for a property that holds on a
// prefix that includes 0. A whole warp searches, 32 probes at a time; every
// lane gets the result.
template <typename F>
__device__ __forceinline__ int warp_last(int count, int lane, F holds) {
  int lo = 0, hi = count;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned m = __ballot_sync(kFullMask, i < hi && holds(i)) | 1u;
    const int last = m == kFullMask ? 31 : __ffs(~m) - 2;
    hi = min(hi, lo + (last + 1) * step);
    lo += last * step;
  }
  return lo;
}

// The first row of sequence b (b == num_seqs: of the rows past the last).
__device__ __forceinline__ int first_row(const SequencesView& s, int b, int T) {
  return s.q_offsets == nullptr ? min(b, T) : min(max(__ldg(s.q_offsets + b), 0), T);
}

// Keys that a row of the page table has room for, up to kMaxKeys.
__device__ __forceinline__ int table_room(const SequencesView& s, int page_shift) {
  return (int)min((int64_t)s.max_pages << page_shift, (int64_t)kMaxKeys);
}

// Sequence b of the call; b == num_seqs stands for the rows past the last
// sequence, which have no keys. Offsets are cut to [0, T].
__device__ __forceinline__ SeqRows sequence_rows(const SequencesView& s, int b, int T,
                                                 int page_shift, unsigned long long* status,
                                                 bool count_errors) {
  SeqRows r;
  const bool past = b >= s.num_seqs;
  r.first = first_row(s, b, T);
  r.count = max((past ? T : first_row(s, b + 1, T)) - r.first, 0);
  r.len = past ? 0 : max(__ldg(s.seq_lens + b), 0);
  const int room = table_room(s, page_shift);
  if (r.len > room) {
    r.len = room;
    if (count_errors) atomicAdd(&status[kStatusBadPages], 1ull);
  }
  r.pos0 = r.len - r.count;
  return r;
}

// Query tiles without a prefix sum over the sequences: with n tokens to a
// tile, sequence b owns the tile slots floor(q_offsets[b] / n) + b up to the
// next sequence's first, always enough for its ceil(count / n) tiles (x, y >=
// 0: floor(y) - floor(x) + 1 >= ceil(y - x)); the spare ones are empty. The
// slots of T tokens number floor(T / n) + num_seqs + 1.
inline int64_t query_tile_slots(const SequencesView& s, int T, int n) {
  return s.q_offsets == nullptr ? (int64_t)s.num_seqs : (int64_t)T / n + s.num_seqs + 1;
}

// The sequence (0 .. num_seqs) that owns query tile slot `slot` (n tokens to
// a tile). One row per sequence without offsets: slot b is sequence b.
__device__ __forceinline__ int sequence_of_slot(const SequencesView& s, int slot, int T, int n,
                                                int lane) {
  if (s.q_offsets == nullptr) return min(slot, s.num_seqs);
  return warp_last(s.num_seqs + 1, lane,
                   [&](int b) { return first_row(s, b, T) / n + b <= slot; });
}

// Page of key j, or -1 where the table's id is out of range.
__device__ __forceinline__ int64_t page_of(const SequencesView& s, const KvCacheView& c, int b,
                                           int page_index) {
  const int id = __ldg(s.page_table + (int64_t)b * s.table_stride + page_index);
  return (unsigned)id < (uint64_t)c.num_pages ? (int64_t)id : (int64_t)-1;
}

// Whether the query at position a sees key j (j < len is the caller's).
__device__ __forceinline__ bool key_visible(int j, int a, int window, int sinks) {
  return j <= a && (window == 0 || a - j < window || j < sinks);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace mxfp4el

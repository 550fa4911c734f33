// kv_append.cu -- norms of the query and key heads, position rotation, and
// the write of the new keys and values into the paged cache.
//
// Per token: every query and key row of head_dim elements is divided by its
// root mean square and weighted (when a norm is given), its first rotary_dim
// elements are turned in pairs by the token's angle, and the row is rounded
// once to the token dtype. Queries go to a dense array, keys and (unchanged)
// values to the token's slot of the cache.
//
// Bound: bytes. (heads + 2 kv_heads) head_dim elements are read and as many
// written; the rotation table adds rotary_dim floats per token. 8192 tokens, 64
// query and 8 key heads of 128, normed and turned: 58.5 us, 5.8 TB/s. A handful
// of tokens: 2.3 us, a launch.
//
// Layout: a row's lanes hold two chunks of 8 elements each (chunk j of the
// first half of the turned elements and its partner in the second half, so
// both rotation styles pair elements inside one thread; the chunks past
// rotary_dim pair up among themselves). head_dim / 16 lanes make a row, so a
// warp takes 32 / (head_dim / 16) rows at a time, of one token: the cosines
// and sines of the token stay in the lanes' registers for all of its rows.
// Queries, keys and values are separate runs of steps, so that each step's
// addresses are sums and its arithmetic (two float32 at a time) has no cases:
// 41,900 instructions per scheduler and 58.5 us; with the cases inside one loop
// 63,800 and 65; one step per warp, each looking its token up anew, 92 us.
#include <algorithm>

#include "attn.cuh"

namespace mxfp4el {
namespace {

constexpr int kAppendWarps = 4;
constexpr int kFlight = 4;
constexpr int kAppendBlocks = 4;        // per SM
constexpr int kFillWarps = 152 * 32;

template <typename Tok> struct Chunk8;   // 8 elements <-> 4 pairs of floats, 16-byte accesses

template <> struct Chunk8<__nv_bfloat16> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void unpack(float2 (&x)[4]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void pack(const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    raw = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = raw; }
};

template <> struct Chunk8<float> {
  uint4 raw[2];
  __device__ __forceinline__ void load(const float* p) {
    raw[0] = __ldg(reinterpret_cast<const uint4*>(p));
    raw[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void unpack(float2 (&x)[4]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] = make_float2(__uint_as_float(raw[i].x), __uint_as_float(raw[i].y));
      x[2 * i + 1] = make_float2(__uint_as_float(raw[i].z), __uint_as_float(raw[i].w));
    }
  }
  __device__ __forceinline__ void pack(const float2 (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      raw[i] = make_uint4(__float_as_uint(x[2 * i].x), __float_as_uint(x[2 * i].y),
                          __float_as_uint(x[2 * i + 1].x), __float_as_uint(x[2 * i + 1].y));
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = raw[0];
    reinterpret_cast<uint4*>(p)[1] = raw[1];
  }
};

// The pair (x, y) of chunks turned in place, two elements at a time. Half
// style: element i of x with element i of y by (c[i], s[i]). Interleaved:
// elements 2i and 2i + 1 of x by (c[i], s[i]), of y by (c[4 + i], s[4 + i]).
template <bool kInter>
__device__ __forceinline__ void turn(float2 (&x)[4], float2 (&y)[4], const float2 (&c)[4],
                                     const float2 (&s)[4]) {
  if constexpr (kInter) {
    auto one = [](float2& v, float ci, float si) {
      v = ffma2(v, make_float2(ci, ci),
                fmul2(make_float2(v.y, v.x), make_float2(-si, si)));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      one(x[2 * i], c[i].x, s[i].x);
      one(x[2 * i + 1], c[i].y, s[i].y);
      one(y[2 * i], c[2 + i].x, s[2 + i].x);
      one(y[2 * i + 1], c[2 + i].y, s[2 + i].y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = x[i], b = y[i];
      x[i] = ffma2(a, c[i], fmul2(b, make_float2(-s[i].x, -s[i].y)));
      y[i] = ffma2(b, c[i], fmul2(a, s[i]));
    }
  }
}

// What a warp knows about its token.
struct TokenPlace {
  int64_t page;
  int slot;
  bool rotate;   // its position has a row of angles (or there are none)
  bool store;    // its key and value have a place
};

// The warp's steps of one kind of rows: kRows rows at a time, kInFlight steps'
// loads issued together. src and dst are the token's rows. Returns the step at
// which the warp goes on with the next kind.
enum class Rows { kQuery, kKey, kValue };
template <Rows kKind, typename Tok, int D, bool kInter>
__device__ __forceinline__ int rows_of_kind(const Tok* src, int64_t src_head, Tok* dst,
                                            int64_t dst_head, const Tok* norm, float eps, int rows,
                                            int step, int slices, int c0, int c1, bool turns,
                                            const float2 (&cs)[4], const float2 (&sn)[4],
                                            const TokenPlace& place, int lane) {
  constexpr int kLanes = D / 16, kRows = 32 / kLanes;
  constexpr int kInFlight = sizeof(Tok) == 2 ? kFlight : kFlight / 2;
  const int steps = (rows + kRows - 1) / kRows;
  float2 n0[4], n1[4];
  if (kKind != Rows::kValue && norm != nullptr && step < steps) {
    Chunk8<Tok> a, b;
    a.load(norm + 8 * c0);
    b.load(norm + 8 * c1);
    a.unpack(n0);
    b.unpack(n1);
  }
  src += (int64_t)min(step * kRows + lane / kLanes, rows - 1) * src_head;
  for (; step < steps; step += slices * kInFlight) {
    Chunk8<Tok> u[kInFlight], w[kInFlight];
    const int h0 = step * kRows + lane / kLanes;
    const Tok* from = src;
#pragma unroll
    for (int f = 0; f < kInFlight; ++f) {
      if (h0 + f * slices * kRows < rows) {
        u[f].load(from + 8 * c0);
        w[f].load(from + 8 * c1);
      }
      from += (int64_t)slices * kRows * src_head;
    }
    src = from;
#pragma unroll
    for (int f = 0; f < kInFlight; ++f) {
      if (f > 0 && step + f * slices >= steps) return step + f * slices - steps;
      const int h = h0 + f * slices * kRows;
      if constexpr (kKind != Rows::kValue) {
        float2 x[4], y[4];
        u[f].unpack(x);
        w[f].unpack(y);
        if (norm != nullptr) {
          // The row's mean square over its lanes (all lanes of the warp take
          // part in the shuffles).
          float2 sq = fmul2(x[0], x[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) sq = ffma2(x[i], x[i], sq);
#pragma unroll
          for (int i = 0; i < 4; ++i) sq = ffma2(y[i], y[i], sq);
          float sum = sq.x + sq.y;
#pragma unroll
          for (int o = kLanes / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
          const float inv = rsqrtf(sum * (1.0f / D) + eps);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[i] = fmul2(fmul2(x[i], make_float2(inv, inv)), n0[i]);
            y[i] = fmul2(fmul2(y[i], make_float2(inv, inv)), n1[i]);
          }
        }
        if (turns && place.rotate) turn<kInter>(x, y, cs, sn);
        if (kKind == Rows::kQuery && !place.rotate) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = y[i] = make_float2(0.f, 0.f);
        }
        u[f].pack(x);
        w[f].pack(y);
      }
      if (h < rows && (kKind == Rows::kQuery || place.store)) {
        u[f].store(dst + h * dst_head + 8 * c0);
        w[f].store(dst + h * dst_head + 8 * c1);
      }
    }
  }
  return step - steps;
}

template <typename Tok, int D, bool kInter>
__global__ void __launch_bounds__(kAppendWarps * 32, kAppendBlocks)
append_kv_kernel(const AppendArgs a, int slices) {
  constexpr int kLanes = D / 16;          // lanes of a row
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int t = (int)(unit / slices), slice = (int)(unit - (int64_t)t * slices);
  if (t >= a.T) return;

  // The token's sequence and position (the same in every lane).
  const int seq = a.seqs.q_offsets == nullptr
                      ? min(t, a.seqs.num_seqs)
                      : warp_last(a.seqs.num_seqs + 1, lane,
                                  [&](int b) { return first_row(a.seqs, b, a.T) <= t; });
  const bool past = seq >= a.seqs.num_seqs;
  int pos = -1;
  if (!past)
    pos = __ldg(a.seqs.seq_lens + seq) - first_row(a.seqs, seq + 1, a.T) + t;
  const bool pos_ok = pos >= 0 && (pos >> a.cache.page_shift) < a.seqs.max_pages;
  TokenPlace place;
  place.rotate = !past && (a.rotary_dim == 0 || (pos_ok && pos < a.max_positions));
  place.page = -1;
  if (pos_ok) place.page = page_of(a.seqs, a.cache, seq, pos >> a.cache.page_shift);
  place.store = place.rotate && place.page >= 0;
  place.slot = pos & (a.cache.page_size - 1);
  if (!past && !place.store && slice == 0 && lane == 0)
    atomicAdd(&a.status[kStatusBadPages], 1ull);

  // This lane's two chunks, and the cosines and sines of its pairs.
  const int j = lane % kLanes, rot = a.rotary_dim / 16;      // chunk pairs that turn
  const bool turns = j < rot;
  int c0, c1;
  if (kInter) {
    c0 = 2 * j;
    c1 = 2 * j + 1;
  } else {
    c0 = turns ? j : 2 * rot + 2 * (j - rot);
    c1 = turns ? j + rot : c0 + 1;
  }
  float2 cs[4] = {}, sn[4] = {};
  if (turns && place.rotate) {
    const float4* row = reinterpret_cast<const float4*>(a.cos_sin + (int64_t)pos * a.rotary_dim) + 2 * j;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = __ldg(row + i), s = __ldg(row + a.rotary_dim / 8 + i);
      cs[2 * i] = make_float2(c.x, c.y);
      cs[2 * i + 1] = make_float2(c.z, c.w);
      sn[2 * i] = make_float2(s.x, s.y);
      sn[2 * i + 1] = make_float2(s.z, s.w);
    }
  }

  // The token's steps are its query rows', then its keys', then its values'.
  const KvCacheView& kv = a.cache;
  int step = rows_of_kind<Rows::kQuery, Tok, D, kInter>(
      static_cast<const Tok*>(a.q) + t * a.q_token, a.q_head,
      static_cast<Tok*>(a.q_out) + (int64_t)t * a.heads * D, D, static_cast<const Tok*>(a.q_norm),
      a.eps, a.heads, slice, slices, c0, c1, turns, cs, sn, place, lane);
  step = rows_of_kind<Rows::kKey, Tok, D, kInter>(
      static_cast<const Tok*>(a.k) + t * a.k_token, a.k_head,
      static_cast<Tok*>(kv.k) + place.page * kv.k_page + place.slot * kv.k_slot, kv.k_head,
      static_cast<const Tok*>(a.k_norm), a.eps, kv.kv_heads, step, slices, c0, c1, turns, cs, sn,
      place, lane);
  rows_of_kind<Rows::kValue, Tok, D, kInter>(
      static_cast<const Tok*>(a.v) + t * a.v_token, a.v_head,
      static_cast<Tok*>(kv.v) + place.page * kv.v_page + place.slot * kv.v_slot, kv.v_head,
      nullptr, 0.f, kv.kv_heads, step, slices, c0, c1, turns, cs, sn, place, lane);
}

template <typename Tok, int D, bool kInter>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  constexpr int kRows = 32 / (D / 16);
  const int steps = (a.heads + kRows - 1) / kRows + 2 * ((a.cache.kv_heads + kRows - 1) / kRows);
  // Few tokens: a warp for every step, for the shortest path. Many: as few
  // warps per token as still fill the GPU (kFillWarps), since each of them
  // looks its token up anew, a chain of four or five loads.
  const int slices = (int)std::min<int64_t>(steps, (kFillWarps + a.T - 1) / a.T);
  const int64_t warps = (int64_t)a.T * slices;
  const int64_t blocks = (warps + kAppendWarps - 1) / kAppendWarps;
  return launch_after_previous(append_kv_kernel<Tok, D, kInter>, dim3((unsigned)blocks),
                               dim3(kAppendWarps * 32), 0, stream, a, slices);
}

template <typename Tok, int D>
cudaError_t launch_style(const AppendArgs& a, bool interleaved, cudaStream_t stream) {
  return interleaved ? launch<Tok, D, true>(a, stream) : launch<Tok, D, false>(a, stream);
}

}  // namespace

cudaError_t launch_append_kv(const AppendArgs& a, bool interleaved, cudaStream_t stream) {
  if (a.cache.token_dtype == kTokenBF16)
    return a.cache.head_dim == 64 ? launch_style<__nv_bfloat16, 64>(a, interleaved, stream)
                                  : launch_style<__nv_bfloat16, 128>(a, interleaved, stream);
  return a.cache.head_dim == 64 ? launch_style<float, 64>(a, interleaved, stream)
                                : launch_style<float, 128>(a, interleaved, stream);
}

}  // namespace mxfp4el

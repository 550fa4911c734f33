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
// written; the rotation table adds rotary_dim floats per token.
//
// Layout: a row's lanes hold two chunks of 8 elements each (chunk j of the
// first half of the turned elements and its partner in the second half, so
// both rotation styles pair elements inside one thread; the chunks past
// rotary_dim pair up among themselves). head_dim / 16 lanes make a row, so a
// warp takes 32 / (head_dim / 16) rows at a time, of one token: the cosines
// and sines of the token stay in the lanes' registers for all of its rows.
#include "attn.cuh"

namespace mxfp4el {
namespace {

constexpr int kAppendWarps = 4;

template <typename Tok> struct Chunk8;   // 8 elements <-> 8 floats, 16-byte accesses

template <> struct Chunk8<__nv_bfloat16> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { raw = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
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
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(raw[i].x);
      x[4 * i + 1] = __uint_as_float(raw[i].y);
      x[4 * i + 2] = __uint_as_float(raw[i].z);
      x[4 * i + 3] = __uint_as_float(raw[i].w);
    }
  }
  __device__ __forceinline__ void pack(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      raw[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                          __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3]));
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<uint4*>(p)[0] = raw[0];
    reinterpret_cast<uint4*>(p)[1] = raw[1];
  }
};

// The pair (x, y) of chunks turned in place. Half style: element i of x with
// element i of y by (c[i], s[i]). Interleaved: elements 2i and 2i + 1 of x by
// (c[i], s[i]), of y by (c[4 + i], s[4 + i]).
template <bool kInter>
__device__ __forceinline__ void turn(float (&x)[8], float (&y)[8], const float (&c)[8],
                                     const float (&s)[8]) {
  if constexpr (kInter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1], e = y[2 * i], f = y[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = b * c[i] + a * s[i];
      y[2 * i] = e * c[4 + i] - f * s[4 + i];
      y[2 * i + 1] = f * c[4 + i] + e * s[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = y[i];
      x[i] = a * c[i] - b * s[i];
      y[i] = b * c[i] + a * s[i];
    }
  }
}

template <typename Tok, int D, bool kInter>
__global__ void __launch_bounds__(kAppendWarps * 32)
append_kv_kernel(const AppendArgs a, int slices) {
  constexpr int kLanes = D / 16;          // lanes of a row
  constexpr int kRows = 32 / kLanes;      // rows a warp holds at a time
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
  const bool turn_ok = a.rotary_dim == 0 || (pos_ok && pos < a.max_positions);
  int64_t page = -1;
  if (pos_ok) page = page_of(a.seqs, a.cache, seq, pos >> a.cache.page_shift);
  const bool store_ok = turn_ok && page >= 0;
  if (!past && !store_ok && slice == 0 && lane == 0) atomicAdd(&a.status[kStatusBadPages], 1ull);
  const int slot = pos & (a.cache.page_size - 1);

  // This lane's two chunks, and their cosines and sines.
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
  float cs[8], sn[8];
  if (turns && turn_ok) {
    const float* row = a.cos_sin + (int64_t)pos * a.rotary_dim + 8 * j;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = __ldg(row + i);
      sn[i] = __ldg(row + a.rotary_dim / 2 + i);
    }
  }

  const int rows = a.heads + 2 * a.cache.kv_heads;
  for (int h = slice * kRows + lane / kLanes; h < (rows + kRows - 1) / kRows * kRows;
       h += slices * kRows) {
    const bool live = h < rows;
    const bool is_q = h < a.heads, is_k = !is_q && h < a.heads + a.cache.kv_heads;
    const Tok* src;
    Tok* dst;
    const Tok* norm = nullptr;
    if (is_q) {
      src = static_cast<const Tok*>(a.q) + t * a.q_token + h * a.q_head;
      dst = static_cast<Tok*>(a.q_out) + ((int64_t)t * a.heads + h) * D;
      norm = static_cast<const Tok*>(a.q_norm);
    } else if (is_k) {
      const int kh = h - a.heads;
      src = static_cast<const Tok*>(a.k) + t * a.k_token + kh * a.k_head;
      dst = static_cast<Tok*>(a.cache.k) + page * a.cache.k_page + kh * a.cache.k_head +
            slot * a.cache.k_slot;
      norm = static_cast<const Tok*>(a.k_norm);
    } else {
      const int vh = min(h, rows - 1) - a.heads - a.cache.kv_heads;
      src = static_cast<const Tok*>(a.v) + t * a.v_token + vh * a.v_head;
      dst = static_cast<Tok*>(a.cache.v) + page * a.cache.v_page + vh * a.cache.v_head +
            slot * a.cache.v_slot;
    }
    Chunk8<Tok> u, w;
    u.load(src + 8 * c0);
    w.load(src + 8 * c1);
    float x[8], y[8];
    u.unpack(x);
    w.unpack(y);
    // The row's mean square over its lanes. Every lane of the warp takes part
    // in the shuffles; rows without a norm drop the result.
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += x[i] * x[i] + y[i] * y[i];
#pragma unroll
    for (int o = kLanes / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    if (is_q || is_k) {
      if (norm != nullptr) {
        const float inv = rsqrtf(sum * (1.0f / D) + a.eps);
        Chunk8<Tok> n0, n1;
        n0.load(norm + 8 * c0);
        n1.load(norm + 8 * c1);
        float f[8], g[8];
        n0.unpack(f);
        n1.unpack(g);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = x[i] * inv * f[i];
          y[i] = y[i] * inv * g[i];
        }
      }
      if (turns && turn_ok) turn<kInter>(x, y, cs, sn);
      if (is_q && (past || !turn_ok)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
      }
      u.pack(x);
      w.pack(y);
    }
    if (live && (is_q || store_ok)) {
      u.store(dst + 8 * c0);
      w.store(dst + 8 * c1);
    }
  }
}

template <typename Tok, int D, bool kInter>
cudaError_t launch(const AppendArgs& a, cudaStream_t stream) {
  constexpr int kRows = 32 / (D / 16);
  const int rows = a.heads + 2 * a.cache.kv_heads;
  const int slices = (rows + kRows - 1) / kRows;
  const int64_t warps = (int64_t)a.T * slices;
  const int64_t blocks = (warps + kAppendWarps - 1) / kAppendWarps;
  append_kv_kernel<Tok, D, kInter><<<(unsigned)blocks, kAppendWarps * 32, 0, stream>>>(a, slices);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) note_launch();
  return err;
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

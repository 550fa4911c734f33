// attn_simt.cu -- attention over the paged cache on the CUDA cores: any
// dtype, any number of new tokens, float32 arithmetic throughout.
//
// One block takes a tile of up to 64 query rows of one key head: n tokens of
// one sequence times the query heads that share the head (row i is token
// i / heads, head i % heads), so every key and value row is read once for all
// of them. The block walks the keys that any of its rows sees in tiles of 64,
// with the running maximum and sum of each row:
//
//   m' = max(m, max_j s_j),  l' = l e^(m - m') + sum_j e^(s_j - m'),
//   o' = o e^(m - m') + sum_j e^(s_j - m') v_j,   out = o / l
//
// in powers of two (log2 e is folded into the scale).
//
// Bound: FMA issue (2 D multiply-adds per row and key). 256 threads hold a
// 4 x 4 block of scores each and then 4 rows by D / 16 widths of the result:
// 16 multiply-adds per two 16-byte shared-memory reads.
#include "attn.cuh"

namespace mxfp4el {
namespace {

constexpr int kThreads = 256;
constexpr int kRowsTile = 64;     // query rows per block
constexpr int kKeysTile = 64;     // keys per step

template <typename Tok>
__device__ __forceinline__ float4 load4(const Tok* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

template <int D>
struct Smem {
  float q[kRowsTile][D + 4];       // row strides of D + 4: 16-byte reads of 8 rows hit all banks
  float k[kKeysTile][D + 4];
  float v[kKeysTile][D];
  float p[kRowsTile][kKeysTile + 4];
};

template <typename Tok, int D>
__global__ void __launch_bounds__(kThreads)
attention_simt_kernel(const AttnArgs a, int heads_tile, int head_blocks, int tokens_tile) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D>& sh = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int lane = threadIdx.x & 31;
  const int kvh = blockIdx.y / head_blocks;
  const int h0 = kvh * a.group + (blockIdx.y % head_blocks) * heads_tile;  // first query head
  const int nh = min(heads_tile, (kvh + 1) * a.group - h0);

  const int slot = blockIdx.x;
  const int b = sequence_of_slot(a.seqs, slot, a.T, tokens_tile, lane);
  const SeqRows r = sequence_rows(a.seqs, b, a.T, a.cache.page_shift, a.status,
                                  blockIdx.y == 0 && threadIdx.x == 0);
  const int tile = a.seqs.q_offsets == nullptr ? 0 : slot - (r.first / tokens_tile + b);
  const int t0 = tile * tokens_tile;                     // first new token of the tile
  const int nt = min(tokens_tile, r.count - t0);
  if (nt <= 0) return;
  const int rows = nt * nh;
  const int pos_lo = r.pos0 + t0, pos_hi = pos_lo + nt - 1;

  // Query rows; rows past the tile are zeros.
  for (int i = threadIdx.x; i < kRowsTile * (D / 4); i += kThreads) {
    const int row = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows)
      x = load4(static_cast<const Tok*>(a.q) + (int64_t)(r.first + t0 + row / nh) * a.q_token +
                (int64_t)(h0 + row % nh) * a.q_head + c);
    *reinterpret_cast<float4*>(&sh.q[row][c]) = x;
  }

  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // 4 rows ty * 4.., keys tx + 16 j
  const float scale = a.scale * kLog2e;
  float m[4], l[4], o[4][D / 16];
  int pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = ty * 4 + i;
    pos[i] = row < rows ? pos_lo + row / nh : -1;        // -1: sees nothing
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[i][d] = 0.f;
  }

  // Keys any row of the tile sees: [0, sinks) and [first, last].
  const int last = min(pos_hi, r.len - 1);
  const int first = a.window ? max(0, pos_lo - a.window + 1) : 0;
  for (int j0 = 0; j0 <= last; j0 += kKeysTile) {
    if (j0 >= a.sinks && j0 + kKeysTile <= first) {       // between the sinks and the window
      j0 = first / kKeysTile * kKeysTile - kKeysTile;
      continue;
    }
    __syncthreads();                                      // the last tile's readers are done
    for (int i = threadIdx.x; i < kKeysTile * (D / 4); i += kThreads) {
      const int j = i / (D / 4), c = i % (D / 4) * 4, key = j0 + j;
      float4 kx = make_float4(0.f, 0.f, 0.f, 0.f), vx = kx;
      if (key <= last && (key >= first || key < a.sinks)) {
        const int64_t page = page_of(a.seqs, a.cache, b, key >> a.cache.page_shift);
        const int s = key & (a.cache.page_size - 1);
        if (page >= 0) {
          kx = load4(static_cast<const Tok*>(a.cache.k) + page * a.cache.k_page +
                     kvh * a.cache.k_head + s * a.cache.k_slot + c);
          vx = load4(static_cast<const Tok*>(a.cache.v) + page * a.cache.v_page +
                     kvh * a.cache.v_head + s * a.cache.v_slot + c);
        } else if (c == 0 && (s == 0 || j == 0) && a.status != nullptr) {
          atomicAdd(&a.status[kStatusBadPages], 1ull);
        }
      }
      *reinterpret_cast<float4*>(&sh.k[j][c]) = kx;
      *reinterpret_cast<float4*>(&sh.v[j][c]) = vx;
    }
    __syncthreads();

    float s[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 qx[4], kx[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) qx[i] = *reinterpret_cast<const float4*>(&sh.q[ty * 4 + i][c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) kx[j] = *reinterpret_cast<const float4*>(&sh.k[tx + 16 * j][c]);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(qx[i].x, kx[j].x, s[i][j]);
          s[i][j] = fmaf(qx[i].y, kx[j].y, s[i][j]);
          s[i][j] = fmaf(qx[i].z, kx[j].z, s[i][j]);
          s[i][j] = fmaf(qx[i].w, kx[j].w, s[i][j]);
        }
    }
    // The mask cuts this tile when some row does not see all of its keys. Its
    // keys then carry p = -1 where a row does not see them, and the second
    // product skips those: a key or value that is not seen may be infinite
    // or NaN.
    const bool whole = rows == kRowsTile && j0 + kKeysTile - 1 <= pos_lo &&
                       (a.window == 0 || pos_hi - j0 < a.window);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx + 16 * j;
        s[i][j] *= scale;
        if (!whole && !(key <= last && key_visible(key, pos[i], a.window, a.sinks)))
          s[i][j] = -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1)
        top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
      const float base = top == -INFINITY ? 0.f : top;    // no key so far: every power is 0
      const float keep = exp2_approx(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx + 16 * j;
        float p = exp2_approx(s[i][j] - base);
        const bool hidden = !whole && !(key <= last && key_visible(key, pos[i], a.window, a.sinks));
        if (!hidden) sum += p;
        else p = -1.f;
        sh.p[ty * 4 + i][tx + 16 * j] = p;
      }
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) sum += __shfl_xor_sync(kFullMask, sum, off);
      m[i] = top;
      l[i] = l[i] * keep + sum;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[i][d] *= keep;
    }
    __syncwarp();                                         // a row's p stays in its half warp
#pragma unroll 2
    for (int j = 0; j < kKeysTile; j += 4) {
      float4 px[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) px[i] = *reinterpret_cast<const float4*>(&sh.p[ty * 4 + i][j]);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
        for (int d = 0; d < D / 64; ++d) {
          const float4 vx = *reinterpret_cast<const float4*>(&sh.v[j + jj][d * 64 + tx * 4]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float p = jj == 0 ? px[i].x : jj == 1 ? px[i].y : jj == 2 ? px[i].z : px[i].w;
            if (whole || p >= 0.f || p != p) {
              o[i][4 * d + 0] = fmaf(p, vx.x, o[i][4 * d + 0]);
              o[i][4 * d + 1] = fmaf(p, vx.y, o[i][4 * d + 1]);
              o[i][4 * d + 2] = fmaf(p, vx.z, o[i][4 * d + 2]);
              o[i][4 * d + 3] = fmaf(p, vx.w, o[i][4 * d + 3]);
            }
          }
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = ty * 4 + i;
    if (row >= rows) continue;
    const int h = h0 + row % nh;
    float total = l[i], f = 1.f;
    if (a.sink_logits != nullptr) {
      const float z = __ldg(a.sink_logits + h) * kLog2e;
      const float top = fmaxf(m[i], z), base = top == -INFINITY ? 0.f : top;
      f = exp2_approx(m[i] - base);
      total = total * f + exp2_approx(z - base);
    }
    const float inv = total == 0.f ? 0.f : f / total;
    Tok* out = static_cast<Tok*>(a.out) + ((int64_t)(r.first + t0 + row / nh) * a.heads + h) * D;
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
      store4(out + d * 64 + tx * 4, make_float4(o[i][4 * d] * inv, o[i][4 * d + 1] * inv,
                                                o[i][4 * d + 2] * inv, o[i][4 * d + 3] * inv));
  }
}

template <typename Tok, int D>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
  const int heads_tile = a.group < kRowsTile ? a.group : kRowsTile;
  const int head_blocks = (a.group + heads_tile - 1) / heads_tile;
  const int tokens_tile = kRowsTile / heads_tile;
  const dim3 grid((unsigned)query_tile_slots(a.seqs, a.T, tokens_tile),
                  (unsigned)(a.cache.kv_heads * head_blocks));
  const int smem = (int)sizeof(Smem<D>);
  cudaError_t err = cudaFuncSetAttribute(attention_simt_kernel<Tok, D>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  attention_simt_kernel<Tok, D><<<grid, kThreads, smem, stream>>>(a, heads_tile, head_blocks,
                                                                 tokens_tile);
  err = cudaGetLastError();
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace

cudaError_t launch_attention_simt(const AttnArgs& a, cudaStream_t stream) {
  if (a.cache.token_dtype == kTokenBF16)
    return a.cache.head_dim == 64 ? launch<__nv_bfloat16, 64>(a, stream)
                                  : launch<__nv_bfloat16, 128>(a, stream);
  return a.cache.head_dim == 64 ? launch<float, 64>(a, stream) : launch<float, 128>(a, stream);
}

}  // namespace mxfp4el

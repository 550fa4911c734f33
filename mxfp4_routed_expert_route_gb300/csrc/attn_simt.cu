// attn_simt.cu -- float32 attention of prompts over the paged cache, on the
// CUDA cores: the tensor cores take no float32 operands. (Split into three bf16
// terms each, with six of the nine products, they would keep the 24 bits at up
// to a sixth of the bf16 rate. Not built.)
//
// One block takes a tile of 16 kR query rows of one key head: n tokens of one
// sequence times the query heads that share the head (row i is token
// i / heads, head i % heads), so every key and value row is read once for all
// of them. The block walks the keys that any of its rows sees in tiles of 64,
// with the running maximum and sum of each row:
//
//   m' = max(m, max_j s_j),  l' = l e^(m - m') + sum_j e^(s_j - m'),
//   o' = o e^(m - m') + sum_j e^(s_j - m') v_j,   out = o / l
//
// in powers of two (log2 e is folded into the scale).
//
// Bound: FMA issue (2 D multiply-adds per row and key) for long prompts, the
// chain of one tile after another for short ones. 256 threads hold a kR x 4
// block of scores each and then kR rows by D / 16 widths of the result; with
// kR = 4 that is 64 multiply-adds per eight 16-byte shared-memory reads. The
// next tile is copied while this one is computed. Three prompts of up to 301
// tokens, 16 query and 4 key heads of 64: 34 us, five tiles one after another. A
// prompt of 4096 tokens, 16 query and 4 key heads of 128: 2.37 ms, 29 TFLOP/s
// of unmasked work. Where the heads of a group leave rows of a tile unused (3,
// 5, 6 or 7 heads), no tile counts as whole, and every step of the second product
// asks each row what it sees: 1024 tokens, 4 key heads of 128, 12.6 TFLOP/s with
// 3 heads to each and 15.4 with 4; 20.1 with 7 and 23.0 with 8.
//
// Few rows: where the tiles are fewer than the SMs, the keys of each are split
// over several blocks. Each leaves its (m, l, o) in the workspace, and the
// last to arrive joins them in their order along the keys (30 tokens behind
// 30000 keys, one key head: 3.2 ms in one block, 228 us split).
#include <algorithm>
#include <mutex>

#include "attn.cuh"

namespace mxfp4el {
namespace {

constexpr int kThreads = 256;
constexpr int kKeysTile = 64;     // keys per step

template <int D, int kR>
struct Smem {
  float q[16 * kR][D + 4];         // row strides of D + 4: 16-byte reads of 8 rows hit all banks
  float k[2][kKeysTile][D + 4];
  float v[2][kKeysTile][D];
  float p[16 * kR][kKeysTile + 4];
};

// 16 bytes global -> shared without a register; zeros where !valid.
__device__ __forceinline__ void copy16(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

// What the blocks of one tile share: `parts` of them, a counter per tile, and
// per (tile, part) 16 kR rows of o and then their m and l.
struct Split {
  int parts;
  unsigned int* counters;
  float* pieces;
};
constexpr int kMinPartTiles = 4;  // key tiles to a part at least: less than that costs a join

template <int D, int kR, bool kSplit>
__global__ void __launch_bounds__(kThreads)
attention_simt_kernel(const AttnArgs a, int heads_tile, int head_blocks, int tokens_tile,
                      const Split split) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem<D, kR>& sh = *reinterpret_cast<Smem<D, kR>*>(smem_raw);
  constexpr int kRowsTile = 16 * kR;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int kvh = blockIdx.y / head_blocks;
  const int h0 = kvh * a.group + (blockIdx.y % head_blocks) * heads_tile;  // first query head
  const int nh = min(heads_tile, (kvh + 1) * a.group - h0);

  const int slot = blockIdx.x;
  const int b = sequence_of_slot(a.seqs, slot, a.T, tokens_tile, lane);
  const SeqRows r = sequence_rows(a.seqs, b, a.T, a.cache.page_shift, a.status,
                                  blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0);
  const int tile = a.seqs.q_offsets == nullptr ? 0 : slot - (r.first / tokens_tile + b);
  const int t0 = tile * tokens_tile;                     // first new token of the tile
  const int nt = min(tokens_tile, r.count - t0);
  if (nt <= 0) return;
  const int rows = nt * nh;
  const int pos_lo = r.pos0 + t0, pos_hi = pos_lo + nt - 1;

  // Keys any row of the tile sees: [0, sinks) and [first, last], in tiles of
  // kKeysTile; this block takes tiles [i0, i1) of them.
  const int last = min(pos_hi, r.len - 1);
  const int first = a.window ? max(0, pos_lo - a.window + 1) : 0;
  const int first_tile = first / kKeysTile;
  const int sink_tiles = min((a.sinks + kKeysTile - 1) / kKeysTile, first_tile);
  const int tiles = last < 0 ? 0 : sink_tiles + last / kKeysTile - first_tile + 1;
  const int parts = kSplit ? max(1, min(split.parts, tiles / kMinPartTiles)) : 1;
  if ((int)blockIdx.z >= parts) return;
  const int i0 = kSplit ? (int)((int64_t)tiles * blockIdx.z / parts) : 0;
  const int i1 = kSplit ? (int)((int64_t)tiles * (blockIdx.z + 1) / parts) : tiles;

  // Query rows; rows past the tile are zeros.
  for (int i = threadIdx.x; i < kRowsTile * (D / 4); i += kThreads) {
    const int row = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < rows)
      x = __ldg(reinterpret_cast<const float4*>(
          static_cast<const float*>(a.q) + (int64_t)(r.first + t0 + row / nh) * a.q_token +
          (int64_t)(h0 + row % nh) * a.q_head + c));
    *reinterpret_cast<float4*>(&sh.q[row][c]) = x;
  }

  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // rows ty * kR.., keys tx + 16 j
  const float scale = a.scale * kLog2e;
  float m[kR], l[kR], o[kR][D / 16];
  int pos[kR];
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int row = ty * kR + i;
    pos[i] = row < rows ? pos_lo + row / nh : -1;        // -1: sees nothing
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[i][d] = 0.f;
  }

  auto tile_key = [&](int i) {
    return (i < sink_tiles ? i : first_tile + i - sink_tiles) * kKeysTile;
  };
  // Four threads copy a key's row and its value's; keys that no row sees and
  // page ids out of range become zeros.
  const int row = threadIdx.x >> 2;
  auto copy_tile = [&](int j0, int buf) {
    const int key = j0 + row;
    const bool want = key <= last && (key >= first || key < a.sinks);
    int64_t page = -1;
    const int s = key & (a.cache.page_size - 1);
    if (want) {
      page = page_of(a.seqs, a.cache, b, key >> a.cache.page_shift);
      // Counted at the page's first key that this tile wants.
      if (page < 0 && (threadIdx.x & 3) == 0 && (s == 0 || row == 0 || key == first))
        atomicAdd(&a.status[kStatusBadPages], 1ull);
    }
    const float* k = static_cast<const float*>(a.cache.k);
    const float* v = static_cast<const float*>(a.cache.v);
    if (page >= 0) {
      k += page * a.cache.k_page + kvh * a.cache.k_head + s * a.cache.k_slot;
      v += page * a.cache.v_page + kvh * a.cache.v_head + s * a.cache.v_slot;
    }
#pragma unroll
    for (int c = (threadIdx.x & 3) * 4; c < D; c += 16) {
      copy16(&sh.k[buf][row][c], k + (page >= 0 ? c : 0), page >= 0);
      copy16(&sh.v[buf][row][c], v + (page >= 0 ? c : 0), page >= 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (i0 < i1) copy_tile(tile_key(i0), 0);
  for (int it = i0, buf = 0; it < i1; ++it, buf ^= 1) {
    const int j0 = tile_key(it);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                   // this tile is there, the other buffer's readers are done
    if (it + 1 < i1) copy_tile(tile_key(it + 1), buf ^ 1);

    float s[kR][4];
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 qx[kR], kx[4];
#pragma unroll
      for (int i = 0; i < kR; ++i) qx[i] = *reinterpret_cast<const float4*>(&sh.q[ty * kR + i][c]);
#pragma unroll
      for (int j = 0; j < 4; ++j) kx[j] = *reinterpret_cast<const float4*>(&sh.k[buf][tx + 16 * j][c]);
#pragma unroll
      for (int i = 0; i < kR; ++i)
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
    for (int i = 0; i < kR; ++i) {
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
        sh.p[ty * kR + i][tx + 16 * j] = p;
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
      float4 px[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) px[i] = *reinterpret_cast<const float4*>(&sh.p[ty * kR + i][j]);
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
#pragma unroll
        for (int d = 0; d < D / 64; ++d) {
          const float4 vx = *reinterpret_cast<const float4*>(&sh.v[buf][j + jj][d * 64 + tx * 4]);
#pragma unroll
          for (int i = 0; i < kR; ++i) {
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

  if (kSplit && parts > 1) {
    constexpr size_t kPiece = (size_t)kRowsTile * (D + 2);
    const size_t at = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
    float* base = split.pieces + at * split.parts * kPiece;
    float* mine = base + blockIdx.z * kPiece;
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int row = ty * kR + i;
#pragma unroll
      for (int d = 0; d < D / 64; ++d)
        *reinterpret_cast<float4*>(mine + row * D + d * 64 + tx * 4) =
            make_float4(o[i][4 * d], o[i][4 * d + 1], o[i][4 * d + 2], o[i][4 * d + 3]);
      if (tx == 0) {
        mine[kRowsTile * D + row] = m[i];
        mine[kRowsTile * (D + 1) + row] = l[i];
      }
    }
    __threadfence();
    __shared__ int joins;
    __syncthreads();
    if (threadIdx.x == 0)
      joins = atomicInc(split.counters + at, (unsigned)(parts - 1)) == (unsigned)(parts - 1);
    __syncthreads();
    if (!joins) return;
    __threadfence();
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const float* stats = base + kRowsTile * D + ty * kR + i;
      m[i] = -INFINITY;
      for (int k = 0; k < parts; ++k) m[i] = fmaxf(m[i], __ldcg(stats + k * kPiece));
      l[i] = 0.f;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) o[i][d] = 0.f;
    }
    for (int k = 0; k < parts; ++k) {
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float* piece = base + k * kPiece;
        const int row = ty * kR + i;
        const float f = exp2_approx(__ldcg(piece + kRowsTile * D + row) -
                                    (m[i] == -INFINITY ? 0.f : m[i]));
        l[i] = fmaf(__ldcg(piece + kRowsTile * (D + 1) + row), f, l[i]);
#pragma unroll
        for (int d = 0; d < D / 64; ++d) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(piece + row * D + d * 64 + tx * 4));
          o[i][4 * d] = fmaf(x.x, f, o[i][4 * d]);
          o[i][4 * d + 1] = fmaf(x.y, f, o[i][4 * d + 1]);
          o[i][4 * d + 2] = fmaf(x.z, f, o[i][4 * d + 2]);
          o[i][4 * d + 3] = fmaf(x.w, f, o[i][4 * d + 3]);
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int row = ty * kR + i;
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
    float* out = static_cast<float*>(a.out) + ((int64_t)(r.first + t0 + row / nh) * a.heads + h) * D;
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
      *reinterpret_cast<float4*>(out + d * 64 + tx * 4) =
          make_float4(o[i][4 * d] * inv, o[i][4 * d + 1] * inv, o[i][4 * d + 2] * inv,
                      o[i][4 * d + 3] * inv);
  }
}

template <int D, int kR, bool kSplit>
cudaError_t launch_kernel(const AttnArgs& a, dim3 grid, int heads_tile, int head_blocks,
                          int tokens_tile, const Split& split, cudaStream_t stream) {
  const int smem = (int)sizeof(Smem<D, kR>);
  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t err = cudaSuccess;
  std::call_once(once[dev & 63], [&] {
    err = cudaFuncSetAttribute(attention_simt_kernel<D, kR, kSplit>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (err != cudaSuccess) return err;
  return launch_after_previous(attention_simt_kernel<D, kR, kSplit>, grid, dim3(kThreads), smem,
                               stream, a, heads_tile, head_blocks, tokens_tile, split);
}

template <int D, int kR>
cudaError_t launch(const AttnArgs& a, void* workspace, cudaStream_t stream) {
  const int heads_tile = std::min(a.group, 16 * kR);
  const int head_blocks = (a.group + heads_tile - 1) / heads_tile;
  const int tokens_tile = 16 * kR / heads_tile;
  dim3 grid((unsigned)query_tile_slots(a.seqs, a.T, tokens_tile),
            (unsigned)(a.cache.kv_heads * head_blocks));
  // Parts: up to two blocks per SM in all, and no more than the longest keys
  // that a row could see allow.
  const int64_t tiles = (int64_t)grid.x * grid.y, sms = attention_num_sms();
  Split split = {};
  split.parts = 1;
  split.counters = prefill_counters(workspace);
  split.pieces = static_cast<float*>(workspace_pieces(workspace));
  if (tiles < sms && tiles <= kPrefillCounters) {
    int64_t keys = (int64_t)a.seqs.max_pages << a.cache.page_shift;
    if (a.window > 0) keys = std::min<int64_t>(keys, (int64_t)a.window + a.sinks + tokens_tile + 128);
    split.parts = (int)std::max<int64_t>(
        1, std::min<int64_t>(2 * sms / tiles, keys / (kMinPartTiles * kKeysTile)));
  }
  grid.z = (unsigned)split.parts;
  return split.parts > 1 ? launch_kernel<D, kR, true>(a, grid, heads_tile, head_blocks, tokens_tile,
                                                      split, stream)
                         : launch_kernel<D, kR, false>(a, grid, heads_tile, head_blocks,
                                                       tokens_tile, split, stream);
}

// Tiles of 64 rows, or of 32 where 64 would leave SMs without a second block
// to hide the first one's waits behind. 16 query and 4 key heads of 128, us with
// 64 and 32 rows: 300 tokens 59 and 43, 2048 tokens 708 and 911, 4096 tokens 2370
// and 3280; heads of 64: 300 tokens 44 and 33, 4096 tokens 1245 and 1558. (Between
// them heads of 128 would take 64 rows sooner: 1024 tokens 241 and 279.)
template <int D>
cudaError_t launch_rows(const AttnArgs& a, void* workspace, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.T * a.heads;
  return rows >= 2 * 64 * (int64_t)attention_num_sms() ? launch<D, 4>(a, workspace, stream)
                                                       : launch<D, 2>(a, workspace, stream);
}

}  // namespace

cudaError_t launch_attention_simt(const AttnArgs& a, void* workspace, cudaStream_t stream) {
  return a.cache.head_dim == 64 ? launch_rows<64>(a, workspace, stream)
                                : launch_rows<128>(a, workspace, stream);
}

}  // namespace mxfp4el

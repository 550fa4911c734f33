// gemm_mx.cu -- products of MXFP4 tokens and MXFP4 weights on the 5th-gen
// tensor cores (tcgen05 kind::mxf4 with block scales, TMEM, TMA).
//
//   D[t, o] = sum_g 2^(sx[t,g]-127) 2^(sw[o,g]-127) sum_{i in g} cx[t,i] cw[o,i]
//
// over groups g of 32: both operands stay in 4 bits from memory to the tensor
// core, which multiplies the E2M1 codes, applies both groups' scale bytes and
// adds in float32 into tensor memory. Nothing is decoded by this kernel.
//
// Shape ("swap AB"): M = 128 weight rows, N = up to kN tokens of one block (a
// multiple of 16), K in stages of 256 values (128 bytes of codes per row, the
// width of a 128-byte swizzle atom), four MMAs of K = 64 each. With few tokens
// the weights alone are read from HBM, so the weights take the operand with
// the fixed 128 rows and the tokens the one whose width can be small.
//
// Routed (kRouted): a block is up to kN of one expert's pairs in the lists of
// route.cu; the token rows are gathered by the copies themselves (four rows
// each, tile::gather4), and float32 results go to part[pair][split][o]. Dense:
// a block is consecutive tokens and results go to out[t][o], or to
// part[t][split][o] where K is split over several units.
//
// Scale bytes. The tensor core wants them in tensor memory, 32 lanes by 4
// bytes of 128 rows' scales for four groups (512 bytes); tcgen05.cp brings
// such a block from shared memory and repeats it for the four lane quarters.
// In memory they are rows of I/32 bytes on no particular alignment, so four
// warps read them with ordinary loads (32 bytes of a row at a time, one row
// per thread, one chunk ahead) and store each row's four bytes of four groups
// where the block has them: row r at 16 (r % 32) + 4 (r / 32).
//
// K that is no multiple of 256: the copies fill codes past a row's end with
// zeros, and scale bytes past it are set to 0, so what is added is exactly 0;
// MMAs wholly past the end are not issued.
//
// Warp roles in a CTA of 12 warps (one CTA per SM, persistent over units
// (block, 128-row tile, K split) in a fixed order):
//   warp 0      copies of codes (weights and tokens), TMEM allocation
//   warp 1      scale copies to tensor memory and MMAs, one elected lane
//   warp 2      prefix of the experts' blocks at start (routed)
//   warps 4-7   scale bytes
//   warps 8-11  epilogue: tensor memory -> float32 or bf16 results
// Two accumulators, so the epilogue of a unit runs beside the next unit's
// MMAs. Every wait is bounded; a role whose wait gives up records it and
// stops, and the CTA waits (bounded) for its own copies and MMAs before
// freeing TMEM.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "quant.h"

namespace mxfp4el {
namespace {

constexpr int kThreads = 384;
constexpr int kBM = 128;                       // weight rows per tile
constexpr int kBK = 256;                       // K values per stage
constexpr int kMmaK = 64;                      // K values per MMA
constexpr int kGroupsPerStage = kBK / 32;
constexpr uint32_t kRowBytes = kBK / 2;        // codes of a row per stage
constexpr uint32_t kStageA = kBM * kRowBytes;
constexpr uint32_t kSfBlock = 512;             // 128 rows' scales of four groups
constexpr int kSfPerStage = kGroupsPerStage / 4;
constexpr int kMaxStages = 12;
constexpr uint32_t kTmemCols = 512;
constexpr int kScaleWarp0 = 4, kScaleWarps = 4, kEpiWarp0 = 8, kEpiWarps = 4;
constexpr int kChunkStages = 4;                // stages whose scales one read brings (32 bytes)
constexpr size_t kSmemLimit = 227 * 1024;

template <int kN>
struct Shape {
  static constexpr int kBRowBlocks = (kN + 127) / 128;    // 128-row scale blocks of the tokens
  static constexpr uint32_t kStageB = kN * kRowBytes;
  static constexpr uint32_t kSfA = kSfPerStage * kSfBlock;
  static constexpr uint32_t kSfB = kSfPerStage * kBRowBlocks * kSfBlock;
  static constexpr uint32_t kStage = kStageA + kStageB + kSfA + kSfB;
  // TMEM: two accumulators of kN columns, then per stage the scales.
  static constexpr uint32_t kSfColsA = kSfPerStage * 4, kSfColsB = kSfPerStage * kBRowBlocks * 4;
  static constexpr uint32_t kSfCol = 2 * kN;
  static constexpr int kTmemStages = (int)((kTmemCols - kSfCol) / (kSfColsA + kSfColsB));
  static_assert(kStage % 1024 == 0 && kStageB % 1024 == 0, "stages keep 1024-byte alignment");
};

struct MxMaps {
  CUtensorMap a;      // weights' codes [E][O][I/2], box {128, 128, 1}, 128-byte swizzle
  CUtensorMap b;      // tokens' codes [T][I/2], box {128, 32} (dense) or {128, 1} (gathered)
};

struct MxKernelArgs {
  RoutePlan plan;               // routed
  const uint8_t* w_scales;      // [E][O][G]
  const uint8_t* x_scales;      // [T][G]
  void* out;
  unsigned long long* status;
  int T, O, G, K;
  int mtiles, splits, stages, max_active;
};

struct __align__(16) MxShared {
  uint64_t full_tma[kMaxStages], full_sf[kMaxStages], empty[kMaxStages];
  uint64_t d_full[2], d_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int num_units, num_active;
};

__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " .reg .b32 r;\n"
      " elect.sync r|p, 0xffffffff;\n"
      " selp.u32 %0, 1, 0, p;\n"
      "}"
      : "=r"(e));
  return e != 0;
}

// Four rows of 128 bytes by their row indices, one after another at dst.
__device__ __forceinline__ void tma_gather4(void* dst, const void* tmap, int x, int4 rows,
                                            uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(x), "r"(rows.x), "r"(rows.y), "r"(rows.z), "r"(rows.w), "r"(smem_addr(bar)),
      "l"(policy)
      : "memory");
}

// A 512-byte block of scales from shared to tensor memory, four columns.
__device__ __forceinline__ void tc_copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc)
               : "memory");
}

// D[tmem] (+)= A[smem] x B[smem] with block scales of 32 values in tensor memory.
__device__ __forceinline__ void tc_mma_mxf4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " setp.ne.b32 p, %6, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n"
      "}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::mxf4: E2M1 operands, both K-major, E8M0
// scales, shape 128 x n, the scales' bytes sf and sf + 1 of each 32-bit word.
__device__ __forceinline__ uint32_t mma_idesc(int n, uint32_t sf) {
  return (sf << 4)                       // B scale bytes
         | (1u << 7) | (1u << 10)        // A and B format: E2M1
         | ((uint32_t)(n >> 3) << 17)    // N / 8
         | (1u << 23)                    // scale format: E8M0
         | ((uint32_t)(kBM >> 4) << 24)  // M / 16
         | (sf << 29);                   // A scale bytes
}

// K-major tile with the 128-byte swizzle: 128-byte rows, 8-row atoms 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// Rows of 16 bytes without a swizzle: 8-row atoms 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_rows16(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}

struct RingPos {
  int idx = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int n) {
    if (++idx == n) {
      idx = 0;
      phase ^= 1u;
    }
  }
};

// One unit of work, derived identically by every role from its index.
struct Unit {
  int e;              // expert (0 when dense)
  int m0;             // first weight row
  int tok0, ntok;     // block: first position (in the lists, or token) and tokens
  int nmma;           // MMA N: ntok rounded up to 16
  int split;
  int kt0, kt1;       // stages of K
};

template <int kN, bool kRouted>
__device__ __forceinline__ Unit unit_at(const MxKernelArgs& a, const int* prefix, int num_active,
                                        int idx) {
  Unit w;
  const int per_block = a.mtiles * a.splits;
  int first = 0, nblk, cnt, local;
  if constexpr (kRouted) {
    const int blk = idx / per_block;
    int lo = 0, hi = num_active;           // prefix[u] <= blk < prefix[u + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= blk) lo = mid;
      else hi = mid;
    }
    w.e = a.plan.active[lo];
    first = a.plan.offsets[w.e];
    cnt = a.plan.offsets[w.e + 1] - first;
    nblk = prefix[lo + 1] - prefix[lo];
    local = idx - prefix[lo] * per_block;
  } else {
    w.e = 0;
    cnt = a.T;
    nblk = (a.T + kN - 1) / kN;
    local = idx;
  }
  // The blocks of a tile follow one another, so its codes come from L2 after
  // the first. Equal blocks, each a multiple of 16 tokens but the last.
  const int rest = local / nblk, j = local - rest * nblk;
  const int bsz = ((cnt + nblk - 1) / nblk + 15) / 16 * 16;
  w.tok0 = first + j * bsz;
  w.ntok = max(0, min(bsz, cnt - j * bsz));
  w.nmma = (w.ntok + 15) / 16 * 16;
  w.split = rest / a.mtiles;
  w.m0 = (rest - w.split * a.mtiles) * kBM;
  const int nk = (a.G + kGroupsPerStage - 1) / kGroupsPerStage;
  w.kt0 = (int)((int64_t)w.split * nk / a.splits);
  w.kt1 = (int)((int64_t)(w.split + 1) * nk / a.splits);
  return w;
}

// 32 bytes from p as eight words; bytes at `end` and past it are 0. Reads
// only aligned words that hold a byte before `end`.
__device__ __forceinline__ void load_scales(const uint8_t* p, const uint8_t* end,
                                            uint32_t (&w)[8]) {
  const int64_t left = end - p;
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && left >= 32) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint4 v = *reinterpret_cast<const uint4*>(p + 16);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
    return;
  }
  const uint32_t sh = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 3) * 8;
  const uint8_t* at = p - sh / 8;
  uint32_t v[9];
#pragma unroll
  for (int i = 0; i < 9; ++i)
    v[i] = at + 4 * i < end ? *reinterpret_cast<const uint32_t*>(at + 4 * i) : 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = __funnelshift_r(v[i], v[i + 1], sh);
    const int64_t n = left - 4 * i;
    if (n < 4) w[i] = n > 0 ? w[i] & ((1u << (8 * (int)n)) - 1u) : 0u;
  }
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <int kN, typename Out, bool kRouted>
__global__ void __launch_bounds__(kThreads, 1)
gemm_mx_kernel(const __grid_constant__ MxMaps maps, const MxKernelArgs a) {
  using S = Shape<kN>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  MxShared& sh = *reinterpret_cast<MxShared*>(ring + (size_t)a.stages * S::kStage);
  int* prefix = reinterpret_cast<int*>(&sh + 1);       // [max_active + 1] (routed)

  const int warp = __shfl_sync(kFullMask, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sh.full_tma[s], 1);
      mbar_init(&sh.full_sf[s], kScaleWarps);
      mbar_init(&sh.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.d_full[b], 1);
      mbar_init(&sh.d_empty[b], kEpiWarps);
    }
    mbar_init(&sh.drain, 32);                          // every lane of the MMA warp
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem_base, kTmemCols);
    tmem_relinquish();
    if (lane == 0) {
      prefetch_tensor_map(&maps.a);
      prefetch_tensor_map(&maps.b);
    }
  }
  pdl_wait();                    // the operands and the routing lists are ready
  if (warp == 2) {
    if constexpr (kRouted) {
      const int na = a.plan.meta[kMetaNumActive];
      int run = 0;
      for (int base = 0; base < na; base += 32) {
        const int u = base + lane;
        int nb = 0;
        if (u < na) {
          const int e = a.plan.active[u];
          nb = (a.plan.offsets[e + 1] - a.plan.offsets[e] + kN - 1) / kN;
        }
        int incl = nb;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int v = __shfl_up_sync(kFullMask, incl, off);
          if (lane >= off) incl += v;
        }
        if (u < na) prefix[u] = run + incl - nb;
        run += __shfl_sync(kFullMask, incl, 31);
      }
      if (lane == 0) {
        prefix[na] = run;
        sh.num_active = na;
        sh.num_units = run * a.mtiles * a.splits;
      }
    } else if (lane == 0) {
      sh.num_active = 0;
      sh.num_units = (a.T + kN - 1) / kN * a.mtiles * a.splits;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(kFullMask, sh.tmem_base, 0);
  const int num_units = sh.num_units, num_active = sh.num_active;
  const uint32_t ring_addr = __shfl_sync(kFullMask, smem_addr(ring), 0);
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------ copies of codes
    const uint64_t pol_once = l2_evict_first_policy(), pol_keep = l2_evict_last_policy();
    const uint64_t pol_reuse = l2_evict_normal_policy();
    RingPos pos;
    int issued = 0;
    for (int idx = blockIdx.x; idx < num_units && ok; idx += gridDim.x) {
      const Unit w = unit_at<kN, kRouted>(a, prefix, num_active, idx);
      if (w.ntok <= 0) continue;
      // Weights that one block reads pass through L2 once.
      const bool once = kRouted ? w.ntok <= kN && w.tok0 == a.plan.offsets[w.e] &&
                                      w.ntok == a.plan.offsets[w.e + 1] - w.tok0
                                : a.T <= kN;
      const uint64_t pol = once ? pol_once : pol_reuse;
      const uint32_t box = kRouted ? (uint32_t)w.nmma : (uint32_t)(w.nmma + 31) / 32 * 32;
      // Rows of this lane's gathers, four each; past the block its last token.
      constexpr int kGathers = (kN / 4 + 31) / 32;
      int4 rows[kGathers];
      if constexpr (kRouted) {
#pragma unroll
        for (int q = 0; q < kGathers; ++q) {
          int r[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int n = min((lane + 32 * q) * 4 + i, w.ntok - 1);
            r[i] = a.plan.pair_list[w.tok0 + n] / a.K;
          }
          rows[q] = make_int4(r[0], r[1], r[2], r[3]);
        }
      }
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++issued) {
        if (!mbar_wait_warp(&sh.empty[pos.idx], pos.phase ^ 1u)) {
          ok = false;
          break;
        }
        unsigned char* stage = ring + (size_t)pos.idx * S::kStage;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sh.full_tma[pos.idx], kStageA + box * kRowBytes);
          tma_load_3d(stage, &maps.a, kt * (int)kRowBytes, w.m0, w.e, &sh.full_tma[pos.idx], pol);
          if constexpr (!kRouted)
            for (int r = 0; r < (int)box; r += 32)
              tma_load_2d(stage + kStageA + r * kRowBytes, &maps.b, kt * (int)kRowBytes,
                          w.tok0 + r, &sh.full_tma[pos.idx], pol_keep);
        }
        __syncwarp();
        if constexpr (kRouted) {
#pragma unroll
          for (int q = 0; q < kGathers; ++q)
            if ((lane + 32 * q) * 4 < w.nmma)
              tma_gather4(stage + kStageA + (lane + 32 * q) * 4 * kRowBytes, &maps.b,
                          kt * (int)kRowBytes, rows[q], &sh.full_tma[pos.idx], pol_keep);
          __syncwarp();
        }
        pos.next(a.stages);
      }
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
    // Wait (bounded) until the copies this warp issued have landed: the last
    // min(issued, stages) uses of the ring.
    if (lane == 0) {
      for (int k = 0; k < min(issued, a.stages); ++k) {
        int idx = pos.idx - 1 - k;
        uint32_t ph = pos.phase;
        if (idx < 0) { idx += a.stages; ph ^= 1u; }
        if (!mbar_wait(&sh.full_tma[idx], ph)) break;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    RingPos pos;
    int it = 0;
    for (int idx = blockIdx.x; idx < num_units && ok; idx += gridDim.x) {
      const Unit w = unit_at<kN, kRouted>(a, prefix, num_active, idx);
      if (w.ntok <= 0) continue;
      const int buf = it & 1;
      if (!mbar_wait_warp(&sh.d_empty[buf], ((uint32_t)(it >> 1) & 1u) ^ 1u)) { ok = false; break; }
      tc_fence_after_sync();
      const uint32_t d = tmem + buf * kN;
      for (int kt = w.kt0; kt < w.kt1; ++kt) {
        if (!mbar_wait_warp(&sh.full_sf[pos.idx], pos.phase) ||
            !mbar_wait_warp(&sh.full_tma[pos.idx], pos.phase)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        if (elect_one()) {
          const uint32_t stage = ring_addr + pos.idx * S::kStage;
          const uint32_t sf = stage + kStageA + S::kStageB;
          const uint32_t tsfa = tmem + S::kSfCol + pos.idx * (S::kSfColsA + S::kSfColsB);
          const uint32_t tsfb = tsfa + S::kSfColsA;
#pragma unroll
          for (int b = 0; b < kSfPerStage; ++b) {
            tc_copy_scales(tsfa + 4 * b, smem_desc_rows16(sf + b * kSfBlock));
#pragma unroll
            for (int r = 0; r < S::kBRowBlocks; ++r)
              tc_copy_scales(tsfb + 4 * (b * S::kBRowBlocks + r),
                             smem_desc_rows16(sf + S::kSfA + (b * S::kBRowBlocks + r) * kSfBlock));
          }
          const uint64_t da = smem_desc_sw128(stage), db = smem_desc_sw128(stage + kStageA);
          const int left = a.G * 32 - kt * kBK;
#pragma unroll
          for (int j = 0; j < kBK / kMmaK; ++j) {
            if (j * kMmaK < left) {
              const int b = j / 2;
              tc_mma_mxf4(d, da + j * 2, db + j * 2, mma_idesc(w.nmma, (j & 1) * 2), tsfa + 4 * b,
                          tsfb + 4 * b * S::kBRowBlocks, kt > w.kt0 || j > 0 ? 1u : 0u);
            }
          }
          tc_commit(&sh.empty[pos.idx]);
          if (kt == w.kt1 - 1) tc_commit(&sh.d_full[buf]);
        }
        __syncwarp();
        pos.next(a.stages);
      }
      ++it;
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
    // Any lane may have been the elected one.
    tc_commit(&sh.drain);
    mbar_wait(&sh.drain, 0);
    __syncwarp();
  } else if (warp >= kScaleWarp0 && warp < kScaleWarp0 + kScaleWarps) {
    // ---------------------------------------------------------- scale bytes
    constexpr int kRows = 1 + S::kBRowBlocks;     // rows of this thread: a weight, 1 or 2 tokens
    const int m = (warp - kScaleWarp0) * 32 + lane;
    RingPos pos;
    for (int idx = blockIdx.x; idx < num_units && ok; idx += gridDim.x) {
      const Unit w = unit_at<kN, kRouted>(a, prefix, num_active, idx);
      if (w.ntok <= 0) continue;
      const uint8_t* p[kRows];
      const uint8_t* end[kRows];
      p[0] = a.w_scales + ((size_t)w.e * a.O + min(w.m0 + m, a.O - 1)) * a.G;
#pragma unroll
      for (int r = 1; r < kRows; ++r) {
        const int n = w.tok0 + min(m + 128 * (r - 1), w.ntok - 1);
        const int t = kRouted ? a.plan.pair_list[n] / a.K : n;
        p[r] = a.x_scales + (size_t)t * a.G;
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        end[r] = p[r] + a.G;
        p[r] += w.kt0 * kGroupsPerStage;
      }
      uint32_t cur[kRows][8], nxt[kRows][8];
#pragma unroll
      for (int r = 0; r < kRows; ++r) load_scales(p[r], end[r], cur[r]);
      for (int kt = w.kt0; kt < w.kt1 && ok; kt += kChunkStages) {
        if (kt + kChunkStages < w.kt1) {
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            p[r] += kChunkStages * kGroupsPerStage;
            load_scales(p[r], end[r], nxt[r]);
          }
        }
#pragma unroll
        for (int j = 0; j < kChunkStages; ++j) {
          if (kt + j >= w.kt1) break;
          if (!mbar_wait_warp(&sh.empty[pos.idx], pos.phase ^ 1u)) {
            ok = false;
            break;
          }
          unsigned char* sf = ring + (size_t)pos.idx * S::kStage + kStageA + S::kStageB +
                              (m & 31) * 16 + (m >> 5) * 4;
#pragma unroll
          for (int b = 0; b < kSfPerStage; ++b) {
            *reinterpret_cast<uint32_t*>(sf + b * kSfBlock) = cur[0][kSfPerStage * j + b];
#pragma unroll
            for (int r = 1; r < kRows; ++r)
              *reinterpret_cast<uint32_t*>(sf + S::kSfA +
                                           (b * S::kBRowBlocks + r - 1) * kSfBlock) =
                  cur[r][kSfPerStage * j + b];
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full_sf[pos.idx]);
          pos.next(a.stages);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int i = 0; i < 8; ++i) cur[r][i] = nxt[r][i];
      }
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------- epilogue
    const int quarter = warp - kEpiWarp0;
    Out* out = static_cast<Out*>(a.out);
    int it = 0;
    for (int idx = blockIdx.x; idx < num_units; idx += gridDim.x) {
      const Unit w = unit_at<kN, kRouted>(a, prefix, num_active, idx);
      if (w.ntok <= 0) continue;
      const int buf = it & 1;
      if (!mbar_wait_warp(&sh.d_full[buf], (uint32_t)(it >> 1) & 1u)) { ok = false; break; }
      tc_fence_after_sync();
      const int o = w.m0 + quarter * 32 + lane;
      for (int c0 = 0; c0 < w.ntok; c0 += 32) {
        const int n = min(32, w.ntok - c0);
        int row = w.tok0 + c0 + min(lane, n - 1);
        if constexpr (kRouted) row = a.plan.pair_list[row];
        float v[32];
        tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * kN + c0, v);
        tmem_wait_ld();
        if (c0 + 32 >= w.ntok) {                 // the accumulator may be written again
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.d_empty[buf]);
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const int r = __shfl_sync(kFullMask, row, c);
          if (c < n && o < a.O)
            store_out(out + ((int64_t)r * a.splits + w.split) * a.O + o, v[c]);
        }
      }
      ++it;
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// Joins the splits of a dense product: out[t, o] = sum_s part[t][s][o], s in order.
template <typename Out>
__global__ void __launch_bounds__(256)
join_splits_kernel(const float* __restrict__ part, int splits, int64_t T, int64_t O,
                   Out* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t n = T * O, step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) {
    const int64_t t = i / O, o = i - t * O;
    const float* p = part + t * splits * O + o;
    float v = p[0];
    for (int s = 1; s < splits; ++s) v += p[(int64_t)s * O];
    store_out(out + i, v);
  }
}

int num_sms() {
  static std::mutex mu;
  static int cached[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  std::lock_guard<std::mutex> lock(mu);
  if (cached[dev] == 0) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cached[dev] = n > 0 ? n : 152;
  }
  return cached[dev];
}

template <int kN>
size_t smem_bytes(int stages, int max_active) {
  return 1024 + (size_t)stages * Shape<kN>::kStage + sizeof(MxShared) +
         ((size_t)max_active + 1) * sizeof(int);
}

template <int kN>
int stages_for(int max_active) {
  int s = std::min(kMaxStages, Shape<kN>::kTmemStages);
  while (s > 0 && smem_bytes<kN>(s, max_active) > kSmemLimit) --s;
  return s;
}

template <int kN, typename Out, bool kRouted>
cudaError_t launch_typed(const MxMaps& maps, MxKernelArgs args, int64_t units,
                         cudaStream_t stream) {
  args.stages = stages_for<kN>(args.max_active);
  if (args.stages < 2) return cudaErrorInvalidValue;
  const size_t smem = smem_bytes<kN>(args.stages, args.max_active);
  static std::mutex mu;
  static size_t opted[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 0 && dev < 64 && opted[dev] < smem) {
      const cudaError_t err =
          cudaFuncSetAttribute(gemm_mx_kernel<kN, Out, kRouted>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (err != cudaSuccess) return err;
      opted[dev] = smem;
    }
  }
  const unsigned grid = (unsigned)std::min<int64_t>(units, num_sms());
  return launch_after_previous(gemm_mx_kernel<kN, Out, kRouted>, dim3(grid), dim3(kThreads), smem,
                               stream, maps, args);
}

bool encode(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 enc =
      reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  const cuuint32_t one[3] = {1, 1, 1};
  return enc != nullptr &&
         enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims,
             strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Wide blocks where experts (or the dense call) average more tokens than a
// narrow block holds; a batch of up to 32 tokens has no wider block.
bool gemm_mx_wide(int64_t T, int64_t blocks_of, int64_t K) {
  return T > 32 && T * K > 16 * blocks_of;
}

int gemm_mx_splits(int64_t T, int64_t E, int64_t I, int64_t O, int64_t K, bool routed) {
  const int64_t active = routed ? std::min(E, T * K) : 1;
  const bool wide = gemm_mx_wide(T, active, routed ? K : 1);
  const int64_t n = wide ? 192 : 32;
  const int64_t blocks = routed ? active : (T + n - 1) / n;
  const int64_t tiles = blocks * ((O + kBM - 1) / kBM);
  const int64_t nk = (I + kBK - 1) / kBK;
  return (int)std::max<int64_t>(1, std::min(std::min<int64_t>(304 / tiles, nk / 2),
                                            (int64_t)8));
}

bool gemm_mx_supported(int64_t T, int64_t E, int64_t K) {
  return std::min(E, T * K) <= kMxMaxActive;
}

cudaError_t launch_gemm_mx(const MxGemm& g, cudaStream_t stream) {
  MxMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  const cuuint64_t row = (cuuint64_t)(g.I / 2);
  {
    const cuuint64_t dims[3] = {row, (cuuint64_t)g.O, (cuuint64_t)g.E};
    const cuuint64_t strides[2] = {row, row * (cuuint64_t)g.O};
    const cuuint32_t box[3] = {kRowBytes, kBM, 1};
    if (!encode(&maps.a, g.w_packed, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  const bool routed = g.plan != nullptr;
  {
    const cuuint64_t dims[2] = {row, (cuuint64_t)g.T};
    const cuuint64_t strides[1] = {row};
    const cuuint32_t box[2] = {kRowBytes, routed ? 1u : 32u};
    if (!encode(&maps.b, g.x_packed, 2, dims, strides, box)) return cudaErrorInvalidValue;
  }
  MxKernelArgs a;
  std::memset(static_cast<void*>(&a), 0, sizeof(a));
  if (routed) a.plan = *g.plan;
  a.w_scales = g.w_scales;
  a.x_scales = g.x_scales;
  a.out = g.splits > 1 || routed ? static_cast<void*>(g.part) : g.out;
  a.status = device_status_words();
  if (a.status == nullptr) return cudaErrorUnknown;
  a.T = (int)g.T;
  a.O = (int)g.O;
  a.G = (int)(g.I / 32);
  a.K = (int)g.K;
  a.mtiles = (int)((g.O + kBM - 1) / kBM);
  a.splits = g.splits;
  const int64_t active = routed ? std::min(g.E, g.T * g.K) : 1;
  a.max_active = routed ? (int)active : 0;
  const bool wide = gemm_mx_wide(g.T, active, routed ? g.K : 1);
  const int64_t n = wide ? 192 : 32;
  // At most this many blocks: each expert's last one may be short.
  const int64_t blocks = routed ? active + g.T * g.K / n : (g.T + n - 1) / n;
  const int64_t units = blocks * a.mtiles * a.splits;
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t err;
  if (routed)
    err = wide ? launch_typed<192, float, true>(maps, a, units, stream)
               : launch_typed<32, float, true>(maps, a, units, stream);
  else if (g.splits > 1 || g.out_dtype == kTokenF32)
    err = wide ? launch_typed<192, float, false>(maps, a, units, stream)
               : launch_typed<32, float, false>(maps, a, units, stream);
  else
    err = wide ? launch_typed<192, __nv_bfloat16, false>(maps, a, units, stream)
               : launch_typed<32, __nv_bfloat16, false>(maps, a, units, stream);
  if (err != cudaSuccess || routed || g.splits == 1) return err;
  const unsigned grid = (unsigned)std::min<int64_t>((g.T * g.O + 255) / 256, num_sms() * 8);
  if (g.out_dtype == kTokenF32)
    return launch_after_previous(join_splits_kernel<float>, dim3(grid), dim3(256), 0, stream,
                                 static_cast<const float*>(g.part), g.splits, g.T, g.O,
                                 static_cast<float*>(g.out));
  return launch_after_previous(join_splits_kernel<__nv_bfloat16>, dim3(grid), dim3(256), 0, stream,
                               static_cast<const float*>(g.part), g.splits, g.T, g.O,
                               static_cast<__nv_bfloat16*>(g.out));
}

}  // namespace mxfp4el

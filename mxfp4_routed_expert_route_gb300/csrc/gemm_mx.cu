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
// Routed: a block is up to kN of one expert's pairs in the lists of route.cu,
// and float32 results go to part[pair][split][o]. Narrow blocks (kN = 32)
// gather their token rows with the copies themselves (four rows each,
// tile::gather4); wide ones read a copy of the rows in the lists' order, since
// gathers issue one at a time (some 75 cycles each; with them the skewed
// prefill's product took 4.0 ms, without the tokens 1.5). Dense: a block is
// consecutive tokens and results go to out[t][o], or to part[t][split][o] where
// K is split over several units (gemm_mx_plan).
//
// Scale bytes. The tensor core wants them in tensor memory, 32 lanes by 4
// bytes of 128 rows' scales for four groups (512 bytes, row r at 16 (r % 32) +
// 4 (r / 32)); tcgen05.cp brings such a block from shared memory and repeats it
// for the four lane quarters. In memory they are rows of I/32 bytes on no
// particular alignment, so a few warps read them with ordinary loads and store
// the blocks, lane l the rows l, l + 32, ..., whose words lie together in the
// block. A warp takes two stages at a time (16 bytes of a row) and has its next
// two stages' loads under way while it stores these. Two teams of warps take two
// stages in turn. From a team's last stage to its next it is then three, and the
// ring has more (from one further on than the ring is long a warp could not
// tell a stage's phases apart, and would store into one still in use).
//
// K that is no multiple of 256: the copies fill codes past a row's end with
// zeros, and scale bytes past it are set to 0, so what is added is exactly 0;
// MMAs wholly past the end are not issued.
//
// Every CTA copies its own operands: this library is loaded wherever the
// framework runs, and its copies name one CTA's memory alone. In wide blocks an SM
// reads 40 KB of codes per stage from L2, which bounds the dense product.
//
// Warp roles in a CTA of 14 warps (one CTA per SM, persistent over units
// (block, 128-row tile, K split)):
//   warp 0      copies of codes (weights and tokens), one elected lane; TMEM
//   warp 1      scale copies to tensor memory and MMAs, one elected lane
//   warp 2      lists of the experts with tokens at start (routed; for up to 256
//               pairs all warps have made the routing lists before, which saves
//               route.cu's launch: 16 tokens over 384 experts 281 -> 268 us, 8 over
//               128 57 -> 55 us, a call among others)
//   warp 3      the units: finds each next one and hands it to the other roles
//               through a ring in shared memory, ahead of them
//   warps 4-7   epilogue: tensor memory -> float32 or bf16 results
//   warps 8-13  scale bytes (8-11 for narrow blocks)
// Two accumulators, so the epilogue of a unit runs beside the next unit's
// MMAs. Every wait is bounded; a role whose wait gives up records it and
// stops, and the CTA waits (bounded) for its own copies and MMAs before
// freeing TMEM.
//
// What bounds it, on one GB300. Few tokens: the weights' bytes (16 tokens over
// 384 experts of 7168 x 4096, 1.71 GB: 273 us, 6.3 TB/s, 94 % of a plain copy;
// 8 tokens over 128 experts of 2880 x 5760, 253 MB: 53 us with lists and
// combine, of which some 8 us are the chain ids -> lists -> units -> first
// copies). Many: dense 8192 x 7168 x 4096 in 98 us, 4.9 PFLOP/s. Parts of it left
// out: copies alone 85 us (40 KB a stage, 1.6 GB from L2 at 18 TB/s), MMAs alone
// 81, MMAs and their scale copies 82, all but the copies of codes 87, all but the
// MMAs 89, all but the stores of results 95, all but the scale copies 98. So reads
// from L2 and the MMAs bound it together, the first a little more, and the scale
// copies hide. (The tensor pipe's counter says 54 % active, 55 us: of the 520 cycles
// that a stage takes with MMAs alone some 170 are not accounted for.) The skewed prefill (8192 tokens, 8 of 384 experts, 7.3 GB of
// weights, rows and float32 results) takes 1.56 ms here, 4.7 TB/s.
// Measured on the way (dense 8192 x 7168 x 4096, other steps then missing): copies
// and MMAs from loops of one thread 114 us, from uniform warps 108 (the operands
// of copies and tcgen05 otherwise have to be made uniform at every issue).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "quant.h"

namespace mxfp4el {
namespace {

constexpr int kThreads = 448;
constexpr int kBM = 128;                       // weight rows per tile
constexpr int kBK = 256;                       // K values per stage
constexpr int kMmaK = 64;                      // K values per MMA
constexpr int kGroupsPerStage = kBK / 32;
constexpr uint32_t kRowBytes = kBK / 2;        // codes of a row per stage
constexpr uint32_t kStageA = kBM * kRowBytes;
constexpr uint32_t kSfBlock = 512;             // 128 rows' scales of four groups
constexpr int kSfPerStage = kGroupsPerStage / 4;
constexpr int kMxNarrow = 32, kMxWide = 192;   // tokens of a block, at most
constexpr uint32_t kTmemCols = 512;
constexpr int kUnitWarp = 3, kScaleWarp0 = 8, kEpiWarp0 = 4, kEpiWarps = 4;
constexpr int kUnitRing = 8;                   // a scale warp looks a few short units ahead
constexpr int kRingMax = 8;                    // stages, at most
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
  // More stages would fit, and do not help: what they leave of the SM's memory
  // caches the scale bytes (8192 x 7168 x 4096: 5 stages 105 us, 4 stages 98).
  static constexpr int kStages = kN == kMxNarrow ? 8 : 4;
  // Scale warps: two teams of one warp for the weights' rows and one for the
  // tokens', or two (128 and 64 rows) when wide.
  static constexpr int kTeams = 2;
  static constexpr int kChunk = 2;               // stages whose scales one read brings
  static constexpr int kTeamWarps = kN == kMxNarrow ? 2 : 3;
  static constexpr int kUnitReaders = 2 + kTeams * kTeamWarps + kEpiWarps;
  static constexpr int kMinStages = (kTeams - 1) * kChunk + 2;
  static_assert(kN == kMxNarrow || kN == kMxWide, "a narrow and a wide form");
  static_assert(kStage % 1024 == 0 && kStageB % 1024 == 0, "stages keep 1024-byte alignment");
};

struct MxMaps {
  CUtensorMap a;      // weights' codes [E][O][I/2], box {128, 128, 1}, 128-byte swizzle
  CUtensorMap b[kMxWide / 32];   // tokens' codes [rows][I/2], boxes {128, 32 (i + 1)}; narrow:
                                 // the first alone, {128, 32}, or {128, 1} (gathered)
};

struct MxKernelArgs {
  RoutePlan plan;               // routed, unless the kernel makes its own lists:
  const void* sel;              // the T * K ids, or null
  int sel64, E;
  const uint8_t* w_scales;      // [E][O][G]
  const uint8_t* x_scales;      // [rows][x_pitch]
  void* out;
  unsigned long long* status;
  int T, O, G, K, x_pitch;
  int mtiles, splits, blocks, stages, max_active;
};

// One unit of work.
struct __align__(16) Unit {
  int e;              // expert (0 when dense); -1: no more units
  int m0;             // first weight row
  int tok0, ntok;     // block: first position (in the lists, or token) and tokens
  int nmma;           // MMA N: ntok rounded up to 16
  int split;
  int kt0, kt1;       // stages of K
  int once;           // this block alone reads the weights
};

// The experts with tokens, in shared memory: id, first position in the lists
// and blocks before, with one entry more of the latter two for the end; behind
// them room for the kernel's own lists.
struct ExpertLists {
  int *blocks, *first, *id, *own;
  __device__ __forceinline__ ExpertLists(void* base, int max_active)
      : blocks(static_cast<int*>(base)), first(blocks + max_active + 1),
        id(first + max_active + 1), own(id + max_active) {}
};
constexpr size_t list_bytes(int max_active, int own_pairs) {
  return (3 * (size_t)max_active + 2 + 3 * (size_t)own_pairs) * sizeof(int);
}

template <int kRows>
struct __align__(16) MxShared {
  uint64_t full[kRingMax], empty[kRingMax];
  uint64_t d_full[2], d_empty[2];
  uint64_t u_full[kUnitRing], u_empty[kUnitRing];
  uint64_t drain;
  uint32_t tmem_base;
  int num_units, num_active;
  Unit units[kUnitRing];
  int rows[kUnitRing][kRows];   // token of each row of the block (gathered)
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

template <int kN, bool kRouted>
__device__ __forceinline__ Unit unit_at(const MxKernelArgs& a, const ExpertLists& ex,
                                        int num_active, int idx) {
  Unit w;
  const int per_block = a.mtiles * a.splits;
  int first = 0, nblk, cnt, local;
  if constexpr (kRouted) {
    const int blk = idx / per_block;
    int lo = 0, hi = num_active;           // blocks[lo] <= blk < blocks[lo + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ex.blocks[mid] <= blk) lo = mid;
      else hi = mid;
    }
    w.e = ex.id[lo];
    first = ex.first[lo];
    cnt = ex.first[lo + 1] - first;
    nblk = ex.blocks[lo + 1] - ex.blocks[lo];
    local = idx - ex.blocks[lo] * per_block;
  } else {
    w.e = 0;
    cnt = a.T;
    nblk = a.blocks;
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
  w.once = nblk == 1;
  return w;
}

// The scales of kChunk stages from any address: aligned words and one more while
// they are on their way (load), then the words themselves (settle). Reads only
// aligned words that hold one of the row's bytes, `left` from p on; bytes past
// them are 0. wide: p is 16-byte aligned, as the row's end is.
template <int kChunk>
struct RawScales {
  static constexpr int kWords = 2 * kChunk;
  uint32_t v[kWords + 1];
  uint32_t shift;
  __device__ __forceinline__ void load(const uint8_t* p, int left, bool wide) {
    if (wide) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (i == 0 || left > 4 * i) u = *reinterpret_cast<const uint4*>(p + 4 * i);
        v[i] = u.x; v[i + 1] = u.y; v[i + 2] = u.z; v[i + 3] = u.w;
      }
    } else {
      const int skip = (int)(reinterpret_cast<uintptr_t>(p) & 3);
      const uint32_t* at = reinterpret_cast<const uint32_t*>(p - skip);
#pragma unroll
      for (int i = 0; i <= kWords; ++i) v[i] = 4 * i < left + skip ? at[i] : 0u;
      shift = 8u * (uint32_t)skip;
    }
  }
  __device__ __forceinline__ void settle(int left) {     // not after a wide load
#pragma unroll
    for (int i = 0; i < kWords; ++i) v[i] = __funnelshift_r(v[i], v[i + 1], shift);
    if (left < 4 * kWords) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int n = left - 4 * i;
        if (n < 4) v[i] = n > 0 ? v[i] & ((1u << (8 * n)) - 1u) : 0u;
      }
    }
  }
};

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A warp's wait. The first test alone is inline: a stage of the copies and
// MMAs is a few hundred cycles, of which loops and clock reads took a third.
__device__ __noinline__ bool wait_longer(uint64_t* bar, uint32_t parity) {
  return __all_sync(kFullMask, mbar_wait_suspend(bar, parity)) != 0;
}
__device__ __forceinline__ bool wait_short(uint64_t* bar, uint32_t parity) {
  if (__all_sync(kFullMask, mbar_try_wait(bar, parity))) return true;
  return wait_longer(bar, parity);
}

// The next unit of this role; its fields are the same in every lane, and known
// to be (values that feed the copies and tcgen05 otherwise have to be made
// uniform at every issue).
template <int kRows>
__device__ __forceinline__ bool pop_unit(MxShared<kRows>& sh, RingPos& pu, Unit* w) {
  if (!wait_short(&sh.u_full[pu.idx], pu.phase)) return false;
  const Unit u = sh.units[pu.idx];
  w->e = __shfl_sync(kFullMask, u.e, 0);
  w->m0 = __shfl_sync(kFullMask, u.m0, 0);
  w->tok0 = __shfl_sync(kFullMask, u.tok0, 0);
  w->ntok = __shfl_sync(kFullMask, u.ntok, 0);
  w->nmma = __shfl_sync(kFullMask, u.nmma, 0);
  w->split = __shfl_sync(kFullMask, u.split, 0);
  w->kt0 = __shfl_sync(kFullMask, u.kt0, 0);
  w->kt1 = __shfl_sync(kFullMask, u.kt1, 0);
  w->once = __shfl_sync(kFullMask, u.once, 0);
  return true;
}
template <int kRows>
__device__ __forceinline__ void release_unit(MxShared<kRows>& sh, RingPos& pu) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.u_empty[pu.idx]);
  pu.next(kUnitRing);
}

// Stages kChunk at a time, in the order of the units, dealt to kTeams teams in
// turn: next() moves to this team's next ones. Lane l has the rows row0 + l + 32 i
// of the tile (kTokens: of the block), i < kRows.
template <int kRows, int kTeams, int kChunk, bool kTokens, bool kGather>
struct ScaleWalk {
  Unit w;
  int kt;                 // first of the stages
  int slot;               // its place in the ring of stages
  uint32_t phase;
  int turn;               // whose turn it is
  bool wide;              // every row on 16-byte boundaries
  const uint8_t* base[kRows];
  RingPos pu;

  __device__ __forceinline__ void start() {
    w.e = 0;
    w.kt1 = kt = -kChunk;                      // nothing yet: the first step loads a unit
    slot = 0;
    phase = 0;
    turn = kTeams - 1;
  }
  template <typename Sh>
  __device__ __forceinline__ bool load_unit(const MxKernelArgs& a, Sh& sh, int row0, int lane) {
    if (!pop_unit(sh, pu, &w)) {
      w.e = -2;
      return false;
    }
    if (w.e >= 0) {
      const uint8_t* from = kTokens ? a.x_scales : a.w_scales;
      const int pitch = kTokens ? a.x_pitch : a.G;
      wide = (reinterpret_cast<uintptr_t>(from) | (uintptr_t)pitch | (uintptr_t)(8 * w.kt0)) % 16 == 0 &&
             a.G % 16 == 0;
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if constexpr (kTokens) {
          const int n = min(row0 + lane + 32 * i, w.ntok - 1);
          const int t = kGather ? sh.rows[pu.idx][n] : w.tok0 + n;
          base[i] = from + (size_t)t * pitch;
        } else {
          base[i] = from + ((size_t)w.e * a.O + min(w.m0 + lane + 32 * i, a.O - 1)) * pitch;
        }
      }
    }
    release_unit(sh, pu);
    return true;
  }
  // False at the end of the units (or after a wait that gave up: w.e == -2).
  template <typename Sh>
  __device__ __forceinline__ bool next(const MxKernelArgs& a, Sh& sh, int team, int row0,
                                       int lane) {
    for (;;) {
      slot += min(kChunk, w.kt1 - kt);
      while (slot >= a.stages) {
        slot -= a.stages;
        phase ^= 1u;
      }
      kt += kChunk;
      while (kt >= w.kt1) {
        if (!load_unit(a, sh, row0, lane) || w.e < 0) return false;
        kt = w.kt0;
      }
      turn = turn + 1 == kTeams ? 0 : turn + 1;
      if (turn == team) return true;
    }
  }
};

// A scale warp's whole work. block0: the offset of its first block in a stage,
// kStride that of the next four groups' block. False after a wait that gave up.
template <int kRows, int kTeams, int kChunk, bool kTokens, bool kGather, uint32_t kStageBytes,
          uint32_t kStride, typename Sh>
__device__ __forceinline__ bool scale_role(const MxKernelArgs& a, Sh& sh, unsigned char* ring,
                                           uint32_t block0, int team, int row0, int lane) {
  ScaleWalk<kRows, kTeams, kChunk, kTokens, kGather> walk;
  walk.start();
  RawScales<kChunk> cur[kRows], nxt[kRows];
  auto fetch = [&](RawScales<kChunk> (&v)[kRows]) {
    const int at = walk.kt * kGroupsPerStage;
#pragma unroll
    for (int i = 0; i < kRows; ++i) v[i].load(walk.base[i] + at, a.G - at, walk.wide);
  };
  bool more = walk.next(a, sh, team, row0, lane);
  if (more) fetch(cur);
  while (more) {
    int slot = walk.slot;
    uint32_t phase = walk.phase;
    const int n = min(kChunk, walk.w.kt1 - walk.kt);
    const int left = a.G - walk.kt * kGroupsPerStage;
    const bool settled = walk.wide;
    more = walk.next(a, sh, team, row0, lane);
    if (more) fetch(nxt);
    if (!settled) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) cur[i].settle(left);
    }
#pragma unroll
    for (int j = 0; j < kChunk; ++j) {
      if (j >= n) break;
      if (!wait_short(&sh.empty[slot], phase ^ 1u)) return false;
      unsigned char* sf = ring + (size_t)slot * kStageBytes + block0 + lane * 16;
#pragma unroll
      for (int b = 0; b < kSfPerStage; ++b) {
        uint32_t w[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i) w[i] = cur[i].v[kSfPerStage * j + b];
        unsigned char* at = sf + b * kStride;
        if constexpr (kRows == 4)
          *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kRows == 2)
          *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(at) = w[0];
      }
      // The MMA warp has the fence between these stores and the tensor core.
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.full[slot]);
      if (++slot == a.stages) {
        slot = 0;
        phase ^= 1u;
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) cur[i] = nxt[i];
  }
  return walk.w.e != -2;
}

// The lists of route.cu for up to kMxOwnPairs pairs, by one block, a thread per
// pair: its place is the number of pairs before it by (expert, pair). Ids out
// of range are left out (and counted by block 0). Returns the experts' number;
// ex.own: the pairs in the lists' order, then scratch.
__device__ __forceinline__ int own_lists(const MxKernelArgs& a, const ExpertLists& ex, int P) {
  static_assert(kMxOwnPairs <= kThreads, "a thread per pair");
  int *list = ex.own, *key = list + P, *head = key + P;
  const int i = (int)threadIdx.x;
  long long e = -1;
  if (i < P)
    e = a.sel64 ? (long long)static_cast<const int64_t*>(a.sel)[i]
                : (long long)static_cast<const int32_t*>(a.sel)[i];
  const bool valid = e >= 0 && e < a.E;
  const int k = valid ? (int)e : 0x7fffffff;           // beyond every id
  if (i < P) key[i] = k;
  const int total = __syncthreads_count(valid);
  int less = 0, before = 0;
  if (valid) {
    for (int j = 0; j < P; ++j) {
      const int other = key[j];
      less += other < k;
      before += other == k && j < i;
    }
    list[less + before] = i;
  }
  const bool first = valid && before == 0;
  if (i < P) head[i] = first;
  const int experts = __syncthreads_count(first);
  if (first) {
    int u = 0;
    for (int j = 0; j < P; ++j) u += head[j] && key[j] < k;
    ex.id[u] = k;
    ex.first[u] = less;
  }
  if (i == 0) {
    ex.first[experts] = total;
    if (blockIdx.x == 0 && total < P)
      atomicAdd(&a.status[kStatusBadPairs], (unsigned long long)(P - total));
  }
  __syncthreads();
  return experts;
}

template <int kN, typename Out, bool kRouted>
__global__ void __launch_bounds__(kThreads, 1)
gemm_mx_kernel(const __grid_constant__ MxMaps maps, const MxKernelArgs a) {
  using S = Shape<kN>;
  constexpr bool kGather = kRouted && kN == kMxNarrow;
  using Shared = MxShared<kGather ? kN : 1>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  Shared& sh = *reinterpret_cast<Shared*>(ring + (size_t)a.stages * S::kStage);
  const ExpertLists ex(&sh + 1, a.max_active);

  const int warp = __shfl_sync(kFullMask, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(&sh.full[s], 1 + S::kTeamWarps);       // the copies (bytes), a team's warps
      mbar_init(&sh.empty[s], 1);                      // the MMAs
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.d_full[b], 1);
      mbar_init(&sh.d_empty[b], kEpiWarps);
    }
    for (int r = 0; r < kUnitRing; ++r) {
      mbar_init(&sh.u_full[r], 1);
      mbar_init(&sh.u_empty[r], S::kUnitReaders);
    }
    mbar_init(&sh.drain, 32);                          // every lane of the MMA warp
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sh.tmem_base, kTmemCols);
    tmem_relinquish();
    if (lane == 0) {
      prefetch_tensor_map(&maps.a);
      prefetch_tensor_map(&maps.b[0]);
    }
  }
  pdl_wait();                    // the operands and the routing lists are ready
  const bool own = kGather && a.sel != nullptr;
  int own_experts = 0;
  if constexpr (kGather) {
    __syncwarp();
    if (own) own_experts = own_lists(a, ex, a.T * a.K);
  }
  const int* pairs_by_expert = own ? ex.own : a.plan.pair_list;
  if (warp == 2) {
    if constexpr (kRouted) {
      const int na = own ? own_experts : a.plan.meta[kMetaNumActive];
      int run = 0;
      for (int base = 0; base < na; base += 32) {
        const int u = base + lane;
        int nb = 0;
        if (u < na) {
          int beg, end;
          if (own) {
            beg = ex.first[u];
            end = ex.first[u + 1];
          } else {
            const int e = a.plan.active[u];
            beg = a.plan.offsets[e];
            end = a.plan.offsets[e + 1];
            ex.id[u] = e;
            ex.first[u] = beg;
            if (u == na - 1) ex.first[na] = end;     // the lists have no gaps
          }
          nb = (end - beg + kN - 1) / kN;
        }
        int incl = nb;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int v = __shfl_up_sync(kFullMask, incl, off);
          if (lane >= off) incl += v;
        }
        if (u < na) ex.blocks[u] = run + incl - nb;
        run += __shfl_sync(kFullMask, incl, 31);
      }
      if (lane == 0) {
        ex.blocks[na] = run;
        sh.num_active = na;
        sh.num_units = run * a.mtiles * a.splits;
      }
    } else if (lane == 0) {
      sh.num_active = 0;
      sh.num_units = a.blocks * a.mtiles * a.splits;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(kFullMask, sh.tmem_base, 0);
  const uint32_t ring_addr = __shfl_sync(kFullMask, smem_addr(ring), 0);
  bool ok = true;

  if (warp == kUnitWarp) {
    // ------------------------------------------------------------ the units
    const int num_units = sh.num_units, num_active = sh.num_active;
    RingPos pu;
    for (int idx = blockIdx.x;; idx += gridDim.x) {
      Unit w;
      w.e = -1;
      if (idx < num_units) w = unit_at<kN, kRouted>(a, ex, num_active, idx);
      if (w.e >= 0 && w.ntok <= 0) continue;
      int t = 0;
      if (kGather && w.e >= 0)                  // past the block its last token
        t = pairs_by_expert[w.tok0 + min(lane, w.ntok - 1)] / a.K;
      if (!wait_short(&sh.u_empty[pu.idx], pu.phase ^ 1u)) {
        ok = false;
        break;
      }
      if (kGather) sh.rows[pu.idx][lane] = t;
      // The tile's scale bytes lie together: have them in L2 by the time the
      // scale warps ask, which they do only a few stages ahead.
      if (lane == 0 && w.e >= 0) {
        const uint8_t* from = a.w_scales + ((size_t)w.e * a.O + w.m0) * a.G;
        const uintptr_t lo = (reinterpret_cast<uintptr_t>(from) + 15) & ~(uintptr_t)15;
        const uintptr_t hi =
            reinterpret_cast<uintptr_t>(from + (size_t)min(kBM, a.O - w.m0) * a.G) & ~(uintptr_t)15;
        if (hi > lo)                                   // 64 KB: rows of 16384 values
          prefetch_l2(reinterpret_cast<const void*>(lo),
                      (uint32_t)min(hi - lo, (uintptr_t)65536));
      }
      if (lane == 0) sh.units[pu.idx] = w;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.u_full[pu.idx]);
      pu.next(kUnitRing);
      if (w.e < 0) break;
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
  } else if (warp == 0) {
    // ------------------------------------------------------ copies of codes
    const uint64_t pol_once = l2_evict_first_policy(), pol_keep = l2_evict_last_policy();
    const uint64_t pol_reuse = l2_evict_normal_policy();
    RingPos pos, pu;
    int issued = 0;
    Unit w;
    while (ok) {
      if (!pop_unit(sh, pu, &w)) {
        ok = false;
        break;
      }
      // Weights that one block reads pass through L2 once.
      const uint64_t pol = w.once ? pol_once : pol_reuse;
      const int load = (w.nmma + 31) / 32 - 1;           // the token box: 32 (load + 1) rows
      const uint32_t box = kGather ? (uint32_t)w.nmma : 32u * (uint32_t)(load + 1);
      int4 rows[kGather ? kN / 4 : 1];
      if constexpr (kGather) {
        const int t = sh.rows[pu.idx][lane];
#pragma unroll
        for (int q = 0; q < kN / 4; ++q)
          rows[q] = make_int4(__shfl_sync(kFullMask, t, 4 * q), __shfl_sync(kFullMask, t, 4 * q + 1),
                              __shfl_sync(kFullMask, t, 4 * q + 2),
                              __shfl_sync(kFullMask, t, 4 * q + 3));
      }
      release_unit(sh, pu);
      if (w.e < 0) break;
      for (int kt = w.kt0; kt < w.kt1; ++kt, ++issued) {
        if (!wait_short(&sh.empty[pos.idx], pos.phase ^ 1u)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          unsigned char* stage = ring + (size_t)pos.idx * S::kStage;
          uint64_t* bar = &sh.full[pos.idx];
          const int x = kt * (int)kRowBytes;
          mbar_arrive_expect_tx(bar, kStageA + box * kRowBytes);
          tma_load_3d(stage, &maps.a, x, w.m0, w.e, bar, pol);
          if constexpr (kGather) {
#pragma unroll
            for (int q = 0; q < kN / 4; ++q)
              if (4 * q < w.nmma)
                tma_gather4(stage + kStageA + q * 4 * kRowBytes, &maps.b[0], x, rows[q], bar,
                            pol_keep);
          } else {
            tma_load_2d(stage + kStageA, &maps.b[load], x, w.tok0, bar, pol_keep);
          }
        }
        __syncwarp();
        pos.next(a.stages);
      }
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
    // Wait (bounded) until the copies have landed: the last min(issued,
    // stages) uses of the ring.
    for (int k = 0; k < min(issued, a.stages); ++k) {
      int idx = pos.idx - 1 - k;
      uint32_t ph = pos.phase;
      if (idx < 0) { idx += a.stages; ph ^= 1u; }
      if (!wait_short(&sh.full[idx], ph)) break;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA
    RingPos pos, pu;
    Unit w;
    const uint64_t da0 = smem_desc_sw128(ring_addr);
    const uint64_t dsf0 = smem_desc_rows16(ring_addr + kStageA + S::kStageB);
    for (int it = 0; ok; ++it) {
      if (!pop_unit(sh, pu, &w)) {
        ok = false;
        break;
      }
      release_unit(sh, pu);
      if (w.e < 0) break;
      const int buf = it & 1;
      if (!wait_short(&sh.d_empty[buf], ((uint32_t)(it >> 1) & 1u) ^ 1u)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t d = tmem + buf * kN;
      const uint32_t idesc0 = mma_idesc(w.nmma, 0), idesc2 = mma_idesc(w.nmma, 2);
      // MMAs of the last stage: K may end in it.
      const int last = min(kBK / kMmaK, (a.G * 32 - (w.kt1 - 1) * kBK + kMmaK - 1) / kMmaK);
      const bool second = S::kBRowBlocks > 1 && w.nmma > 128;   // token scales' second block
      bool ready = mbar_try_wait(&sh.full[pos.idx], pos.phase);
      for (int kt = w.kt0; kt < w.kt1; ++kt) {
        if (!__all_sync(kFullMask, ready) && !wait_longer(&sh.full[pos.idx], pos.phase)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const int idx = pos.idx;
        pos.next(a.stages);
        // The next stage's state is asked for before this one's MMAs are issued.
        ready = kt + 1 < w.kt1 && mbar_try_wait(&sh.full[pos.idx], pos.phase);
        if (elect_one()) {
          fence_proxy_async_smem();              // the scale warps' stores
          // Descriptors differ in the address alone (16-byte units in the low bits).
          const uint32_t at = (uint32_t)idx * (S::kStage >> 4);
          const uint64_t da = da0 + at, db = da + (kStageA >> 4), dsf = dsf0 + at;
          const uint32_t tsfa = tmem + S::kSfCol + idx * (S::kSfColsA + S::kSfColsB);
          const uint32_t tsfb = tsfa + S::kSfColsA;
#pragma unroll
          for (int b = 0; b < kSfPerStage; ++b) {
            tc_copy_scales(tsfa + 4 * b, dsf + b * (kSfBlock >> 4));
#pragma unroll
            for (int r = 0; r < S::kBRowBlocks; ++r)
              if (r == 0 || second) tc_copy_scales(tsfb + 4 * (b * S::kBRowBlocks + r),
                             dsf + ((S::kSfA + (b * S::kBRowBlocks + r) * kSfBlock) >> 4));
          }
          const bool end = kt == w.kt1 - 1;
          tc_mma_mxf4(d, da, db, idesc0, tsfa, tsfb, kt > w.kt0 ? 1u : 0u);
#pragma unroll
          for (int j = 1; j < kBK / kMmaK; ++j)
            if (!end || j < last)
              tc_mma_mxf4(d, da + j * 2, db + j * 2, (j & 1) ? idesc2 : idesc0,
                          tsfa + 4 * (j / 2), tsfb + 4 * (j / 2) * S::kBRowBlocks, 1u);
          tc_commit(&sh.empty[idx]);
          if (end) tc_commit(&sh.d_full[buf]);
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
    tc_commit(&sh.drain);                          // every lane: any may have been elected
    mbar_wait(&sh.drain, 0);
    __syncwarp();
  } else if (warp >= kScaleWarp0) {
    // ---------------------------------------------------------- scale bytes
    constexpr uint32_t kBlocks = kStageA + S::kStageB, kTokenBlocks = kBlocks + S::kSfA;
    constexpr uint32_t kStrideB = S::kBRowBlocks * kSfBlock;
    const int me = warp - kScaleWarp0, team = me / S::kTeamWarps;
    if (team < S::kTeams) {
      if (me % S::kTeamWarps == 0)
        ok = scale_role<4, S::kTeams, S::kChunk, false, kGather, S::kStage, kSfBlock>(a, sh, ring, kBlocks,
                                                                         team, 0, lane);
      else if constexpr (kN == kMxNarrow)
        ok = scale_role<1, S::kTeams, S::kChunk, true, kGather, S::kStage, kStrideB>(a, sh, ring, kTokenBlocks,
                                                                        team, 0, lane);
      else if (me % S::kTeamWarps == 1)
        ok = scale_role<4, S::kTeams, S::kChunk, true, kGather, S::kStage, kStrideB>(a, sh, ring, kTokenBlocks,
                                                                        team, 0, lane);
      else
        ok = scale_role<2, S::kTeams, S::kChunk, true, kGather, S::kStage, kStrideB>(
            a, sh, ring, kTokenBlocks + kSfBlock, team, 128, lane);
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------- epilogue
    const int quarter = warp - kEpiWarp0;
    Out* out = static_cast<Out*>(a.out);
    const bool pairs = a.O % 2 == 0 && reinterpret_cast<uintptr_t>(a.out) % 4 == 0;
    RingPos pu;
    Unit w;
    for (int it = 0;; ++it) {
      if (!pop_unit(sh, pu, &w)) {
        ok = false;
        break;
      }
      release_unit(sh, pu);
      if (w.e < 0) break;
      const int buf = it & 1;
      if (!wait_short(&sh.d_full[buf], (uint32_t)(it >> 1) & 1u)) { ok = false; break; }
      tc_fence_after_sync();
      const int o = w.m0 + quarter * 32 + lane;
      for (int c0 = 0; c0 < w.ntok; c0 += 32) {
        const int n = min(32, w.ntok - c0);
        int row = w.tok0 + c0 + min(lane, n - 1);
        if constexpr (kRouted) row = pairs_by_expert[row];
        float v[32];
        tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * kN + c0, v);
        tmem_wait_ld();
        if (c0 + 32 >= w.ntok) {                 // the accumulator may be written again
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.d_empty[buf]);
        }
        if constexpr (sizeof(Out) == 2) {        // bf16 is dense and unsplit
          Out* to = out + (int64_t)(w.tok0 + c0) * a.O;
          if (pairs) {
            // Neighbouring lanes share out two columns, so that each stores two rows.
            const bool odd = (lane & 1) != 0;
            to += (odd ? a.O : 0) + (o & ~1);
#pragma unroll
            for (int c = 0; c < 32; c += 2, to += 2 * (int64_t)a.O) {
              const float other = __shfl_xor_sync(kFullMask, odd ? v[c] : v[c + 1], 1);
              const __nv_bfloat162 two = odd ? __floats2bfloat162_rn(other, v[c + 1])
                                             : __floats2bfloat162_rn(v[c], other);
              if (c + (odd ? 1 : 0) < n && o < a.O)
                *reinterpret_cast<__nv_bfloat162*>(to) = two;
            }
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c, to += a.O)
              if (c < n && o < a.O) store_out(to + o, v[c]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int r = __shfl_sync(kFullMask, row, c);
            if (c < n && o < a.O)
              store_out(out + ((int64_t)r * a.splits + w.split) * a.O + o, v[c]);
          }
        }
      }
    }
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

// The token rows of a wide routed call in the lists' order, scale rows on
// 16-byte boundaries; one warp per row.
__global__ void __launch_bounds__(256)
group_rows_kernel(const uint8_t* __restrict__ packed, const uint8_t* __restrict__ scales,
                  RoutePlan plan, int G, int K, int pitch, int64_t max_rows,
                  uint8_t* __restrict__ packed_out, uint8_t* __restrict__ scales_out) {
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t rows = min((int64_t)plan.meta[kMetaNumPairs], max_rows);
  for (int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); r < rows;
       r += (int64_t)gridDim.x * 8) {
    const int64_t t = plan.pair_list[r] / K;
    const uint4* src = reinterpret_cast<const uint4*>(packed) + t * G;
    uint4* dst = reinterpret_cast<uint4*>(packed_out) + r * G;
    for (int i = lane; i < G; i += 32) dst[i] = src[i];
    for (int i = lane; i < pitch; i += 32)
      scales_out[r * pitch + i] = i < G ? scales[t * G + i] : (uint8_t)0;
  }
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
size_t smem_bytes(int stages, int max_active, int own_pairs) {
  return 1024 + (size_t)stages * Shape<kN>::kStage + sizeof(MxShared<kMxNarrow>) +
         list_bytes(max_active, own_pairs);
}

template <int kN>
int stages_for(int max_active, int own_pairs) {
  int s = std::min(Shape<kN>::kStages, Shape<kN>::kTmemStages);
  while (s > 0 && smem_bytes<kN>(s, max_active, own_pairs) > kSmemLimit) --s;
  return s;
}

template <int kN, typename Out, bool kRouted>
cudaError_t launch_typed(const MxMaps& maps, MxKernelArgs args, int64_t units,
                         cudaStream_t stream) {
  const int own_pairs = args.sel != nullptr ? args.T * args.K : 0;
  args.stages = stages_for<kN>(args.max_active, own_pairs);
  if (args.stages < Shape<kN>::kMinStages) return cudaErrorInvalidValue;
  const size_t smem = smem_bytes<kN>(args.stages, args.max_active, own_pairs);
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
  return launch_after_previous(gemm_mx_kernel<kN, Out, kRouted>,
                               dim3((unsigned)std::min<int64_t>(units, num_sms())), dim3(kThreads),
                               smem, stream, maps, args);
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

namespace {

// What units of this shape take, in ns. A round of units takes every SM one unit:
// its stages, each the longer the wider the copies (boxes of 32 tokens), and its
// start and epilogue. With K split results are written and read in float32 for
// every split, by one launch more when dense, by the combine when routed. Fitted to
// 1 to 8192 tokens over weights of 1056 x 1001 to 7168 x 16384 (a round of 28 stages
// takes 6.8 us in narrow units, 8.8 at 128 tokens, 9.4 at 192).
int64_t plan_cost(int64_t blocks, int64_t width, int64_t mtiles, int64_t nk, int64_t splits,
                  int64_t results, bool routed) {
  const int64_t rounds = (blocks * mtiles * splits + 151) / 152;
  const int64_t stage = 210 + (width + 31) / 32 * 32 / 2;
  int64_t cost = rounds * ((nk + splits - 1) / splits * stage + 700);
  if (splits > 1) cost += routed ? results * splits / 200 : 2200 + results * splits / 300;
  return cost;
}

int64_t scale_pitch(int64_t I) { return (I / 32 + 15) / 16 * 16; }

}  // namespace

MxPlan gemm_mx_plan(int64_t T, int64_t E, int64_t I, int64_t O, int64_t K, bool routed) {
  const int64_t mtiles = (O + kBM - 1) / kBM, nk = (I + kBK - 1) / kBK;
  const int64_t most_splits = std::max<int64_t>(1, std::min<int64_t>(nk / 2, 8));
  MxPlan best = {false, 1, 1, 0, 0, false};
  int64_t least = INT64_MAX;
  // Splits are for calls of few units.
  auto splits_for = [&](int64_t units) { return units > 4 * 152 ? 1 : most_splits; };
  if (routed) {
    // Wide blocks where experts average as many tokens as half a narrow block holds:
    // 12 and 16 tokens each on 32 experts of 2880 x 2880 take 38 and 42 us narrow, 40
    // and 42 wide; by Zipf's law (exponent 1.2) over 384 experts of 2880 x 2048, 8
    // picks, 254 and 287 us narrow, 256 and 274 wide. Not up to 128 pairs, since lists
    // and grouped rows are two launches more (4 experts of 4096 x 1024, 64 and 128
    // pairs: narrow 11 and 14 us, wide 15 and 16; 8 experts, 192 and 256 pairs 17 and
    // 20 narrow, 17 and 18 wide), nor for up to 32 tokens, where no block is wider.
    const int64_t active = std::min(E, T * K);
    best.wide = T > kMxNarrow && T * K > 128 && T * K >= 16 * active;
    const int64_t n = best.wide ? kMxWide : kMxNarrow;
    // Each expert's last block may be short.
    best.blocks = active + T * K / n;
    // The cost is that of the blocks to be expected: half of an expert's last one.
    const int64_t blocks = std::max(active, (active + 1) / 2 + (T * K + n - 1) / n);
    const int64_t width = (T * K + blocks - 1) / blocks;
    for (int64_t s = 1; s <= splits_for(blocks * mtiles); ++s) {
      const int64_t cost = plan_cost(blocks, width, mtiles, nk, s, T * K * O, true);
      if (cost < least) {
        least = cost;
        best.splits = (int)s;
      }
    }
    best.own_lists = !best.wide && T * K <= kMxOwnPairs;
    if (best.wide) best.grouped_bytes = (size_t)T * K * (size_t)(I / 2 + scale_pitch(I));
  } else {
    // Up to 512 tokens either form, unsplit narrow / wide in us: 2880 x 5760, 64 tokens
    // 7.4 / 7.6, 128 10.4 / 8.1, 512 20 / 9.9; 4096 x 512, 512 tokens 8.0 / 9.4.
    // Splits pay for few tokens and long sums alone: 1 token of 7168 x 4096 10.5 us in
    // one piece, 8.6 in four; 64 tokens 10.7 and 12.1.
    for (int wide = T <= 512 ? 0 : 1; wide < 2; ++wide) {
      const int64_t n = wide ? kMxWide : kMxNarrow, few = (T + n - 1) / n;
      // More blocks than needed may fill whole rounds of the SMs better.
      for (int64_t b = few; b <= few + std::min<int64_t>(few / 4 + 1, 12); ++b) {
        const int64_t width = ((T + b - 1) / b + 15) / 16 * 16;
        const int64_t blocks = (T + width - 1) / width;   // equal ones, multiples of 16 tokens
        for (int64_t s = 1; s <= splits_for(blocks * mtiles); ++s) {
          const int64_t cost = plan_cost(blocks, width, mtiles, nk, s, T * O, false);
          if (cost < least) {
            least = cost;
            best.wide = wide != 0;
            best.splits = (int)s;
            best.blocks = blocks;
          }
        }
      }
    }
  }
  best.units = best.blocks * mtiles * best.splits;
  return best;
}

cudaError_t launch_gemm_mx(const MxGemm& g, cudaStream_t stream) {
  const bool routed = g.plan != nullptr || g.shape.own_lists;
  const MxPlan& plan = g.shape;
  const bool wide = plan.wide, grouped = routed && wide;
  const int64_t G = g.I / 32, P = g.T * g.K;
  const uint8_t *rows = g.x_packed, *scales = g.x_scales;
  int64_t nrows = g.T, pitch = G;
  if (grouped) {
    nrows = P;
    pitch = scale_pitch(g.I);
    uint8_t* rows_out = static_cast<uint8_t*>(g.grouped);
    uint8_t* scales_out = rows_out + (size_t)P * (size_t)(g.I / 2);
    const unsigned blocks = (unsigned)std::min<int64_t>((P + 7) / 8, (int64_t)num_sms() * 8);
    const cudaError_t err = launch_after_previous(
        group_rows_kernel, dim3(blocks), dim3(256), 0, stream, g.x_packed, g.x_scales, *g.plan,
        (int)G, (int)g.K, (int)pitch, P, rows_out, scales_out);
    if (err != cudaSuccess) return err;
    rows = rows_out;
    scales = scales_out;
  }
  MxMaps maps;
  std::memset(&maps, 0, sizeof(maps));
  const cuuint64_t row = (cuuint64_t)(g.I / 2);
  {
    const cuuint64_t dims[3] = {row, (cuuint64_t)g.O, (cuuint64_t)g.E};
    const cuuint64_t strides[2] = {row, row * (cuuint64_t)g.O};
    const cuuint32_t box[3] = {kRowBytes, kBM, 1};
    if (!encode(&maps.a, g.w_packed, 3, dims, strides, box)) return cudaErrorInvalidValue;
  }
  {
    const cuuint64_t dims[2] = {row, (cuuint64_t)nrows};
    const cuuint64_t strides[1] = {row};
    const bool gather = routed && !grouped;
    for (int i = 0; i < (wide ? kMxWide / 32 : 1); ++i) {
      const cuuint32_t box[2] = {kRowBytes, gather ? 1u : 32u * (unsigned)(i + 1)};
      if (!encode(&maps.b[i], rows, 2, dims, strides, box)) return cudaErrorInvalidValue;
    }
  }
  MxKernelArgs a;
  std::memset(static_cast<void*>(&a), 0, sizeof(a));
  if (plan.own_lists) {
    a.sel = g.sel;
    a.sel64 = g.sel64 ? 1 : 0;
    a.E = (int)g.E;
  } else if (routed) {
    a.plan = *g.plan;
  }
  a.w_scales = g.w_scales;
  a.x_scales = scales;
  a.x_pitch = (int)pitch;
  a.out = plan.splits > 1 || routed ? static_cast<void*>(g.part) : g.out;
  a.status = device_status_words();
  if (a.status == nullptr) return cudaErrorUnknown;
  a.T = (int)g.T;
  a.O = (int)g.O;
  a.G = (int)G;
  a.K = (int)g.K;
  a.mtiles = (int)((g.O + kBM - 1) / kBM);
  a.splits = plan.splits;
  a.blocks = (int)plan.blocks;
  a.max_active = routed ? (int)std::min(g.E, P) : 0;
  cudaError_t err;
  if (routed)
    err = wide ? launch_typed<kMxWide, float, true>(maps, a, plan.units, stream)
               : launch_typed<kMxNarrow, float, true>(maps, a, plan.units, stream);
  else if (plan.splits > 1 || g.out_dtype == kTokenF32)
    err = wide ? launch_typed<kMxWide, float, false>(maps, a, plan.units, stream)
               : launch_typed<kMxNarrow, float, false>(maps, a, plan.units, stream);
  else
    err = wide ? launch_typed<kMxWide, __nv_bfloat16, false>(maps, a, plan.units, stream)
               : launch_typed<kMxNarrow, __nv_bfloat16, false>(maps, a, plan.units, stream);
  if (err != cudaSuccess || routed || plan.splits == 1) return err;
  const unsigned grid = (unsigned)std::min<int64_t>((g.T * g.O + 255) / 256, num_sms() * 8);
  if (g.out_dtype == kTokenF32)
    return launch_after_previous(join_splits_kernel<float>, dim3(grid), dim3(256), 0, stream,
                                 static_cast<const float*>(g.part), plan.splits, g.T, g.O,
                                 static_cast<float*>(g.out));
  return launch_after_previous(join_splits_kernel<__nv_bfloat16>, dim3(grid), dim3(256), 0, stream,
                               static_cast<const float*>(g.part), plan.splits, g.T, g.O,
                               static_cast<__nv_bfloat16*>(g.out));
}

}  // namespace mxfp4el

// attn_prefill.cu -- attention of prompts (or chunks behind a history) over
// the paged cache on the tensor cores: tcgen05, tensor memory and tensor
// copies. bf16 tokens.
//
// Rows. The query heads of one key head share its keys: a tile's 128 rows are
// n = 128 / heads tokens times those heads (row i: token i / heads, head
// i % heads), so a key or value is read once for all of them, short prompts
// and short windows still fill tiles, and the causal edge cuts few of a
// tile's scores. A unit of work is two such tiles (2 n tokens) of one key
// head over every key that a row of it sees, in key tiles of 128:
//
//   S = Q K^T            two tiles' worth, into tensor memory (float32)
//   P = 2^(c S - c m)    m: running row maximum, c = scale log2 e; bf16
//   O += P V             P from tensor memory, V from shared memory
//   l += sum P           out = O / l
//
// Bound: tensor throughput, 4 D operations per row and key, as long as the
// powers keep up: the two tiles take turns, one in the tensor pipe while the
// other's softmax runs. A prompt of 8192 tokens, 64 query and 8 key heads of
// 128, in calls one after another: 743 us, 1.48 PFLOP/s of unmasked work, the
// tensor pipe busy 68 % of the cycles (1.95 GHz, 1.37 kW); the same with
// softmax warps that only pass the tiles on: 641 us. Short units (a window of
// 128) are bound by the chain of their steps: 40 us for 4096 tokens, heads of
// 64.
//
// Warps of a CTA (one CTA per SM, units from a counter, the longest first):
//   0-7, 8-15 softmax and epilogue of row tile 0 and of row tile 1: two
//             threads per row, half of the keys each, which exchange maxima.
//             (One thread per row, with nothing to exchange, took as long for
//             long prompts, 733 against 720 us for 8192 tokens, and 106
//             against 68 us for 4096 tokens under a window of 128, whose short
//             units are a chain of steps.)
//             O is rescaled only when a row's maximum grew by more than 2^8,
//             which fits every format here; the stale maximum is as good a
//             base for the powers as the true one.
//   16        copies queries, keys and values
//   17        issues the matrix instructions
//   18        values of key tiles that the mask cuts: rows that no query sees
//             are zeroed (a masked score gives P = 0, but 0 times what a stale
//             page holds need not be 0), and so are infinities and NaN in rows
//             that some queries see and some do not.
//   19        takes units and looks up their rows and first pages
// A value that is not finite must reach the rows that see it and no other,
// which a matrix product cannot do where the mask cuts. There it counts as
// zero, and since a positive weight times an infinity or NaN is that infinity
// or NaN whatever the weight, the epilogue adds it to the rows that see its
// key: the keys at the two edges of the mask, fewer than a unit's tokens at
// each. (8192 tokens with nothing but NaN for values: 1.16 ms, 0.69 without; 32
// heads with a key head each, whose units are 256 tokens: 2.6 ms, 0.40.)
//
// P and the sum l: P is rounded to bf16 for the second product, whose other
// operand is bf16 (a relative error of 2^-8 at most, as the result's own
// rounding); l adds the float32 values, which the softmax warps have at hand
// (the rounded ones would have to be taken out of their pairs again).
//
// Few rows: where the units are at most half as many as the SMs (and the
// sequences few), the keys of each are split over several CTAs. Each leaves
// (m, l, O) of its rows in the workspace, and the last to arrive joins them in
// their order along the keys.
//
// Every wait is bounded. A role whose wait gives up records it and goes on
// without waiting (the copies stop), so that every role ends; copies that are
// on their way are waited for, with the same bound.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "attn.cuh"

namespace mxfp4el {
namespace {

constexpr int kThreads = 640;
constexpr int kSoftmaxWarps = 16;
constexpr int kRows = 128;              // query rows per tile
constexpr int kKeys = 128;              // keys per tile
constexpr int kLoadWarp = 16, kMmaWarp = 17, kCleanWarp = 18, kUnitWarp = 19;
constexpr int kUnitRing = 4;
constexpr int kUnitReaders = 3 + kSoftmaxWarps;     // copies, MMA, values, softmax
// A CTA takes its next unit while at most one unit, or units of at most this
// many key tiles, are ahead: short units are taken early enough to hide the
// lookup, long ones late enough to spread the last of them over the CTAs.
constexpr int kAheadTiles = 8;
// Up to so many sequences, the unit warp keeps their rows in its lanes, takes
// the longest first and may split units over the keys. Against the form for
// more of them, 32 query and 8 key heads of 128: 30 chunks of 100 to 500 tokens
// behind up to 8000 keys 475 us (518), 20 of 4 tokens behind up to 2000 33 us
// (48), 8 single tokens behind 8000 58 us (90); a chunk of 2048 tokens beside 7
// single tokens 255 us (248), beside 29 344 (343).
constexpr int kFewSeqs = 30;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;         // S of tile t at 128 t, O at kOCol + D t
constexpr float kRescale = 8.f;
// A join reads every part's 128 rows of O, about what a key tile costs: with n
// key tiles sqrt(n) parts leave sqrt(n) tiles and as many pieces to read.
constexpr int kMaxParts = 32;           // one lane each

template <int D>
struct Shape {
  static constexpr int kSubs = D / 64;                       // 128-byte columns of a row
  static constexpr uint32_t kSub = 128 * 128;                // bytes: 128 rows of one column
  static constexpr uint32_t kTileBytes = kSubs * kSub;
  static constexpr int kStages = D == 128 ? 5 : 8;           // key and value tiles in flight
  static constexpr int kQSlots = D == 128 ? 1 : 2;           // units' queries, as far as they fit
};

struct PrefillMaps {
  CUtensorMap q;      // (64, head, column, token), box (64, group, 1, n)
  CUtensorMap k, v;   // as the cache's maps, one column per box
};

struct PrefillArgs {
  AttnArgs a;
  int n;              // tokens per tile
  int box_rows, box_shift;
  int units;          // slots x key heads
  int slots;
  unsigned int* counter;   // next unit; [1]: CTAs that are done; then one per unit and row tile
  float* pieces;           // per (unit part, row tile): 128 rows of O, then their m c and l
};

struct Unit {
  int seq, kvh;       // seq < 0: the end
  int row0, nt;       // first token row of the call, tokens (<= 2 n)
  int pos0;           // position of the first token
  int hi;             // keys below hi may be seen
  int lo;             // first key of the first token's window
  int start;          // first key of the first window tile
  int sinks;          // keys below this are seen beside the window
  int sink_tiles;
  int i0, tiles[2];   // key tiles [i0, tiles[t]) for row tile t (tiles[1] >= tiles[0])
  int parts, piece;   // CTAs that share the unit; this one's piece
  int first_piece, id;   // the first one's piece; the unit's number
};

template <int D>
struct __align__(16) PrefillShared {
  uint64_t full[Shape<D>::kStages], empty[Shape<D>::kStages], raw[Shape<D>::kStages];
  uint64_t q_full[Shape<D>::kQSlots], q_empty[Shape<D>::kQSlots];
  uint64_t s_full[2], p_full[2], o_full[2], o_empty[2];
  uint64_t u_full[kUnitRing], u_empty[kUnitRing];
  uint64_t drain;
  uint32_t tmem_base;
  int joins[2];
  int bad_lo[kUnitRing], bad_hi[kUnitRing];   // keys whose values that are not finite were zeroed
  Unit unit[kUnitRing];
  int first_ids[kUnitRing][16];              // pages of the unit's first key tile
  float row_max[2][2][kRows];                // [tile][half of the keys]
  float row_sum[D == 64 ? 2 : 1][2][D == 64 ? kRows : 1];
};

// Key tile i of a unit: its first key, the keys below which a row may see it
// (tiles of first keys end where the window's tiles begin) and the columns
// that matter.
struct KeyTile {
  int j0, end, cols;
  bool cut;           // the mask hides some of its keys from some of the unit's rows
};
__device__ __forceinline__ KeyTile key_tile(const Unit& u, int i, int window) {
  KeyTile t;
  const bool sink = i < u.sink_tiles;
  t.j0 = sink ? i * kKeys : u.start + (i - u.sink_tiles) * kKeys;
  t.end = sink ? min(u.sinks, u.start) : u.hi;
  t.cols = min(kKeys, t.end - t.j0);
  t.cut = sink || t.j0 + kKeys - 1 > u.pos0 || (window != 0 && t.j0 <= u.pos0 + u.nt - 1 - window);
  return t;
}

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

// Instruction descriptor of tcgen05.mma kind::f16, bf16 operands, float32
// accumulator; b_rows_k: B's rows run along K (its columns are contiguous).
__device__ __forceinline__ constexpr uint32_t mma_idesc(int n, bool b_rows_k) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_rows_k ? 1u << 16 : 0u) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kRows >> 4) << 24);
}
// Shared-memory descriptor, 128-byte swizzle: 8-row groups 1024 bytes apart.
// For a B whose columns are contiguous, blocks of 64 columns are `lead` bytes
// apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// The lowest n bits (n may be negative, or past 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Whether lane's box of a key tile, whose first key is `key`, holds a key that
// a row sees.
__device__ __forceinline__ bool box_wanted(const Unit& u, const KeyTile& kt, int i, int key,
                                           int lane, const PrefillArgs& p) {
  return lane < (kKeys >> p.box_shift) && key < kt.end &&
         (i < u.sink_tiles || key + p.box_rows > u.lo || key < u.sinks);
}
// The key's page; an id out of range is counted (and copied as zeros).
__device__ __forceinline__ int page_id(const PrefillArgs& p, const Unit& u, int key) {
  const AttnArgs& a = p.a;
  const int id = __ldg(a.seqs.page_table + (int64_t)u.seq * a.seqs.table_stride +
                       (key >> a.cache.page_shift));
  if ((unsigned)id >= (uint64_t)a.cache.num_pages) atomicAdd(&a.status[kStatusBadPages], 1ull);
  return id;
}

// 32 bytes at p: at once where p allows it. A thread's rows lie apart, so each
// store instruction touches 32 rows, and their number is what the epilogue
// costs.
__device__ __forceinline__ void store32(__nv_bfloat16* p, const uint32_t* w) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *(reinterpret_cast<uint4*>(p) + 1) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// 1 / (l + e^(sink - m)) in the scale of m (a power of two's exponent), for a
// row with running maximum m and sum l: out = o * that.
__device__ __forceinline__ float finish(const AttnArgs& a, int head, float m, float l) {
  if (l == 0.f) return 0.f;
  float f = 1.f;
  if (a.sink_logits != nullptr) {
    const float z = __ldg(a.sink_logits + head) * kLog2e;
    const float top = fmaxf(m, z), base = top == -INFINITY ? 0.f : top;
    f = exp2_approx(m - base);
    l = l * f + exp2_approx(z - base);
  }
  return f / l;
}

// Whether every token of the unit sees key j, which one of them sees.
__device__ __forceinline__ bool all_see(const Unit& u, int j, int window) {
  return j <= u.pos0 &&
         (window == 0 || j > u.pos0 + u.nt - 1 - window || j < u.sinks);
}

// O of a warp's rows (columns col0 .. col0 + D / 2 - 1 of the head, at o_addr)
// plus the values that are not finite of the keys in [bad_lo, bad_hi] that some
// of the unit's tokens see and some do not: those before the window of the
// last token, and those behind the first token. `pos` is the lane's position,
// pos_last the warp's last.
template <int D>
__device__ __forceinline__ void add_not_finite(const AttnArgs& a, const Unit& u, int bad_lo,
                                               int bad_hi, int pos, int pos_last, bool row,
                                               uint32_t o_addr, int col0, int lane) {
  const __nv_bfloat16* values = static_cast<const __nv_bfloat16*>(a.cache.v) +
                                (int64_t)u.kvh * a.cache.v_head + col0;
#pragma unroll 1
  for (int edge = 0; edge < 2; ++edge) {
    const int from = max(bad_lo, edge == 0 ? max(u.lo, u.sinks) : u.pos0 + 1);
    const int to = min(bad_hi, edge == 1 ? pos_last
                               : a.window == 0 ? -1
                                               : min(u.pos0, u.pos0 + u.nt - 1 - a.window));
#pragma unroll 1
    for (int j0 = from; j0 <= to; j0 += 32) {
      // Lane i looks up key j0 + i; a page id out of range has zeros.
      int64_t at = -1;
      if (j0 + lane <= to) {
        const int64_t page = page_of(a.seqs, a.cache, u.seq, (j0 + lane) >> a.cache.page_shift);
        if (page >= 0)
          at = page * a.cache.v_page + ((j0 + lane) & (a.cache.page_size - 1)) * a.cache.v_slot;
      }
      const uint32_t keys = __ballot_sync(kFullMask, at >= 0);
#pragma unroll 1
      for (int q = 0; q < D / 2; q += 16) {
        uint32_t o[16];
        __syncwarp();
        tmem_ld16(o_addr + q, o);
        tmem_wait_ld();
        for (uint32_t left = keys; left != 0; left &= left - 1) {
          const int i = __ffs(left) - 1;
          const uint4* v = reinterpret_cast<const uint4*>(values + __shfl_sync(kFullMask, at, i) + q);
          if (!row || !key_visible(j0 + i, pos, a.window, a.sinks)) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 x = __ldg(v + h);
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float lo = __uint_as_float(o[8 * h + 2 * e]), hi = __uint_as_float(o[8 * h + 2 * e + 1]);
              if ((w[e] & 0x7f80u) == 0x7f80u) lo += __uint_as_float(w[e] << 16);
              if ((w[e] & 0x7f800000u) == 0x7f800000u) hi += __uint_as_float(w[e] & 0xffff0000u);
              o[8 * h + 2 * e] = __float_as_uint(lo);
              o[8 * h + 2 * e + 1] = __float_as_uint(hi);
            }
          }
        }
        __syncwarp();
        tmem_st16(o_addr + q, o);
        tmem_wait_st();
      }
    }
  }
}

// kSplit: units may be shared by several CTAs.
template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
attention_prefill_kernel(const __grid_constant__ PrefillMaps maps, const PrefillArgs p) {
  using S = Shape<D>;
  constexpr size_t kPieceFloats = (size_t)kRows * (D + 2);
  // Tiles start on 1024-byte boundaries (the swizzle's), and there is no room
  // to move up to one.
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  if ((smem_addr(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicAdd(&p.a.status[kStatusWaitTimeouts], 1ull);
    return;
  }
  unsigned char* q_smem = smem_raw;
  unsigned char* ring = q_smem + S::kQSlots * 2 * S::kTileBytes;
  PrefillShared<D>& sh =
      *reinterpret_cast<PrefillShared<D>*>(ring + (size_t)S::kStages * S::kTileBytes);
  const AttnArgs& a = p.a;
  const int warp = __shfl_sync(kFullMask, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&maps.q);
    prefetch_tensor_map(&maps.k);
    prefetch_tensor_map(&maps.v);
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
      mbar_init(&sh.raw[s], 1);
    }
    for (int s = 0; s < S::kQSlots; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_full[t], kSoftmaxWarps / 2);
      mbar_init(&sh.o_full[t], 1);
      mbar_init(&sh.o_empty[t], kSoftmaxWarps / 2);
    }
    for (int r = 0; r < kUnitRing; ++r) {
      mbar_init(&sh.u_full[r], 1);
      mbar_init(&sh.u_empty[r], kUnitReaders);
    }
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = __shfl_sync(kFullMask, sh.tmem_base, 0);
  pdl_wait();
  bool ok = true;
  struct { int stage, q_slot; uint32_t phase, q_phase, raw_parity; } last = {};   // the copies' state

  // The softmax threads hold 64 scores each: they take registers that the
  // other warps give up (512 x 104 + 128 x 64 = 640 x 96).
  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    // ------------------------------------------------ softmax and epilogue
    const int t = warp >> 3, half = (warp >> 2) & 1;         // row tile, half of the keys
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lanes + (uint32_t)t * 128;
    const uint32_t o_addr = tmem + lanes + kOCol + (uint32_t)(t * D + half * (D / 2));
    const int tok = t * p.n + row / a.group, head = row % a.group;
    const bool in_tile = row < p.n * a.group;
    const int tok_first = t * p.n + (row - lane) / a.group;                  // of the warp's rows
    const int tok_last = t * p.n + min((row - lane + 31) / a.group, p.n - 1);
    const float c = a.scale * kLog2e;
    int slot = 0;
    uint32_t u_phase = 0, s_phase = 0, o_phase = 0;
    for (;;) {
      ok = ok && mbar_wait_warp(&sh.u_full[slot], u_phase);
      if (!ok) break;
      const Unit u = sh.unit[slot];
      if (u.seq < 0) break;
      const int tiles = u.tiles[t];
      const bool write = in_tile && tok < u.nt;
      const int pos = u.pos0 + min(tok, u.nt - 1);
      const int pos_first = u.pos0 + min(tok_first, u.nt - 1);
      const int pos_last = u.pos0 + min(tok_last, u.nt - 1);
      // Key tiles [whole0, whole1) are seen whole by every row of the warp.
      const int whole0 = u.sink_tiles +
                         (a.window ? (max(0, pos_last - a.window + 1 - u.start) + kKeys - 1) / kKeys : 0);
      const int whole1 = u.sink_tiles + max(0, pos_first + 1 - u.start) / kKeys;
      float m = -INFINITY, l = 0.f, mc = 0.f;     // mc: -m c, or 0 while m is -infinity

#pragma unroll 1
      for (int i = u.i0; i < tiles; ++i) {
        if (ok) ok = mbar_wait_warp(&sh.s_full[t], s_phase);
        s_phase ^= 1u;
        tc_fence_after_sync();
        float s[64];
        tmem_ld32(s_addr + 64 * half, s);
        tmem_ld32(s_addr + 64 * half + 32, s + 32);
        tmem_wait_ld();
        // Of this warp's two blocks of 32 keys: `live` has a key that one of
        // its rows sees, `used` takes part in the second product (P of keys
        // that no row of the warp sees is zero).
        bool live[2] = {true, true}, used[2] = {true, true};
        if (i < whole0 || i >= whole1) {
          const KeyTile kt = key_tile(u, i, a.window);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int j0 = kt.j0 + 64 * half + 32 * q;
            used[q] = 64 * half + 32 * q < kt.cols;
            live[q] = j0 <= min(pos_last, kt.end - 1) &&
                      (i < u.sink_tiles || a.window == 0 || j0 + 31 > pos_first - a.window ||
                       j0 < u.sinks);
            const bool all = j0 + 31 <= min(pos_first, kt.end - 1) &&
                             (a.window == 0 || j0 > pos_last - a.window || j0 + 32 <= u.sinks);
            if (live[q] && !all) {
              // Bit j of `seen`: the row sees key j0 + j.
              uint32_t seen = low_bits(min(pos, kt.end - 1) - j0 + 1);
              if (a.window != 0)
                seen &= ~low_bits(pos - a.window + 1 - j0) | low_bits(u.sinks - j0);
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (!((seen >> j) & 1u)) s[32 * q + j] = -INFINITY;
            }
          }
        }
        float mine = -INFINITY;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (live[q]) {
            const float* x = s + 32 * q;
            float tops[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
            for (int j = 4; j < 28; j += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], x[j + 2 * e], x[j + 2 * e + 1]);
            tops[0] = max3(tops[0], x[28], x[29]);
            tops[1] = max3(tops[1], x[30], x[31]);
            mine = max3(mine, max3(tops[0], tops[1], tops[2]), tops[3]);
          }
        }
        // The other half's maximum. Past the barrier both halves hold their
        // scores in registers, so P may overwrite them.
        sh.row_max[t][half][row] = mine;
        tc_fence_before_sync();
        bar_sync(1 + t, 256);
        tc_fence_after_sync();
        const float top = max3(m, mine, sh.row_max[t][half ^ 1][row]);
        // (Rows that hold no token hold anything: they have no say.)
        if (__any_sync(kFullMask, write && (top - m) * c > kRescale)) {
          // A maximum grew by more than kRescale (or was -infinity): O and l
          // move to the new base. O's last product is done: S was issued after
          // it.
          const bool fresh = m == -INFINITY;
          const float keep = fresh ? 0.f : exp2_approx((m - top) * c);
          l *= keep;
          m = top;
          mc = m == -INFINITY ? 0.f : -m * c;
          if (i > u.i0) {
#pragma unroll 1
            for (int q = 0; q < D / 2; q += 16) {
              uint32_t o[16];
              tmem_ld16(o_addr + q, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                o[j] = __float_as_uint(fresh ? 0.f : __uint_as_float(o[j]) * keep);
              tmem_st16(o_addr + q, o);
            }
          }
        }
        // P of a block of 32 keys, and its part of the sum. Each step's
        // instructions are independent of each other.
        auto powers = [&](float* x, int q) {
          uint32_t w[16];
          const float2 c2 = make_float2(c, c), b2 = make_float2(mc, mc);
          float2 sum[4] = {};
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 e = ffma2(make_float2(x[2 * j], x[2 * j + 1]), c2, b2);
            e = make_float2(exp2_approx(e.x), exp2_approx(e.y));
            w[j] = pack_bf16(e.x, e.y);
            sum[j & 3] = fadd2(sum[j & 3], e);
          }
          tmem_st16(s_addr + 32 * half + 16 * q, w);
          const float2 z = fadd2(fadd2(sum[0], sum[1]), fadd2(sum[2], sum[3]));
          l += z.x + z.y;
        };
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          if (live[q]) {
            powers(s + 32 * q, q);
          } else if (used[q]) {
            const uint32_t zero[16] = {};
            tmem_st16(s_addr + 32 * half + 16 * q, zero);
          }
        }
        tmem_wait_st();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[t]);
      }

      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) +
                           ((int64_t)(u.row0 + tok) * a.heads + u.kvh * a.group + head) * D +
                           half * (D / 2);
      if (tiles > u.i0) {
        // The halves' sums, in an array of their own where there is room, else
        // after the last tile's maxima have been read and before the next
        // unit's are written.
        float(*sums)[kRows] = D == 64 ? reinterpret_cast<float(*)[kRows]>(sh.row_sum[D == 64 ? t : 0])
                                      : sh.row_max[t];
        if (D != 64) bar_sync(1 + t, 256);
        sums[half][row] = l;
        bar_sync(1 + t, 256);
        l += sums[half ^ 1][row];
        if (D != 64) bar_sync(1 + t, 256);
        const float inv = finish(a, u.kvh * a.group + head, m * c, l);
        ok = ok && mbar_wait_warp(&sh.o_full[t], o_phase);
        o_phase ^= 1u;
        tc_fence_after_sync();
        // Warp 18 may still be at key tiles that only the other row tile sees;
        // all that these rows see is in the range by now, and what is not
        // theirs changes nothing.
        const int bad_lo = __shfl_sync(kFullMask, *reinterpret_cast<volatile int*>(&sh.bad_lo[slot]), 0);
        const int bad_hi = __shfl_sync(kFullMask, *reinterpret_cast<volatile int*>(&sh.bad_hi[slot]), 0);
        if (bad_lo <= bad_hi)
          add_not_finite<D>(a, u, bad_lo, bad_hi, pos, pos_last, write, o_addr, half * (D / 2), lane);
        if (!kSplit || u.parts == 1) {
#pragma unroll
          for (int q = 0; q < D / 64; ++q) {
            float o[32];
            tmem_ld32(o_addr + 32 * q, o);
            tmem_wait_ld();
            if (write) {
              uint32_t w[16];
#pragma unroll
              for (int j = 0; j < 16; ++j)
                w[j] = l == 0.f ? 0u : pack_bf16(o[2 * j] * inv, o[2 * j + 1] * inv);
              store32(out + 32 * q, w);
              store32(out + 32 * q + 16, w + 8);
            }
          }
        } else {
          float* piece = p.pieces + (size_t)(u.piece * 2 + t) * kPieceFloats;
#pragma unroll 1
          for (int q = 0; q < D / 64; ++q) {
            float o[32];
            tmem_ld32(o_addr + 32 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              *reinterpret_cast<float4*>(piece + (size_t)row * D + half * (D / 2) + 32 * q + j) =
                  make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
          }
          if (half == 0) {
            piece[kRows * D + row] = m * c;
            piece[kRows * D + kRows + row] = l;
          }
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.o_empty[t]);
      } else if (kSplit && u.parts > 1) {
        if (half == 0) {
          float* stats = p.pieces + (size_t)(u.piece * 2 + t) * kPieceFloats + kRows * D + row;
          stats[0] = -INFINITY;
          stats[kRows] = 0.f;
        }
      } else if (write) {
        for (int j = 0; j < D / 16; ++j)
          *reinterpret_cast<uint4*>(out + 8 * j) = make_uint4(0, 0, 0, 0);
      }
      if (kSplit && u.parts > 1) {
        __threadfence();
        bar_sync(1 + t, 256);
        if ((warp & 7) == 0 && lane == 0)
          sh.joins[t] = atomicInc(p.counter + 2 + 2 * u.id + t, (unsigned)(u.parts - 1)) ==
                        (unsigned)(u.parts - 1);
        bar_sync(1 + t, 256);
        if (sh.joins[t]) {
          __threadfence();
          // A warp per row, lane k with part k's m and l.
          const float* first = p.pieces + (size_t)(u.first_piece * 2 + t) * kPieceFloats;
          for (int r = warp & 7; r < p.n * a.group; r += 8) {
            const int token = t * p.n + r / a.group, h = u.kvh * a.group + r % a.group;
            if (token >= u.nt) break;
            float mk = -INFINITY, lk = 0.f;
            if (lane < u.parts) {
              const float* stats = first + (size_t)lane * 2 * kPieceFloats + kRows * D + r;
              mk = __ldcg(stats);
              lk = __ldcg(stats + kRows);
            }
            float top = mk;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
            const float f = exp2_approx(mk - (top == -INFINITY ? 0.f : top));
            float total = lk * f;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
            const float inv = finish(a, h, top, total);
            float o[D / 32] = {};
#pragma unroll 4
            for (int k = 0; k < u.parts; ++k) {
              // A part that saw nothing has left no O.
              const bool has = __shfl_sync(kFullMask, mk, k) != -INFINITY;
              const float fk = __shfl_sync(kFullMask, f, k);
              const float* x = first + (size_t)k * 2 * kPieceFloats + (size_t)r * D + lane * (D / 32);
              if constexpr (D == 128) {
                const float4 v = has ? __ldcg(reinterpret_cast<const float4*>(x))
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
                o[0] = fmaf(v.x, fk, o[0]);
                o[1] = fmaf(v.y, fk, o[1]);
                o[2] = fmaf(v.z, fk, o[2]);
                o[3] = fmaf(v.w, fk, o[3]);
              } else {
                const float2 v = has ? __ldcg(reinterpret_cast<const float2*>(x))
                                     : make_float2(0.f, 0.f);
                o[0] = fmaf(v.x, fk, o[0]);
                o[1] = fmaf(v.y, fk, o[1]);
              }
            }
            uint32_t* to = reinterpret_cast<uint32_t*>(
                static_cast<__nv_bfloat16*>(a.out) +
                ((int64_t)(u.row0 + token) * a.heads + h) * D + lane * (D / 32));
#pragma unroll
            for (int e = 0; e < D / 64; ++e)
              to[e] = total == 0.f ? 0u : pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv);
          }
        }
        bar_sync(1 + t, 256);                          // joins has been read
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.u_empty[slot]);
      if (++slot == kUnitRing) {
        slot = 0;
        u_phase ^= 1u;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
  if (warp == kUnitWarp) {
    // ------------------------------------------------ units
    // Takes units and works out what they hold, some units ahead of the other
    // warps: the lookups are chains of loads. With few sequences their rows
    // stay in the lanes, and the units are taken from the longest sequence
    // down; else from the last one up. Inside a sequence the last tokens, which
    // see the most keys, come first.
    const int n2 = 2 * p.n, seqs = a.seqs.num_seqs;
    const bool few = seqs <= kFewSeqs;
    SeqRows mine = {a.T, 0, 0, 0};                // lane r: the sequence of rank r
    int mine_seq = 0, before = 0, mine_tiles = 0; // query tiles of the sequences before it
    int units = p.units;
    if (few) {
      SeqRows r = mine;
      if (lane <= seqs)
        r = sequence_rows(a.seqs, lane, a.T, a.cache.page_shift, a.status, blockIdx.x == 0);
      int rank = 0;
      for (int b = 0; b <= seqs; ++b) {
        const int len = __shfl_sync(kFullMask, r.len, b);
        rank += len > r.len || (len == r.len && b < lane) ? 1 : 0;
      }
      for (int b = 0; b <= seqs; ++b)
        if (__shfl_sync(kFullMask, rank, b) == lane) mine_seq = b;
      mine.first = __shfl_sync(kFullMask, r.first, mine_seq);
      mine.count = __shfl_sync(kFullMask, r.count, mine_seq);
      mine.pos0 = __shfl_sync(kFullMask, r.pos0, mine_seq);
      mine_tiles = lane <= seqs ? (mine.count + n2 - 1) / n2 : 0;
      int incl = mine_tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kFullMask, incl, o);
        if (lane >= o) incl += up;
      }
      before = incl - mine_tiles;
      units = __shfl_sync(kFullMask, incl, 31) * a.cache.kv_heads;
    }
    // Parts per unit, as far as the CTAs go round; index = unit * parts + part.
    const int parts = kSplit && few && units > 0 && units <= (int)gridDim.x / 2 ? (int)gridDim.x / units : 1;
    units *= parts;
    // Units published and not yet released, and their key tiles (lane s: ring
    // slot s's).
    int published = 0, released = 0, ahead = 0, slot_tiles = 0;
    int idx = blockIdx.x;
    for (;;) {
      Unit u;
      u.seq = -1;
      if (idx < units) {
        u.id = kSplit ? idx / parts : idx;
        const int part = idx - u.id * parts;
        const int s = u.id / a.cache.kv_heads;
        u.kvh = u.id - s * a.cache.kv_heads;
        int tile;
        SeqRows r;
        if (few) {
          const int rank = __popc(__ballot_sync(kFullMask, lane <= seqs && before <= s)) - 1;
          u.seq = __shfl_sync(kFullMask, mine_seq, rank);
          r.first = __shfl_sync(kFullMask, mine.first, rank);
          r.count = __shfl_sync(kFullMask, mine.count, rank);
          r.pos0 = __shfl_sync(kFullMask, mine.pos0, rank);
          tile = __shfl_sync(kFullMask, mine_tiles, rank) - 1 -
                 (s - __shfl_sync(kFullMask, before, rank));
        } else {
          const int at = p.slots - 1 - s;
          u.seq = sequence_of_slot(a.seqs, at, a.T, n2, lane);
          r = sequence_rows(a.seqs, u.seq, a.T, a.cache.page_shift, a.status,
                            lane == 0 && u.kvh == 0);
          tile = a.seqs.q_offsets == nullptr ? 0 : at - (r.first / n2 + u.seq);
        }
        const int t0 = tile * n2;
        u.nt = min(n2, r.count - t0);
        u.row0 = r.first + t0;
        u.pos0 = r.pos0 + t0;
        u.hi = max(0, u.pos0 + u.nt);
        u.lo = a.window ? max(0, u.pos0 - a.window + 1) : 0;
        u.start = u.lo & ~(p.box_rows - 1);
        u.sinks = a.sinks;
        u.sink_tiles = (min(a.sinks, u.start) + kKeys - 1) / kKeys;
        // Keys that the first row tile sees end at its last token.
        const int hi0 = max(0, u.pos0 + min(u.nt, p.n));
        u.tiles[1] = u.hi > 0 ? u.sink_tiles + (u.hi - u.start + kKeys - 1) / kKeys : 0;
        u.tiles[0] = hi0 > 0 ? u.sink_tiles + (hi0 - u.start + kKeys - 1) / kKeys : 0;
        if (u.nt <= p.n) u.tiles[1] = 0;
        u.parts = 1;
        u.i0 = 0;
        u.piece = idx;
        u.first_piece = idx - part;
        if (kSplit && parts > 1) {
          const int all = max(u.tiles[0], u.tiles[1]);
          u.parts = max(1, min(min(parts, kMaxParts), (int)sqrtf((float)all)));
          u.i0 = (int)((long long)all * part / u.parts);
          const int i1 = (int)((long long)all * (part + 1) / u.parts);
          u.tiles[0] = min(u.tiles[0], i1);
          u.tiles[1] = min(u.tiles[1], i1);
          if (part >= u.parts) u.nt = 0;               // the unit has fewer
        }
      }
      if (u.seq < 0 || u.nt > 0) {
        const int tiles = u.seq < 0 ? 0 : max(0, max(u.tiles[0], u.tiles[1]) - u.i0);
        int id = 0;
        if (tiles > 0) {
          const KeyTile kt = key_tile(u, u.i0, a.window);
          const int key = kt.j0 + lane * p.box_rows;
          if (box_wanted(u, kt, u.i0, key, lane, p)) id = page_id(p, u, key);
        }
        const int slot = published % kUnitRing;
        while (published - released >= kUnitRing) {
          if (ok) ok = mbar_wait_warp(&sh.u_empty[released % kUnitRing],
                                      (uint32_t)(released / kUnitRing) & 1u);
          ahead -= __shfl_sync(kFullMask, slot_tiles, released % kUnitRing);
          ++released;
        }
        if (lane == slot) slot_tiles = tiles;
        ahead += tiles;
        if (lane < 16) sh.first_ids[slot][lane] = id;
        if (lane == 0) {
          sh.unit[slot] = u;
          sh.bad_lo[slot] = 0x7fffffff;
          sh.bad_hi[slot] = -1;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.u_full[slot]);
        ++published;
      }
      if (u.seq < 0) break;
      while (published - released >= 2 && ahead > kAheadTiles) {
        if (ok) ok = mbar_wait_warp(&sh.u_empty[released % kUnitRing],
                                    (uint32_t)(released / kUnitRing) & 1u);
        ahead -= __shfl_sync(kFullMask, slot_tiles, released % kUnitRing);
        ++released;
      }
      unsigned taken = 0;
      if (lane == 0) taken = atomicAdd(p.counter, 1u);
      idx = (int)(gridDim.x + __shfl_sync(kFullMask, taken, 0));
    }
    if (lane == 0) {
      // The last CTA to take its end leaves the counters at zero.
      if (atomicAdd(p.counter + 1, 1u) == gridDim.x - 1) {
        p.counter[0] = 0;
        p.counter[1] = 0;
      }
    }
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------ copies
    const uint64_t keep = l2_evict_normal_policy();
    int slot = 0, stage = 0, q_slot = 0;
    uint32_t u_phase = 0, phase = 0, q_phase = 0;
    uint32_t raw_parity = 0;                      // bit s: raw[s]'s next phase
    for (;;) {
      ok = ok && mbar_wait_warp(&sh.u_full[slot], u_phase);
      if (!ok) break;
      const Unit u = sh.unit[slot];
      int id = lane < 16 ? sh.first_ids[slot][lane] : 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.u_empty[slot]);
      if (++slot == kUnitRing) {
        slot = 0;
        u_phase ^= 1u;
      }
      if (u.seq < 0) break;
      const int tiles = max(u.tiles[0], u.tiles[1]);
      if (tiles <= u.i0) continue;

      ok = ok && mbar_wait_warp(&sh.q_empty[q_slot], q_phase ^ 1u);
      if (!ok) break;
      const int row_tiles = u.nt > p.n ? 2 : 1;
      if (elect_one()) {
        mbar_arrive_expect_tx(&sh.q_full[q_slot],
                              (uint32_t)(row_tiles * S::kSubs * p.n * a.group * 128));
        for (int t = 0; t < row_tiles; ++t)
          for (int c = 0; c < S::kSubs; ++c)
            tma_load_4d(q_smem + (q_slot * 2 + t) * S::kTileBytes + c * S::kSub, &maps.q, 0,
                        u.kvh * a.group, c, u.row0 + t * p.n, &sh.q_full[q_slot], keep);
      }
      __syncwarp();
      if (++q_slot == S::kQSlots) {
        q_slot = 0;
        q_phase ^= 1u;
      }
      for (int i = u.i0; i < tiles && ok; ++i) {
        const KeyTile kt = key_tile(u, i, a.window);
        // Lane x copies box x, if a row sees a key of it; the next tile's
        // pages are looked up meanwhile.
        const int key = kt.j0 + lane * p.box_rows;
        const bool want = box_wanted(u, kt, i, key, lane, p);
        int next_id = 0;
        if (i + 1 < tiles) {
          const KeyTile nt = key_tile(u, i + 1, a.window);
          const int next_key = nt.j0 + lane * p.box_rows;
          if (box_wanted(u, nt, i + 1, next_key, lane, p)) next_id = page_id(p, u, next_key);
        }
        const uint32_t bytes = (uint32_t)__popc(__ballot_sync(kFullMask, want)) *
                               (uint32_t)p.box_rows * 128u * S::kSubs;
        for (int v = 0; v < 2; ++v) {
          ok = ok && mbar_wait_warp(&sh.empty[stage], phase ^ 1u);
          if (!ok) break;
          const bool raw = v && kt.cut;
          uint64_t* bar = raw ? &sh.raw[stage] : &sh.full[stage];
          raw_parity ^= raw ? 1u << stage : 0u;
          if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
          __syncwarp();
          if (want) {
            unsigned char* dst = ring + (size_t)stage * S::kTileBytes + (size_t)lane * p.box_rows * 128;
            for (int c = 0; c < S::kSubs; ++c)
              tma_load_5d(dst + c * S::kSub, v ? &maps.v : &maps.k, 0,
                          key & (a.cache.page_size - 1), c, u.kvh, id, bar, keep);
          }
          __syncwarp();
          if (++stage == S::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        id = next_id;
      }
    }
    last = {stage, q_slot, phase, q_phase, raw_parity};
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ matrix instructions
    // The whole warp runs the loop, on values the compiler can tell are the
    // same in every lane (they come through shuffles and votes), so that the
    // instructions' operands stay in uniform registers; one elected lane
    // issues. (A loop that one lane ran alone moved every operand over for
    // each instruction, 140 cycles apiece.) elect.sync elects the same lane
    // every time, so the products run in the order of issue and a commit
    // covers all before it. Per key tile and row tile it issues O += P V and
    // the next S back to back: the copies both need are waited for before P.
    int slot = 0, stage = 0, q_slot = 0;
    uint32_t u_phase = 0, phase = 0, q_phase = 0;
    uint32_t p_phase = 0, o_phase = 0;            // bit t: row tile t
    const uint32_t q_base = __shfl_sync(kFullMask, smem_addr(q_smem), 0);
    const uint32_t ring_addr = __shfl_sync(kFullMask, smem_addr(ring), 0);
    constexpr uint32_t kIdescO = mma_idesc(D, true);
    auto step = [&]() {
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    };
    // S of row tile t with the keys in stage k_stage.
    auto scores = [&](int t, uint32_t q_addr, int k_stage, uint32_t idesc) {
      const uint64_t qd = smem_desc(q_addr + (uint32_t)t * S::kTileBytes, 16);
      const uint64_t kd = smem_desc(ring_addr + (uint32_t)k_stage * S::kTileBytes, 16);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t at = ((uint32_t)(k / 4) * S::kSub + (uint32_t)(k % 4) * 32) >> 4;
        tc_mma_ss(tmem + (uint32_t)t * 128, qd + at, kd + at, idesc, k > 0 ? 1u : 0u);
      }
      tc_commit(&sh.s_full[t]);
    };
    while (ok) {
      ok = mbar_wait_warp(&sh.u_full[slot], u_phase);
      if (!ok) break;
      const Unit v = sh.unit[slot];
      Unit u;
      u.seq = __shfl_sync(kFullMask, v.seq, 0);
      u.nt = __shfl_sync(kFullMask, v.nt, 0);
      u.pos0 = __shfl_sync(kFullMask, v.pos0, 0);
      u.hi = __shfl_sync(kFullMask, v.hi, 0);
      u.start = __shfl_sync(kFullMask, v.start, 0);
      u.sinks = __shfl_sync(kFullMask, v.sinks, 0);
      u.sink_tiles = __shfl_sync(kFullMask, v.sink_tiles, 0);
      u.i0 = __shfl_sync(kFullMask, v.i0, 0);
      u.tiles[0] = __shfl_sync(kFullMask, v.tiles[0], 0);
      u.tiles[1] = __shfl_sync(kFullMask, v.tiles[1], 0);
      if (lane == 0) mbar_arrive(&sh.u_empty[slot]);
      if (++slot == kUnitRing) {
        slot = 0;
        u_phase ^= 1u;
      }
      if (u.seq < 0) break;
      const int tiles = max(u.tiles[0], u.tiles[1]);
      if (tiles <= u.i0) continue;
      const uint32_t q_addr = q_base + (uint32_t)q_slot * 2 * S::kTileBytes;
      if (ok) ok = mbar_wait_warp(&sh.q_full[q_slot], q_phase);
      if (ok) ok = mbar_wait_warp(&sh.full[stage], phase);
      tc_fence_after_sync();
      int cols = key_tile(u, u.i0, a.window).cols;
      if (elect_one()) {
        const uint32_t idesc = mma_idesc((cols + 15) & ~15, false);
        if (u.tiles[0] > u.i0) scores(0, q_addr, stage, idesc);
        if (u.tiles[1] > u.i0) scores(1, q_addr, stage, idesc);
        tc_commit(&sh.empty[stage]);
        if (tiles == u.i0 + 1) tc_commit(&sh.q_empty[q_slot]);
      }
      __syncwarp();
      step();
      for (int i = u.i0; i < tiles; ++i) {
        const int v_stage = stage;
        const uint32_t v_phase = phase;
        step();                                     // now at the next tile's keys
        const bool more = i + 1 < tiles;
        const int next_cols = more ? key_tile(u, i + 1, a.window).cols : 0;
        const int steps = (cols + 15) / 16;
        const uint32_t idesc = mma_idesc((next_cols + 15) & ~15, false);
        if (ok) ok = mbar_wait_warp(&sh.full[v_stage], v_phase);
        if (ok && more) ok = mbar_wait_warp(&sh.full[stage], phase);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (i < u.tiles[t]) {
            if (i == u.i0) {                        // the last unit's O has been read
              if (ok) ok = mbar_wait_warp(&sh.o_empty[t], ((o_phase >> t) & 1u) ^ 1u);
              o_phase ^= 1u << t;
            }
            if (ok) ok = mbar_wait_warp(&sh.p_full[t], (p_phase >> t) & 1u);
            p_phase ^= 1u << t;
            tc_fence_after_sync();
            const uint32_t o_tmem = tmem + kOCol + (uint32_t)t * D, p_tmem = tmem + (uint32_t)t * 128;
            const uint64_t vd = smem_desc(ring_addr + (uint32_t)v_stage * S::kTileBytes, S::kSub);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                if (k < steps)
                  tc_mma_ts(o_tmem, p_tmem + k * 8, vd + (uint32_t)(k * 2048 >> 4), kIdescO,
                            (i > u.i0 || k > 0) ? 1u : 0u);
              if (t == 1 || u.tiles[1] <= i) tc_commit(&sh.empty[v_stage]);
              if (i + 1 == u.tiles[t]) tc_commit(&sh.o_full[t]);
              else scores(t, q_addr, stage, idesc);
            }
            __syncwarp();
          }
        }
        if (more) {
          if (elect_one()) {
            tc_commit(&sh.empty[stage]);
            // All products with Q have been issued.
            if (i + 2 == tiles) tc_commit(&sh.q_empty[q_slot]);
          }
          __syncwarp();
          step();
        }
        cols = next_cols;
      }
      if (++q_slot == S::kQSlots) {
        q_slot = 0;
        q_phase ^= 1u;
      }
    }
    // TMEM is freed only after every product has finished.
    if (elect_one()) tc_commit(&sh.drain);
    mbar_wait(&sh.drain, 0);
  } else if (warp == kCleanWarp) {
    // ------------------------------------------------ values under the mask
    int slot = 0, stage = 0;
    uint32_t u_phase = 0;
    uint32_t raw_phase = 0;                       // one bit per stage
    for (;;) {
      ok = ok && mbar_wait_warp(&sh.u_full[slot], u_phase);
      if (!ok) break;
      const Unit u = sh.unit[slot];
      if (u.seq < 0) break;
      const int tiles = max(u.tiles[0], u.tiles[1]);
      int unit_lo = 0x7fffffff, unit_hi = -1;
      for (int i = u.i0; i < tiles; ++i) {
        const KeyTile kt = key_tile(u, i, a.window);
        const int v_stage = stage + 1 < S::kStages ? stage + 1 : 0;
        if (kt.cut) {
          ok = ok && mbar_wait_warp(&sh.raw[v_stage], (raw_phase >> v_stage) & 1u);
          raw_phase ^= 1u << v_stage;
          unsigned char* v = ring + (size_t)v_stage * S::kTileBytes;
          int bad_lo = 0x7fffffff, bad_hi = -1;
          for (int r = lane; r < ((kt.cols + 15) & ~15); r += 32) {
            const int key = kt.j0 + r;
            const bool seen = key < kt.end && (i < u.sink_tiles || key >= u.lo || key < u.sinks);
            if (seen && all_see(u, key, a.window)) continue;
#pragma unroll
            for (int c = 0; c < 8 * S::kSubs; ++c) {
              // Lanes start at different pieces of their rows: no bank conflicts.
              uint4* at = reinterpret_cast<uint4*>(v + (c / 8) * S::kSub + r * 128 +
                                                   ((c + lane) & 7) * 16);
              if (!seen) {
                *at = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 x = *at;
                uint32_t w[4] = {x.x, x.y, x.z, x.w};
                bool bad = false;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  bad |= (w[e] & 0x7f80u) == 0x7f80u || (w[e] & 0x7f800000u) == 0x7f800000u;
                if (bad) {
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    w[e] &= ((w[e] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) |
                            ((w[e] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
                  *at = make_uint4(w[0], w[1], w[2], w[3]);
                  bad_lo = min(bad_lo, key);
                  bad_hi = max(bad_hi, key);
                }
              }
            }
          }
          bad_lo = __reduce_min_sync(kFullMask, bad_lo);
          bad_hi = __reduce_max_sync(kFullMask, bad_hi);
          unit_lo = min(unit_lo, bad_lo);
          unit_hi = max(unit_hi, bad_hi);
          if (lane == 0 && bad_hi >= 0) {
            sh.bad_lo[slot] = unit_lo;
            sh.bad_hi[slot] = unit_hi;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.full[v_stage]);
        }
        stage = stage + 2 < S::kStages ? stage + 2 : stage + 2 - S::kStages;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.u_empty[slot]);
      if (++slot == kUnitRing) {
        slot = 0;
        u_phase ^= 1u;
      }
    }
  }
  }
  if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
  tc_fence_before_sync();
  const bool gave_up = __syncthreads_or(!ok);
  tc_fence_after_sync();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
  // No copy may outlive the block: where no wait gave up, all have been used.
  if (gave_up && warp == kLoadWarp) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_wait_warp(&sh.raw[s], ((last.raw_parity >> s) & 1u) ^ 1u);
      mbar_wait_warp(&sh.full[s], s < last.stage ? last.phase : last.phase ^ 1u);
    }
    for (int s = 0; s < S::kQSlots; ++s)
      mbar_wait_warp(&sh.q_full[s], s < last.q_slot ? last.q_phase : last.q_phase ^ 1u);
  }
}

template <int D, bool kSplit>
cudaError_t launch_kernel(const PrefillMaps& maps, const PrefillArgs& p, int grid,
                          cudaStream_t stream) {
  using S = Shape<D>;
  constexpr size_t smem =
      (size_t)(2 * S::kQSlots + S::kStages) * S::kTileBytes + sizeof(PrefillShared<D>);
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t err = cudaSuccess;
  std::call_once(once[dev & 63], [&] {
    err = cudaFuncSetAttribute(attention_prefill_kernel<D, kSplit>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (err != cudaSuccess) return err;
  return launch_after_previous(attention_prefill_kernel<D, kSplit>, dim3((unsigned)grid),
                               dim3(kThreads), smem, stream, maps, p);
}

template <int D>
cudaError_t launch(const AttnArgs& a, void* workspace, cudaStream_t stream) {
  using S = Shape<D>;
  PrefillArgs p = {};
  p.a = a;
  p.n = kRows / a.group;
  p.box_rows = std::min(a.cache.page_size, kKeys);
  while ((1 << p.box_shift) < p.box_rows) ++p.box_shift;
  const int64_t slots = query_tile_slots(a.seqs, a.T, 2 * p.n);
  p.slots = (int)slots;
  p.units = (int)(slots * a.cache.kv_heads);   // below 2^31, as the caller has checked
  p.counter = prefill_counters(workspace);
  PrefillMaps maps;
  if (!kv_tensor_map(a.cache, false, p.box_rows, 1, &maps.k) ||
      !kv_tensor_map(a.cache, true, p.box_rows, 1, &maps.v))
    return cudaErrorInvalidValue;
  {
    auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
    if (enc == nullptr) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {64, (cuuint64_t)a.heads, (cuuint64_t)S::kSubs, (cuuint64_t)a.T};
    const cuuint64_t strides[3] = {a.heads > 1 ? (cuuint64_t)a.q_head * 2 : 16, 128,
                                   a.T > 1 ? (cuuint64_t)a.q_token * 2 : 16};
    const cuuint32_t box[4] = {64, (cuuint32_t)a.group, 1, (cuuint32_t)p.n};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    if (enc(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(a.q), dims, strides,
            box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  p.pieces = static_cast<float*>(workspace_pieces(workspace));
  static_assert(sizeof(float) * 2 * 256 * kRows * (D + 2) <= kPiecesBytes, "workspace");
  // Where the units might be few enough to be split and long enough, a CTA per
  // SM. (The form that cannot split is 5 % faster at short units.)
  const int sms = std::min(attention_num_sms(), 256);
  const int64_t room = (int64_t)a.seqs.max_pages << a.cache.page_shift;
  if (a.seqs.num_seqs <= kFewSeqs && p.units <= sms && room >= 4 * kKeys)
    return launch_kernel<D, true>(maps, p, sms, stream);
  return launch_kernel<D, false>(maps, p, std::min(sms, p.units), stream);
}

}  // namespace

cudaError_t launch_attention_prefill(const AttnArgs& a, void* workspace, cudaStream_t stream) {
  return a.cache.head_dim == 64 ? launch<64>(a, workspace, stream) : launch<128>(a, workspace, stream);
}

}  // namespace mxfp4el

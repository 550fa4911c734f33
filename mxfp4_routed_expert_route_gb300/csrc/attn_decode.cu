// attn_decode.cu -- attention of one new token of each sequence over the
// paged cache, split over the cache's length and joined.
//
// The query heads that share a key head are the rows of one unit of work
// (sequence, key head, block of up to 16 kMT query heads), so every key and
// value is read once per unit:
//
//   s = scale q K^T,  m = max s,  l = sum e^(s - m),  o = sum e^(s - m) v / l
//
// kept as a running (m, l, o) over tiles of keys, in powers of two.
//
// Bound: bytes. A unit reads 2 len D elements of cache and does 2 len D
// multiply-adds a row, a few operations per byte, so the design is about
// keeping HBM busy: one warp issues tensor copies of whole pages into a ring
// of stages and never computes; four or eight warps per 16 heads consume. 128
// sequences of up to 16384 keys, 8 key heads of 128: 621 us, 7.0 TB/s, a little
// above a plain copy; two of up to 131072: 160 us, 6.6 TB/s, of which the launch and the join
// take about 5; DRAM reads 1.00 times the keys and values.
//
// Split. Lengths live on the device, so the host launches a fixed grid and
// every CTA derives the same split: the tiles of all units, in unit order,
// are cut into equal runs, one per CTA. A unit that lies inside one run is
// finished there. Otherwise each of its CTAs writes an unnormalised piece
// (m, l, o) to the workspace, and the CTA that arrives last joins the pieces
// in their order along the keys, so the result does not depend on who is
// last. A join costs round trips through L2, so runs hold at least kMinTiles tiles
// (one sequence of 1000 keys: 8.5 us with two, 9.2 with four, 12.6 with six), and
// where no unit has more than kWholeTiles the units are dealt out whole instead
// (one sequence of 333 keys, 8 key heads: 11.1 us with joins, 8.0 without; 16
// sequences of up to 132 visible keys: 11.7 and 6.9).
//
// Matrix products. bf16: mma.sync m16n8k16 with the 16 heads as rows. The
// legacy tensor path is enough here (two instructions per key and 16 heads
// against 512 bytes of cache at D = 128), and its register fragments let the
// softmax follow without a trip through tensor memory. e^(s - m) is rounded
// to bf16 for the second product, whose other operand is bf16 (a relative
// error of 2^-8 at most, as the result's own rounding); the sum l adds the
// rounded values, so that the weights still add to one. float32: CUDA-core
// multiply-adds.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "attn.cuh"

namespace mxfp4el {
namespace {

constexpr int kMinTiles = 2;            // tiles per run at least (see above)
constexpr int kWholeTiles = 8;
constexpr int kMaxCtas = 256;
constexpr int kMaxSeqs = 1024;          // sequences per launch (the prefix sums' shared memory)
constexpr int kRowsMax = 32;            // query heads per unit: 16 kMT, kMT <= 2
constexpr int kQSlots = 2;

// Bytes of a piece in the workspace: rows of o (128 floats), m and l.
constexpr size_t kPieceBytes = (size_t)kRowsMax * 128 * 4 + 2 * kRowsMax * 4;
static_assert(kMaxCtas <= kDecodeCounters && 2 * kMaxCtas * kPieceBytes <= kPiecesBytes, "workspace");

template <typename Tok, int D, int kMT = 1, int kH = 16>
struct Shape {
  // Key groups of a tile: one consumer warp each per 16 heads. float32 works
  // on the CUDA cores and needs more of them: 26 sequences of up to 57434 keys,
  // heads of 64: 147 us with four groups, 111 with eight. bf16 does not (139
  // sequences of up to 1384 keys, heads of 64: 48.2 us with four, 52.0 with
  // eight, whose join is longer).
  static constexpr int kGroups = sizeof(Tok) == 4 ? 8 : 4;
  // 32 KB of keys and values in a tile, or eight float32 keys a group.
  static constexpr int kTile = sizeof(Tok) == 2 ? 8192 / D : kGroups * 8;   // keys per tile
  static constexpr int kPer = kTile / kGroups;                      // keys per consumer warp
  static constexpr int kSub = 128 / sizeof(Tok);                    // elements in 128 bytes
  static constexpr int kSubs = D / kSub;                            // 128-byte columns of a row
  static constexpr uint32_t kHalf = (uint32_t)kTile * D * sizeof(Tok);   // keys (or values) of a tile
  // 160 KB of keys and values in flight per SM, less beside the buffers of 32
  // heads; HBM's latency times an SM's share of its bandwidth is 45 KB.
  static constexpr int kStages = (kMT == 1 ? 5 : 4) * 32768 / (2 * (int)kHalf);
  static constexpr int kQRow = D * (int)sizeof(Tok) + 16;           // padded row in shared memory
  static constexpr int kAcc = kH * D / 32;                          // result elements per lane
  // The join of a unit's warps goes through shared memory in kPasses
  // parts of kPass elements, of which each warp finishes kShare.
  static constexpr int kPasses = sizeof(Tok) == 4 && kAcc == 64 ? 2 : 1;
  static constexpr int kPass = kAcc / kPasses;
  static constexpr int kShare = kPass / kGroups >= 2 ? kPass / kGroups : 2;
};

struct Unit {
  int b, head0, rows;     // sequence, first query head, heads
  int kvh;
  int len, lo;            // keys; first key of the window
  int sink_tiles, first_tile, tiles;
};

struct DecodeArgs {
  AttnArgs a;
  int seq0, num_seqs;     // sequences of this launch
  int units_per_seq;      // key heads x head blocks
  int head_blocks;
  long long units_per_cta;     // all units / CTAs, and the remainder
  int units_over;
  int box_rows, box_shift;     // slots per tensor copy: min(page_size, kTile)
  unsigned int* counters;
  unsigned char* pieces;
};

struct DecodeMaps {
  CUtensorMap k, v;       // (128 bytes, slot, 128-byte column, head, page), 128-byte swizzle
};

template <int kMT, int kGroups>
struct __align__(16) DecodeShared {
  uint64_t full[16], empty[16];
  uint64_t q_full[kQSlots], q_empty[kQSlots];
  float merge_m[kMT][kGroups][16], merge_l[kMT][kGroups][16];
  int last;
  long long scan[1 + kGroups * kMT];  // per warp
  int longest[1 + kGroups * kMT];
  long long prefix[kMaxSeqs + 1];     // tiles of one unit of each sequence before b
};

__device__ __forceinline__ int sequence_len(const DecodeArgs& d, int b) {
  return min(max(__ldg(d.a.seqs.seq_lens + d.seq0 + b), 0),
             table_room(d.a.seqs, d.a.cache.page_shift));
}

// Tiles with a key that the token of a sequence of n keys sees; one (empty)
// tile for a sequence without keys, so that its zeros get written.
template <int kTile>
__device__ __forceinline__ void tiles_of(const AttnArgs& a, int n, int* lo, int* sink_tiles,
                                         int* first_tile, int* tiles) {
  *lo = a.window && n > a.window ? n - a.window : 0;
  *first_tile = *lo / kTile;
  *sink_tiles = min((a.sinks + kTile - 1) / kTile, *first_tile);
  *tiles = max(1, *sink_tiles + (n + kTile - 1) / kTile - *first_tile);
}

// a / b of counts of tiles, which nearly always fit 32 bits: the 64-bit
// division costs some 300 cycles, and the first copy waits for several.
__device__ __forceinline__ long long divide(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The units of a run, one after another.
template <int kTile, int kMT>
struct Walk {
  int i;               // unit of the sequence
  long long first;     // its first tile
  Unit u;
  __device__ __forceinline__ void sequence(const DecodeArgs& d, int b) {
    u.b = b;
    u.len = sequence_len(d, b);
    tiles_of<kTile>(d.a, u.len, &u.lo, &u.sink_tiles, &u.first_tile, &u.tiles);
  }
  __device__ __forceinline__ void unit(const DecodeArgs& d) {
    const int blk = d.head_blocks == 1 ? 0 : i % d.head_blocks;
    u.kvh = d.head_blocks == 1 ? i : i / d.head_blocks;
    u.head0 = u.kvh * d.a.group + blk * 16 * kMT;
    u.rows = min(16 * kMT, d.a.group - blk * 16 * kMT);
  }
  // The unit that holds `tile`; called by a whole warp.
  __device__ __forceinline__ void start(const DecodeArgs& d, const long long* prefix,
                                        long long tile, int lane) {
    const int step = (d.num_seqs + 31) / 32;
    auto before = [&](int b, bool in) {          // the entries at or before `tile`, less one
      return __popc(__ballot_sync(kFullMask, in && b < d.num_seqs &&
                                                 prefix[b] * d.units_per_seq <= tile)) - 1;
    };
    static_assert(kMaxSeqs <= 32 * 32, "two steps");
    int b = step * before(lane * step, true);
    b += before(b + lane, lane < step);
    sequence(d, b);
    first = prefix[b] * d.units_per_seq;
    i = (int)divide(tile - first, u.tiles);
    first += (long long)i * u.tiles;
    unit(d);
  }
  __device__ __forceinline__ void next(const DecodeArgs& d, long long end) {
    first += u.tiles;
    if (first >= end) return;
    if (++i == d.units_per_seq) {
      i = 0;
      sequence(d, u.b + 1);
    }
    unit(d);
  }
};

// ---------------------------------------------------------------- consumers --
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// The keys of a tile: key j lies in row j of its box, boxes of box_rows rows
// of kSubs columns of 128 bytes, 16-byte pieces swapped by the row (the
// tensor copy's 128-byte swizzle).
__device__ __forceinline__ uint32_t box_row(int j, int box_rows, int box_shift, int subs) {
  return (uint32_t)(((j >> box_shift) * subs << box_shift) + (j & (box_rows - 1))) * 128u;
}

// One warp: 16 query heads x the warp's share of each tile's keys.
// Result element i of a lane: row row(i), column col(i).
template <typename Tok, int D, int kH, int kMT>
struct Consumer;

template <int D, int kMT>
struct Consumer<__nv_bfloat16, D, 16, kMT> {
  using S = Shape<__nv_bfloat16, D, kMT>;
  static constexpr int kB = S::kPer / 16;      // blocks of 16 keys
  uint32_t q[D / 16][4];
  float m[2], l[2];          // rows lane / 4 and lane / 4 + 8; l: this lane's keys only
  float acc[S::kAcc];

  static __device__ __forceinline__ int row(int i, int lane) { return lane / 4 + (i & 2) * 4; }
  static __device__ __forceinline__ int col(int i, int lane) {
    return (i >> 2) * 8 + (lane & 3) * 2 + (i & 1);
  }
  __device__ __forceinline__ void start(uint32_t q_addr, int lane) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
      ldmatrix_x4(q_addr + (uint32_t)((lane & 15) * S::kQRow + k * 32 + (lane >> 4) * 16), q[k]);
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < S::kAcc; ++i) acc[i] = 0.f;
  }
  // vis: bit j set: key j of this warp's share is seen (all ones: no mask).
  __device__ __forceinline__ void tile(uint32_t k_addr, uint32_t v_addr, int group, int lane,
                                       float scale, uint32_t vis, const DecodeArgs& d, float*) {
    const int x = lane & 7;
    const uint32_t box = (uint32_t)d.box_rows * 128u;
    float s[2 * kB][4] = {};
#pragma unroll
    for (int y = 0; y < kB; ++y) {
      const uint32_t krow = k_addr + box_row(group * S::kPer + y * 16 + (lane >> 4) * 8 + x,
                                             d.box_rows, d.box_shift, S::kSubs);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        const int c = (k & 3) * 2 + ((lane >> 3) & 1);
        ldmatrix_x4(krow + (uint32_t)(k / 4) * box + (uint32_t)((c ^ x) << 4), b);
        mma_bf16(s[2 * y], q[k], b[0], b[1]);
        mma_bf16(s[2 * y + 1], q[k], b[2], b[3]);
      }
    }
    const int j0 = (lane & 3) * 2;       // this lane's keys: j0, j0 + 1 of each eight
    float top[2] = {-INFINITY, -INFINITY}, base[2];
#pragma unroll
    for (int n = 0; n < 2 * kB; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = (vis >> (n * 8 + j0 + (e & 1))) & 1u ? s[n][e] * scale : -INFINITY;
        top[e >> 1] = fmaxf(top[e >> 1], s[n][e]);
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(kFullMask, top[r], 1));
      top[r] = fmaxf(m[r], fmaxf(top[r], __shfl_xor_sync(kFullMask, top[r], 2)));
    }
    // The maximum rarely moves after the first tiles: rescale only then.
    if (__any_sync(kFullMask, top[0] != m[0] || top[1] != m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float keep = top[r] == -INFINITY ? 0.f : exp2_approx(m[r] - top[r]);
        l[r] *= keep;
#pragma unroll
        for (int i = 0; i < S::kAcc; ++i)
          if (((i >> 1) & 1) == r) acc[i] *= keep;
        m[r] = top[r];
      }
    }
    uint32_t p[kB][4];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      base[r] = top[r] == -INFINITY ? 0.f : top[r];
#pragma unroll
      for (int n = 0; n < 2 * kB; ++n) {
        const uint32_t w = pack_bf16(exp2_approx(s[n][2 * r] - base[r]),
                                     exp2_approx(s[n][2 * r + 1] - base[r]));
        l[r] += bf16_lo(w) + bf16_hi(w);
        p[n / 2][2 * (n & 1) + r] = w;
      }
    }
    // Values of keys that are not seen may be anything: they count as zeros.
    constexpr uint32_t kAll = kB == 2 ? 0xffffffffu : 0xffffu;
    const bool whole = (vis & kAll) == kAll;
#pragma unroll
    for (int y = 0; y < kB; ++y) {
      uint32_t keep[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint32_t pair = vis >> (y * 16 + n * 8 + j0);
        keep[n] = (pair & 1u ? 0x0000ffffu : 0u) | (pair & 2u ? 0xffff0000u : 0u);
      }
      const uint32_t vrow = v_addr + box_row(group * S::kPer + y * 16 + ((lane >> 3) & 1) * 8 + x,
                                             d.box_rows, d.box_shift, S::kSubs);
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t b[4];
        const int c = (n & 3) * 2 + (lane >> 4);
        ldmatrix_x4_trans(vrow + (uint32_t)(n / 4) * box + (uint32_t)((c ^ x) << 4), b);
        if (!whole) {
          b[0] &= keep[0];
          b[1] &= keep[1];
          b[2] &= keep[0];
          b[3] &= keep[1];
        }
        mma_bf16(acc + 8 * n, p[y], b[0], b[1]);
        mma_bf16(acc + 8 * n + 4, p[y], b[2], b[3]);
      }
    }
  }
  // The rows that a share of the result holds: element e of the share that
  // starts at element `first` is in row share_row(first, share_of(e), lane).
  static constexpr int kShareRows = 2;
  static constexpr __device__ __forceinline__ int share_of(int e) { return (e >> 1) & 1; }
  static __device__ __forceinline__ int share_row(int, int q, int lane) { return lane / 4 + 8 * q; }
  // Row statistics to shared memory (16 each).
  __device__ __forceinline__ void stats(float* ms, float* ls, int lane) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float t = l[r];
      t += __shfl_xor_sync(kFullMask, t, 1);
      t += __shfl_xor_sync(kFullMask, t, 2);
      if ((lane & 3) == 0) {
        ms[lane / 4 + 8 * r] = m[r];
        ls[lane / 4 + 8 * r] = t;
      }
    }
  }
};

// kH of the 16 heads that the warp's buffers have room for.
template <int D, int kH, int kMT>
struct Consumer<float, D, kH, kMT> {
  using S = Shape<float, D, kMT, kH>;
  static constexpr int kL = kH / 4;    // heads per lane in the scores
  static constexpr int kW = D / 32;    // result columns per lane
  uint32_t q_addr;
  float m[kL], l[kL];        // heads kL (lane / 8) ..; l: this lane's key (lane % 8) only
  float acc[S::kAcc];        // [kH heads][kW]

  static __device__ __forceinline__ int row(int i, int) { return i / kW; }
  static __device__ __forceinline__ int col(int i, int lane) { return lane * kW + i % kW; }
  __device__ __forceinline__ void start(uint32_t q_smem, int) {
    q_addr = q_smem;
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < S::kAcc; ++i) acc[i] = 0.f;
  }
  __device__ __forceinline__ static float4 lds4(uint32_t addr) {
    const uint4 v = lds128(addr);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                       __uint_as_float(v.w));
  }
  // p: this warp's 8 keys x 16 heads (and 16 factors) in shared memory.
  __device__ __forceinline__ void tile(uint32_t k_addr, uint32_t v_addr, int group, int lane,
                                       float scale, uint32_t vis, const DecodeArgs& d, float* p) {
    const int t = lane & 7, hg = lane >> 3;
    const uint32_t box = (uint32_t)d.box_rows * 128u;
    const uint32_t krow = k_addr + box_row(group * 8 + t, d.box_rows, d.box_shift, S::kSubs);
    // Two sums per head, over 128 bytes of the row at a time: the reads of a
    // step are in flight together.
    float s[kL] = {}, s1[kL] = {};
#pragma unroll(kL == 1 ? 2 : 1)
    for (int c = 0; c < S::kSubs; ++c) {
      const uint32_t at = krow + (uint32_t)c * box;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 kx = lds4(at + (uint32_t)((k ^ t) << 4));
#pragma unroll
        for (int i = 0; i < kL; ++i) {
          const float4 qx = lds4(q_addr + (uint32_t)((hg * kL + i) * S::kQRow + c * 128 + k * 16));
          float& z = k & 1 ? s1[i] : s[i];
          z = fmaf(qx.x, kx.x, z);
          z = fmaf(qx.y, kx.y, z);
          z = fmaf(qx.z, kx.z, z);
          z = fmaf(qx.w, kx.w, z);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kL; ++i) s[i] += s1[i];
    const bool seen = (vis >> t) & 1u;
    float top[kL];
    bool moved = false;
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      s[i] = seen ? s[i] * scale : -INFINITY;
      top[i] = s[i];
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1)
        top[i] = fmaxf(top[i], __shfl_xor_sync(kFullMask, top[i], o));
      top[i] = fmaxf(top[i], m[i]);
      moved |= top[i] != m[i];
    }
    moved = __any_sync(kFullMask, moved);
    __syncwarp();                                // the last tile's p has been read
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      const float base = top[i] == -INFINITY ? 0.f : top[i];
      if (moved) {
        const float keep = top[i] == -INFINITY ? 0.f : exp2_approx(m[i] - top[i]);
        l[i] *= keep;
        if (t == 0) p[128 + hg * kL + i] = keep;
        m[i] = top[i];
      }
      const float e = exp2_approx(s[i] - base);
      l[i] += e;
      p[t * 16 + hg * kL + i] = e;
    }
    __syncwarp();
    if (moved) {
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const float keep = p[128 + h];
#pragma unroll
        for (int w = 0; w < kW; ++w) acc[h * kW + w] *= keep;
      }
    }
    const uint32_t p_addr = smem_addr(p);
    const bool whole = (vis & 0xffu) == 0xffu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t vrow = v_addr + box_row(group * 8 + j, d.box_rows, d.box_shift, S::kSubs);
      float vx[kW];
      if constexpr (kW == 4) {
        const float4 v4 = lds4(vrow + (uint32_t)(lane >> 3) * box + (uint32_t)(((lane & 7) ^ j) << 4));
        vx[0] = v4.x; vx[1] = v4.y; vx[2] = v4.z; vx[3] = v4.w;
      } else {
        const uint32_t at = vrow + (uint32_t)(lane >> 4) * box +
                            (uint32_t)((((lane >> 1) & 7) ^ j) << 4) + (uint32_t)(lane & 1) * 8;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(vx[0]), "=f"(vx[1]) : "r"(at));
      }
      if (!whole && !((vis >> j) & 1u)) {        // not seen: its value may be anything
#pragma unroll
        for (int w = 0; w < kW; ++w) vx[w] = 0.f;
      }
#pragma unroll
      for (int h = 0; h < kH; h += 4) {
        const float4 e = lds4(p_addr + (uint32_t)(j * 16 + h) * 4);
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          acc[(h + 0) * kW + w] = fmaf(e.x, vx[w], acc[(h + 0) * kW + w]);
          acc[(h + 1) * kW + w] = fmaf(e.y, vx[w], acc[(h + 1) * kW + w]);
          acc[(h + 2) * kW + w] = fmaf(e.z, vx[w], acc[(h + 2) * kW + w]);
          acc[(h + 3) * kW + w] = fmaf(e.w, vx[w], acc[(h + 3) * kW + w]);
        }
      }
    }
  }
  static constexpr int kShareRows = S::kShare < kW ? 1 : S::kShare / kW;
  static constexpr __device__ __forceinline__ int share_of(int e) { return e / kW; }
  static __device__ __forceinline__ int share_row(int first, int q, int) { return first / kW + q; }
  __device__ __forceinline__ void stats(float* ms, float* ls, int lane) {
#pragma unroll
    for (int i = 0; i < kL; ++i) {
      float t = l[i];
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) t += __shfl_xor_sync(kFullMask, t, o);
      if ((lane & 7) == 0) {
        ms[(lane >> 3) * kL + i] = m[i];
        ls[(lane >> 3) * kL + i] = t;
      }
    }
  }
};

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16(a, b);
}
__device__ __forceinline__ void store_pair(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}

// 1 / (l + e^(sink - m)) in the scale of m, for a row with running maximum m
// and sum l: out = o * that.
__device__ __forceinline__ float finish(const AttnArgs& a, int head, float m, float l) {
  float f = 1.f;
  if (a.sink_logits != nullptr) {
    const float z = __ldg(a.sink_logits + head) * kLog2e;
    const float top = fmaxf(m, z), base = top == -INFINITY ? 0.f : top;
    f = exp2_approx(m - base);
    l = l * f + exp2_approx(z - base);
  }
  return l == 0.f ? 0.f : f / l;
}

template <typename Tok, int D, int kMT, int kH>
__global__ void __launch_bounds__(32 * (1 + Shape<Tok, D, kMT, kH>::kGroups * kMT), 1)
attention_decode_kernel(const __grid_constant__ DecodeMaps maps, const DecodeArgs d) {
  using S = Shape<Tok, D, kMT, kH>;
  constexpr int kThreads = 32 * (1 + S::kGroups * kMT), kConsumers = kThreads - 32;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* ring = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  unsigned char* q_smem = ring + (size_t)S::kStages * 2 * S::kHalf;
  float* merge = reinterpret_cast<float*>(q_smem + kQSlots * 16 * kMT * S::kQRow);
  float* p_smem = merge + (size_t)kMT * S::kGroups * S::kPass * 32;     // float32: p per warp
  constexpr int kPFloats = sizeof(Tok) == 4 ? 144 : 0;
  DecodeShared<kMT, S::kGroups>& sh =
      *reinterpret_cast<DecodeShared<kMT, S::kGroups>*>(p_smem + S::kGroups * kMT * kPFloats);
  const AttnArgs& a = d.a;
  const int warp = __shfl_sync(kFullMask, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    prefetch_tensor_map(&maps.k);
    prefetch_tensor_map(&maps.v);
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], S::kGroups * kMT);
    }
    for (int s = 0; s < kQSlots; ++s) {
      mbar_init(&sh.q_full[s], 1);
      mbar_init(&sh.q_empty[s], S::kGroups * kMT);
    }
    fence_mbar_init();
  }
  pdl_wait();

  // Prefix sums of the sequences' tiles: each thread sums a run of them, then
  // the runs are scanned.
  {
    const int per = (d.num_seqs + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, d.num_seqs), b1 = min(b0 + per, d.num_seqs);
    long long mine = 0;
    int most = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = sequence_len(d, b);
      int lo, st, ft, tiles;
      tiles_of<S::kTile>(a, n, &lo, &st, &ft, &tiles);
      if (blockIdx.x == 0 && __ldg(a.seqs.seq_lens + d.seq0 + b) > n)
        atomicAdd(&a.status[kStatusBadPages], 1ull);
      mine += tiles;
      most = max(most, tiles);
    }
    most = __reduce_max_sync(kFullMask, most);
    if (lane == 0) sh.longest[warp] = most;
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(kFullMask, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) sh.scan[warp] = incl;
    __syncthreads();
    long long run = incl - mine;
    for (int w = 0; w < warp; ++w) run += sh.scan[w];
    for (int b = b0; b < b1; ++b) {
      int lo, st, ft, tiles;
      tiles_of<S::kTile>(a, sequence_len(d, b), &lo, &st, &ft, &tiles);
      sh.prefix[b] = run;
      run += tiles;
    }
    if (b1 == d.num_seqs && b0 < b1) sh.prefix[d.num_seqs] = run;
    __syncthreads();
  }
  const long long total = sh.prefix[d.num_seqs] * d.units_per_seq;
  const long long per = max(divide(total + gridDim.x - 1, gridDim.x), (long long)kMinTiles);
  long long t0 = per * blockIdx.x, t1 = min(t0 + per, total);
  int longest = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) longest = max(longest, sh.longest[w]);
  if (longest <= kWholeTiles) {
    // Whole units: units_per_cta each, and one more for the first CTAs.
    const long long mine = d.units_per_cta * blockIdx.x +
                           min((int)blockIdx.x, d.units_over);
    auto first_tile = [&](long long unit) {
      const int b = (int)divide(unit, d.units_per_seq);
      if (b >= d.num_seqs) return total;
      return sh.prefix[b] * d.units_per_seq + (unit - (long long)b * d.units_per_seq) *
                                                  (sh.prefix[b + 1] - sh.prefix[b]);
    };
    t0 = first_tile(mine);
    t1 = first_tile(mine + d.units_per_cta + ((int)blockIdx.x < d.units_over ? 1 : 0));
  }
  if (t0 >= t1) return;

  if (warp == 0) {
    // ------------------------------------------------------------- producer
    // Each lane copies one box of a tile at most: lane & 15 says which, lane >> 4
    // keys or values. The ids of the next tile's pages are on their way while
    // this one waits for room.
    static_assert(S::kTile / 8 <= 16, "boxes of a tile (pages have 8 slots at least)");
    bool ok = true;
    int stage = 0, slot = 0;
    uint32_t phase = 0, q_phase = 0;
    const uint64_t once = l2_evict_first_policy(), keep = l2_evict_normal_policy();
    const int x = (lane & 15) << d.box_shift, half = lane >> 4;
    const uint32_t box_bytes = (uint32_t)d.box_rows * D * sizeof(Tok);
    const CUtensorMap* map = half == 0 ? &maps.k : &maps.v;
    Walk<S::kTile, kMT> w;
    w.start(d, sh.prefix, t0, lane);
    for (long long t = t0; t < t1 && ok; w.next(d, t1)) {
      const Unit u = w.u;
      const int i0 = (int)(t - w.first), i1 = (int)min((long long)u.tiles, t1 - w.first);
      t = w.first + i1;
      const int* table = a.seqs.page_table + (int64_t)(d.seq0 + u.b) * a.seqs.table_stride;
      // The lane's box of tile i has a key that is seen; *id is its page.
      auto box = [&](int i, int* id, int* s0) {
        const int j0 = (i < u.sink_tiles ? i : u.first_tile + i - u.sink_tiles) * S::kTile;
        const int k0 = j0 + x, k1 = min(k0 + d.box_rows, u.len);
        const bool seen =
            x < S::kTile && k0 < k1 && (k1 > u.lo || k0 < a.sinks);
        if (seen) *id = __ldg(table + (k0 >> a.cache.page_shift));
        *s0 = k0 & (a.cache.page_size - 1);
        return seen;
      };
      int id = 0, s0;
      bool seen = box(i0, &id, &s0);
      ok = mbar_wait_warp(&sh.q_empty[slot], q_phase ^ 1u);
      if (!ok) break;
      if (lane == 0)
        mbar_arrive_expect_tx(&sh.q_full[slot], (uint32_t)(u.rows * D * sizeof(Tok)));
      __syncwarp();
      const Tok* q = static_cast<const Tok*>(a.q) + (int64_t)(d.seq0 + u.b) * a.q_token +
                     (int64_t)u.head0 * a.q_head;
      for (int r = lane; r < u.rows; r += 32)
        bulk_copy_g2s(q_smem + (size_t)(slot * 16 * kMT + r) * S::kQRow, q + r * a.q_head,
                      D * sizeof(Tok), &sh.q_full[slot], keep);
      if (++slot == kQSlots) {
        slot = 0;
        q_phase ^= 1u;
      }
      for (int i = i0; i < i1; ++i) {
        int next_id = 0, next_s0 = 0;
        const bool next_seen = i + 1 < i1 && box(i + 1, &next_id, &next_s0);
        ok = mbar_wait_warp(&sh.empty[stage], phase ^ 1u);
        if (!ok) break;
        const uint32_t boxes = __ballot_sync(0xffffffffu, seen);
        if (lane == 0) {
          if (boxes == 0) mbar_arrive(&sh.full[stage]);
          else mbar_arrive_expect_tx(&sh.full[stage], __popc(boxes) * box_bytes);
        }
        __syncwarp();
        if (seen) {
          // An id out of range reads as zeros (the copy's fill).
          if (half == 0 && (unsigned)id >= (uint64_t)a.cache.num_pages)
            atomicAdd(&a.status[kStatusBadPages], 1ull);
          tma_load_5d(ring + (size_t)stage * 2 * S::kHalf + (size_t)half * S::kHalf +
                          (size_t)x * D * sizeof(Tok),
                      map, 0, s0, 0, u.kvh, id, &sh.full[stage], once);
        }
        seen = next_seen;
        id = next_id;
        s0 = next_s0;
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // No copy may outlive the block, also where a consumer's wait gave up: the
    // last one into every stage and query slot (before a first one, the wait
    // ends at once).
    for (int s = 0; s < S::kStages; ++s)
      ok &= mbar_wait_warp(&sh.full[s], s < stage ? phase : phase ^ 1u);
    for (int s = 0; s < kQSlots; ++s)
      ok &= mbar_wait_warp(&sh.q_full[s], s < slot ? q_phase : q_phase ^ 1u);
    if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
    return;
  }

  // --------------------------------------------------------------- consumers
  // A wait that gives up is recorded; the warp then goes on without waiting,
  // so that every warp still reaches every barrier and the workspace's
  // counters end as they should.
  const int cw = warp - 1, group = cw % S::kGroups, mt = cw / S::kGroups;
  const int bar = 1 + mt;                                   // the warps of 16 heads
  float* buf = merge + (size_t)mt * S::kGroups * S::kPass * 32;
  float* p_warp = p_smem + cw * kPFloats;
  const float scale = a.scale * kLog2e;
  using C = Consumer<Tok, D, kH, kMT>;
  C c;
  bool ok = true;
  int stage = 0, slot = 0;
  uint32_t phase = 0, q_phase = 0;
  Walk<S::kTile, kMT> walk;
  walk.start(d, sh.prefix, t0, lane);
  for (long long t = t0; t < t1; walk.next(d, t1)) {
    const Unit u = walk.u;
    const long long first = walk.first;
    const int i0 = (int)(t - first), i1 = (int)min((long long)u.tiles, t1 - first);
    t = first + i1;
    ok = ok && mbar_wait_warp(&sh.q_full[slot], q_phase);
    c.start(smem_addr(q_smem) + (uint32_t)((slot * kMT + mt) * 16 * S::kQRow), lane);
    if constexpr (sizeof(Tok) == 2) {                       // the queries are in registers now
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_empty[slot]);
    }
    for (int i = i0; i < i1; ++i) {
      const int j0 = (i < u.sink_tiles ? i : u.first_tile + i - u.sink_tiles) * S::kTile;
      uint32_t vis = 0xffffffffu;
      if (!(j0 + S::kTile <= u.len && (j0 >= u.lo || j0 + S::kTile <= a.sinks))) {
        const int key = j0 + group * S::kPer + lane;
        vis = __ballot_sync(kFullMask, lane < S::kPer && key < u.len &&
                                           (key >= u.lo || key < a.sinks));
      }
      ok = ok && mbar_wait_warp(&sh.full[stage], phase);
      const uint32_t at = smem_addr(ring) + (uint32_t)stage * 2 * S::kHalf;
      c.tile(at, at + S::kHalf, group, lane, scale, vis, d, p_warp);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stage]);
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    if constexpr (sizeof(Tok) == 4) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_empty[slot]);
    }
    if (++slot == kQSlots) {
      slot = 0;
      q_phase ^= 1u;
    }

    // The warps' (m, l, o) meet in shared memory, and each warp joins and
    // writes a share of the result.
    const bool whole = i0 == 0 && i1 == u.tiles;
    bar_sync(bar, 32 * S::kGroups);                 // the last unit's have been read
    c.stats(sh.merge_m[mt][group], sh.merge_l[mt][group], lane);
    // Row r: the warps' factors, the common maximum and the sum.
    auto join_row = [&](int r, float (&f)[S::kGroups], float* m) {
      *m = -INFINITY;
#pragma unroll
      for (int k = 0; k < S::kGroups; ++k) *m = fmaxf(*m, sh.merge_m[mt][k][r]);
      const float base = *m == -INFINITY ? 0.f : *m;
      float l = 0.f;
#pragma unroll
      for (int k = 0; k < S::kGroups; ++k) {
        f[k] = exp2_approx(sh.merge_m[mt][k][r] - base);
        l = fmaf(sh.merge_l[mt][k][r], f[k], l);
      }
      return l;
    };
    float* piece = reinterpret_cast<float*>(
        d.pieces + (size_t)(2 * blockIdx.x + (i0 == 0 ? 1 : 0)) * kPieceBytes);
    Tok* unit_out = static_cast<Tok*>(a.out) + ((int64_t)(d.seq0 + u.b) * a.heads + u.head0) * D;
#pragma unroll
    for (int pass = 0; pass < S::kPasses; ++pass) {
      if (pass > 0) bar_sync(bar, 32 * S::kGroups);
#pragma unroll
      for (int i = 0; i < S::kPass; ++i)
        buf[(group * S::kPass + i) * 32 + lane] = c.acc[pass * S::kPass + i];
      bar_sync(bar, 32 * S::kGroups);
      const int mine = group * S::kShare;
      if (mine >= S::kPass) continue;
      const int first_i = pass * S::kPass + mine;
      float f[C::kShareRows][S::kGroups];
      int rr[C::kShareRows];
#pragma unroll
      for (int q = 0; q < C::kShareRows; ++q) {
        const int r = C::share_row(first_i, q, lane);
        rr[q] = mt * 16 + r;
        float m;
        const float l = join_row(r, f[q], &m);
        if (whole) {
          const float inv = rr[q] < u.rows ? finish(a, u.head0 + rr[q], m, l) : 0.f;
#pragma unroll
          for (int k = 0; k < S::kGroups; ++k) f[q][k] *= inv;
        }
      }
#pragma unroll
      for (int e = 0; e < S::kShare; e += 2) {
        const int q = C::share_of(e);
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int k = 0; k < S::kGroups; ++k) {
          x = fmaf(buf[(k * S::kPass + mine + e) * 32 + lane], f[q][k], x);
          y = fmaf(buf[(k * S::kPass + mine + e + 1) * 32 + lane], f[q][k], y);
        }
        const int col = C::col(first_i + e, lane);
        if (rr[q] < u.rows) {
          if (whole) store_pair(unit_out + (int64_t)rr[q] * D + col, x, y);
          else *reinterpret_cast<float2*>(piece + rr[q] * D + col) = make_float2(x, y);
        }
      }
    }
    if (!whole) {
      if (group == 0 && lane < 16 && mt * 16 + lane < u.rows) {
        float f[S::kGroups], m;
        const float l = join_row(lane, f, &m);
        piece[kRowsMax * 128 + mt * 16 + lane] = m;
        piece[kRowsMax * 128 + kRowsMax + mt * 16 + lane] = l;
      }
      __threadfence();
    }
    if (!whole) {
      // The unit's CTAs are those that own its tiles' runs; the first owns
      // the counter. The last to arrive joins.
      const int c_first = (int)divide(first, per),
                c_last = (int)divide(first + u.tiles - 1, per);
      bar_sync(1 + kMT, kConsumers);
      if (cw == 0 && lane == 0)
        sh.last = atomicInc(d.counters + c_first, (unsigned)(c_last - c_first)) ==
                  (unsigned)(c_last - c_first);
      bar_sync(1 + kMT, kConsumers);
      if (sh.last) {
        __threadfence();
        const int n = c_last - c_first + 1;
        auto piece = [&](int k) {
          return reinterpret_cast<const float*>(
              d.pieces + (size_t)(2 * (c_first + k) + (k == 0 ? 1 : 0)) * kPieceBytes);
        };
        // kR rows of the result a warp at a time, their reads in flight
        // together.
        constexpr int kStep = S::kGroups * kMT;
        auto join = [&](auto rows_at_once) {
          constexpr int kR = decltype(rows_at_once)::value;
          for (int r0 = cw; r0 < u.rows; r0 += kStep * kR) {
            int rr[kR];
            float m[kR], l[kR] = {}, o[kR][D / 32] = {};
#pragma unroll
            for (int q = 0; q < kR; ++q) {
              rr[q] = min(r0 + q * kStep, u.rows - 1);
              m[q] = -INFINITY;
            }
            for (int k = lane; k < n; k += 32)
#pragma unroll
              for (int q = 0; q < kR; ++q)
                m[q] = fmaxf(m[q], __ldcg(piece(k) + kRowsMax * 128 + rr[q]));
#pragma unroll
            for (int s = 16; s >= 1; s >>= 1)
#pragma unroll
              for (int q = 0; q < kR; ++q)
                m[q] = fmaxf(m[q], __shfl_xor_sync(kFullMask, m[q], s));
#pragma unroll(kR == 1 ? 4 : 2)
            for (int k = 0; k < n; ++k) {
              const float* pk = piece(k);
#pragma unroll
              for (int q = 0; q < kR; ++q) {
                const float base = m[q] == -INFINITY ? 0.f : m[q];
                const float f = exp2_approx(__ldcg(pk + kRowsMax * 128 + rr[q]) - base);
                l[q] = fmaf(__ldcg(pk + kRowsMax * 128 + kRowsMax + rr[q]), f, l[q]);
                if constexpr (D == 128) {
                  const float4 x = __ldcg(reinterpret_cast<const float4*>(pk + rr[q] * D) + lane);
                  o[q][0] = fmaf(x.x, f, o[q][0]);
                  o[q][1] = fmaf(x.y, f, o[q][1]);
                  o[q][2] = fmaf(x.z, f, o[q][2]);
                  o[q][3] = fmaf(x.w, f, o[q][3]);
                } else {
                  const float2 x = __ldcg(reinterpret_cast<const float2*>(pk + rr[q] * D) + lane);
                  o[q][0] = fmaf(x.x, f, o[q][0]);
                  o[q][1] = fmaf(x.y, f, o[q][1]);
                }
              }
            }
#pragma unroll
            for (int q = 0; q < kR; ++q) {
              if (r0 + q * kStep >= u.rows) break;
              const float inv = finish(a, u.head0 + rr[q], m[q], l[q]);
#pragma unroll
              for (int w = 0; w < D / 32; w += 2)
                store_pair(unit_out + (int64_t)rr[q] * D + lane * (D / 32) + w, o[q][w] * inv,
                           o[q][w + 1] * inv);
            }
          }
        };
        if (kMT > 1 || u.rows <= kStep) join(std::integral_constant<int, 1>());
        else join(std::integral_constant<int, 2>());
      }
    }
  }
  if (!ok && lane == 0) atomicAdd(&a.status[kStatusWaitTimeouts], 1ull);
}

template <typename Tok, int D, int kMT, int kH = 16>
cudaError_t launch(const AttnArgs& a, void* workspace, cudaStream_t stream) {
  using S = Shape<Tok, D, kMT, kH>;
  DecodeArgs d = {};
  d.a = a;
  d.head_blocks = (a.group + 16 * kMT - 1) / (16 * kMT);
  d.units_per_seq = a.cache.kv_heads * d.head_blocks;
  d.box_rows = std::min(a.cache.page_size, S::kTile);
  while ((1 << d.box_shift) < d.box_rows) ++d.box_shift;
  d.counters = decode_counters(workspace);
  d.pieces = static_cast<unsigned char*>(workspace_pieces(workspace));
  DecodeMaps maps;
  if (!kv_tensor_map(a.cache, false, d.box_rows, S::kSubs, &maps.k) ||
      !kv_tensor_map(a.cache, true, d.box_rows, S::kSubs, &maps.v))
    return cudaErrorInvalidValue;
  constexpr size_t smem = 1024 + (size_t)S::kStages * 2 * S::kHalf +
                          (size_t)kQSlots * 16 * kMT * S::kQRow +
                          (size_t)kMT * S::kGroups * S::kPass * 32 * 4 +
                          (sizeof(Tok) == 4 ? (size_t)S::kGroups * kMT * 144 * 4 : 0) +
                          sizeof(DecodeShared<kMT, S::kGroups>);
  static_assert(smem <= 227 * 1024, "shared memory");
  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t err = cudaSuccess;
  std::call_once(once[dev & 63], [&] {
    err = cudaFuncSetAttribute(attention_decode_kernel<Tok, D, kMT, kH>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  });
  if (err != cudaSuccess) return err;
  // No more CTAs than runs of kMinTiles tiles at the longest lengths the page
  // tables could hold.
  const int64_t room = ((int64_t)a.seqs.max_pages << a.cache.page_shift) / S::kTile + 2;
  for (int b = 0; b < a.seqs.num_seqs; b += kMaxSeqs) {
    d.seq0 = b;
    d.num_seqs = std::min(kMaxSeqs, a.seqs.num_seqs - b);
    const int64_t units = (int64_t)d.num_seqs * d.units_per_seq;
    const int64_t most = std::max(units, (units * room + kMinTiles - 1) / kMinTiles);
    const int grid = (int)std::min<int64_t>(std::min(attention_num_sms(), kMaxCtas), most);
    d.units_per_cta = units / grid;
    d.units_over = (int)(units % grid);
    err = launch_after_previous(attention_decode_kernel<Tok, D, kMT, kH>, dim3((unsigned)grid),
                                dim3(32 * (1 + S::kGroups * kMT)), smem, stream, maps, d);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

template <typename Tok, int D>
cudaError_t launch_heads(const AttnArgs& a, void* workspace, cudaStream_t stream) {
  // float32: the CUDA cores' work grows with the heads that a warp carries, so
  // groups of up to 4 and 8 have kernels of their own (24 sequences of up to
  // 3001 keys, 4 heads to a key head, four warps: 130 us with 16 carried, 40
  // with 4; 8 heads to a key head, heads of 128, eight warps: 60 us with 16
  // carried, 41 with 8). Wider groups are blocks of 16 heads.
  if constexpr (sizeof(Tok) == 4) {
    if (a.group <= 4) return launch<Tok, D, 1, 4>(a, workspace, stream);
    if (a.group <= 8) return launch<Tok, D, 1, 8>(a, workspace, stream);
    return launch<Tok, D, 1>(a, workspace, stream);
  } else {
    // bf16: the instruction takes 16 rows whatever the group. Units of 32 heads
    // read a tile once for two blocks of 16: 32 sequences of up to 4096 keys, 32
    // heads to a key head of 128: 28.9 us, as units of 16 heads 37.0; of up to
    // 8192 keys, 128 heads to a key head: 72.5 and 83.9. (A handful of short
    // sequences loses by it, 15.3 against 11.8 us for four of up to 1000 keys.)
    return a.group <= 16 ? launch<Tok, D, 1>(a, workspace, stream)
                         : launch<Tok, D, 2>(a, workspace, stream);
  }
}

}  // namespace

// The keys (or values) as (128 bytes, slot, 128-byte column of the row, head,
// page), copied box_rows slots and box_subs columns of one head of one page at a
// time: each column lands as box_rows rows of 128 bytes, swizzled. A dimension of one element
// needs no stride; 16 stands in.
bool kv_tensor_map(const KvCacheView& c, bool values, int box_rows, int box_subs,
                   CUtensorMap* map) {
  auto enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder());
  if (enc == nullptr) return false;
  const bool bf16 = c.token_dtype == kTokenBF16;
  const cuuint64_t es = bf16 ? 2 : 4, sub = 128 / es, subs = c.head_dim / sub;
  const int64_t page = values ? c.v_page : c.k_page, head = values ? c.v_head : c.k_head,
                slot = values ? c.v_slot : c.k_slot;
  const cuuint64_t dims[5] = {sub, (cuuint64_t)c.page_size, subs, (cuuint64_t)c.kv_heads,
                              (cuuint64_t)c.num_pages};
  const cuuint64_t strides[4] = {(cuuint64_t)slot * es, 128,
                                 c.kv_heads > 1 ? (cuuint64_t)head * es : 16,
                                 c.num_pages > 1 ? (cuuint64_t)page * es : 16};
  const cuuint32_t box[5] = {(cuuint32_t)sub, (cuuint32_t)box_rows, (cuuint32_t)box_subs, 1, 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 5,
             values ? c.v : c.k, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int attention_num_sms() {
  static int cached[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return 152;
  if (cached[dev] == 0) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cached[dev] = n > 0 ? n : 152;
  }
  return cached[dev];
}

cudaError_t launch_attention_decode(const AttnArgs& a, void* workspace, cudaStream_t stream) {
  if (a.cache.token_dtype == kTokenBF16)
    return a.cache.head_dim == 64 ? launch_heads<__nv_bfloat16, 64>(a, workspace, stream)
                                  : launch_heads<__nv_bfloat16, 128>(a, workspace, stream);
  return a.cache.head_dim == 64 ? launch_heads<float, 64>(a, workspace, stream)
                                : launch_heads<float, 128>(a, workspace, stream);
}

}  // namespace mxfp4el

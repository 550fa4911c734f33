// route_experts.cu -- experts and mixture weights from router logits
// (include/mxfp4el_quantized.h): softmax or sigmoid scores, a bias that only
// steers the choice, groups of experts, the K highest, normalised weights.
//
// One warp per token. The choice is float64's: float32 scores of different
// experts often fall together next to the border of the top K, and then the
// selection would depend on the last bit of an exponential. Float64 is slow
// here (all tokens in float64 took 1237 us for 32768 x 384, 165 times what
// reading the logits takes), so a token is first ranked in float32, which
// bounds the error of every choice, and what the bound does not decide is
// decided in float64: the order of the few candidates, or, where that does not
// settle it, the whole token.
//
// In float32 (route_fast) every lane holds E/32 choices as order-preserving
// integers. The (K+1)-th largest of the 32 lanes' maxima is at most the
// (K+1)-th largest choice, so the choices from there up are candidates: a few
// more than K while K is well below 32. They are gathered to one lane each and
// ranked by counting; a token with more than 32 of them goes to float64 as a whole.
// That bounds the speed from some 16 picks on (32768 x 384, sigmoid with a bias): 8
// picks 28 us, 12 31, 16 53, 18 119, 20 386, 24 819, 32 801.
// 32768 x 384 with a bias: 28 to 30 us against 7.8 us for reading the logits,
// 690 instructions a token at 70 % of the issue rate (38 us and 840 with both
// kinds of score in one kernel, 48 us and 1120 with a NaN check per expert
// besides).
#include <algorithm>

#include "common.cuh"
#include "quant.h"

namespace mxfp4el {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// exp(logit - top) for a softmax whose largest logit is `top`: an expert that
// has the largest logit counts 1, also where it is infinite; NaN counts 0.
__device__ __forceinline__ double softmax_term(float logit, float top) {
  return logit == top ? 1.0 : logit < top ? exp((double)logit - (double)top) : 0.0;
}

// A double as an unsigned integer of the same order, at least 1; 0 for NaN.
// (Comparisons of doubles go through the float64 pipe, which is slow.)
__device__ __forceinline__ unsigned long long order_key(double v) {
  const long long u = __double_as_longlong(v + 0.0);
  return v == v ? (unsigned long long)u ^ ((unsigned long long)(u >> 63) | (1ull << 63)) : 0ull;
}

// The highest key of the warp, and the lowest index that has it; -1 where every
// key is 0.
__device__ __forceinline__ int warp_best(unsigned long long key, int index) {
  const unsigned hi = __reduce_max_sync(kFullMask, (unsigned)(key >> 32));
  const bool in = (unsigned)(key >> 32) == hi;
  const unsigned lo = __reduce_max_sync(kFullMask, in ? (unsigned)key : 0u);
  if ((hi | lo) == 0u) return -1;
  return (int)__reduce_min_sync(kFullMask, in && (unsigned)key == lo ? (unsigned)index : ~0u);
}

// One token by one warp, in float64. scratch: E doubles of shared memory.
template <typename Tok>
__device__ __noinline__ void route_token(const RouteArgs& a, const Tok* row, double* scratch,
                                         int64_t t) {
  const int lane = threadIdx.x & 31;
  unsigned long long* key = reinterpret_cast<unsigned long long*>(scratch);
  float top = -INFINITY;
  double inv = 1.0;
  if (a.softmax) {
    double sum = 0.0;
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, to_f32(row[e]));   // NaN loses
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
    for (int e = lane; e < a.E; e += 32) {
      scratch[e] = softmax_term(to_f32(row[e]), top);
      sum += scratch[e];
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
    inv = 1.0 / sum;
  }
  auto score_of = [&](float logit) {
    return a.softmax ? softmax_term(logit, top) * inv : 1.0 / (1.0 + exp(-(double)logit));
  };
  // A choice that is NaN cannot be taken; nor, later on, one that is 0.
  for (int e = lane; e < a.E; e += 32) {
    const float l = to_f32(row[e]);
    const double score = a.softmax ? scratch[e] * inv : score_of(l);
    const double c = l == l ? score + (a.bias != nullptr ? (double)a.bias[e] : 0.0) : (double)NAN;
    if (a.groups > 1) scratch[e] = c;
    else key[e] = order_key(a.bias != nullptr || !(c == c) ? c : (double)l);
  }
  __syncwarp();
  if (a.groups > 1) {
    double v = (double)NAN;
    if (lane < a.groups) {
      double b0 = 0.0, b1 = 0.0;
      int n = 0;
      for (int j = 0; j < a.group_size; ++j) {
        const double c = scratch[lane * a.group_size + j];
        if (!(c == c)) continue;
        if (n == 0 || c > b0) {
          b1 = b0;
          b0 = c;
        } else if (n == 1 || c > b1) {
          b1 = c;
        }
        ++n;
      }
      if (n > 0) v = a.group_best > 1 && n > 1 ? b0 + b1 : b0;
    }
    unsigned kept = 0u;
    unsigned long long mine = order_key(v);
    for (int i = 0; i < a.top_groups; ++i) {
      const int g = warp_best(mine, lane);
      if (g < 0) break;
      kept |= 1u << g;
      if (lane == g) mine = 0ull;
    }
    __syncwarp();
    for (int e = lane; e < a.E; e += 32) {
      const double c = scratch[e];
      const bool in = (kept >> (e / a.group_size) & 1u) != 0u && c == c;
      key[e] = in ? order_key(a.bias != nullptr ? c : (double)to_f32(row[e])) : 0ull;
    }
    __syncwarp();
  }
  int pick = -1;                                   // lane k: the k-th pick
  for (int k = 0; k < a.K; ++k) {
    unsigned long long best = 0ull;
    int at = 0;
    for (int e = lane; e < a.E; e += 32)
      if (key[e] > best) {
        best = key[e];
        at = e;
      }
    const int e = warp_best(best, at);
    if (e < 0) break;
    if (lane == k) pick = e;
    if (lane == (e & 31)) key[e] = 0ull;
    __syncwarp();
  }
  double w = pick >= 0 ? score_of(to_f32(row[pick])) : 0.0;
  if (a.normalize) {
    double total = w;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
    w /= total + 1e-20;
  }
  if (lane < a.K) {
    a.sel[t * a.K + lane] = pick;
    a.p[t * a.K + lane] = (float)(w * a.scaling);
  }
  __syncwarp();
}

// A float as an unsigned integer of the same order. -0 must have been turned
// to +0 before; NaN as arithmetic makes it (positive) is beyond infinity.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int)~k >> 31) | 0x80000000u));
}
constexpr uint32_t kInfKey = 0xff800000u;       // order_key(+infinity)

__device__ __forceinline__ float exp_approx(float x) {   // 2^(x log2 e), ex2.approx
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The kept groups of one token as a bit mask. choice: the warp's E choices, or
// with by_logit (one expert stands for its group, no bias) the logits, which
// rank as the choices do but for choices that round to the same number (NaN: not
// to be taken). *sure: no other group's sum can be as large as a kept one's, each
// sum being off by the two choices' error `err`, the roundings of those choices and
// its own. Choices of opposite sign may be far larger than their sum, so their
// roundings go by |best| + |second|: half an ulp (2^-24) for the choices, at most
// that much again for the sum and once more for the border worked out here, under
// 2^-22 of it together. score: of a logit.
template <typename Score>
__device__ __forceinline__ unsigned route_groups(const RouteArgs& a, const float* choice,
                                                 bool by_logit, float err, Score score,
                                                 bool* sure) {
  const int lane = threadIdx.x & 31;
  // `lanes` neighbouring lanes (a power of two) share a group.
  const int lanes = 1 << (31 - __clz(32 / a.groups));
  const int g = lane / lanes;
  float b0 = -INFINITY, b1 = -INFINITY;
  int n = 0;
  if (g < a.groups) {
    for (int j = lane % lanes; j < a.group_size; j += lanes) {
      const float c = choice[g * a.group_size + j];
      if (c == c) {
        b1 = fmaxf(b1, fminf(b0, c));
        b0 = fmaxf(b0, c);
        ++n;
      }
    }
  }
  for (int o = lanes >> 1; o >= 1; o >>= 1) {
    const float c0 = __shfl_xor_sync(kFullMask, b0, o), c1 = __shfl_xor_sync(kFullMask, b1, o);
    n += __shfl_xor_sync(kFullMask, n, o);
    b1 = fmaxf(fminf(b0, c0), fmaxf(b1, c1));
    b0 = fmaxf(b0, c0);
  }
  float v = n == 0 ? NAN : a.group_best > 1 && n > 1 ? b0 + b1 : b0;
  v = __shfl_sync(kFullMask, v, min(lane * lanes, 31));      // lane g: group g
  if (lane >= a.groups) v = NAN;
  int rank = 0;
  for (int i = 0; i < a.groups; ++i) {
    const float u = __shfl_sync(kFullMask, v, i);
    if (u > v || (u == v && i < lane)) ++rank;
  }
  const bool valid = v == v, in = valid && rank < a.top_groups;
  const unsigned kept = __ballot_sync(kFullMask, in);
  if (!by_logit) {
    // An infinite choice has no rounding (experts may be kept out by -infinity);
    // finite ones whose sum passes float32 say nothing.
    float size = fabsf(b0) < INFINITY ? fabsf(b0) : 0.f;
    if (a.group_best > 1 && fabsf(b1) < INFINITY) size += fabsf(b1);
    size = __shfl_sync(kFullMask, size, min(lane * lanes, 31));
    const float off = 2.f * err + size * 0x1p-22f;
    const float low = off < INFINITY ? v - off : -INFINITY;
    const float high = off < INFINITY ? v + off : INFINITY;
    const uint32_t lo = __reduce_min_sync(kFullMask, in ? order_key(low + 0.f) : 0xffffffffu);
    const uint32_t hi = __reduce_max_sync(kFullMask, valid && !in ? order_key(high + 0.f) : 0u);
    *sure = lo > hi;
    return kept;
  }
  const uint32_t k = valid ? order_key(v) : 0u;
  const uint32_t lo = __reduce_min_sync(kFullMask, in ? k : 0xffffffffu);
  const uint32_t hi = __reduce_max_sync(kFullMask, valid && !in ? k : 0u);
  auto apart = [&](uint32_t upper, uint32_t lower) {
    return score(key_value(upper)) - score(key_value(lower)) > 4.f * err;
  };
  if (hi != 0u && kept != 0u) {
    if (lo != hi) {
      *sure = apart(lo, hi);
    } else {
      // Groups of the border's very logit are true ties and go by index; the
      // others have to be above or below them for certain.
      const uint32_t up = __reduce_min_sync(kFullMask, in && k > lo ? k : 0xffffffffu);
      const uint32_t down = __reduce_max_sync(kFullMask, valid && !in && k < lo ? k : 0u);
      *sure = (up == 0xffffffffu || apart(up, lo)) && (down == 0u || apart(lo, down));
    }
  }
  return kept;
}

// One token by one warp in float32. scratch: at least max(E, 32) floats of
// the warp. False, with nothing written, where float32 cannot decide it.
// kFull: E is 32 kPer.
template <int kPer, bool kFull, bool kSoftmax, typename Tok>
__device__ __forceinline__ bool route_fast(const RouteArgs& a, const Tok* row, float* scratch,
                                           int64_t t) {
  const int lane = threadIdx.x & 31;
  const bool by_choice = a.bias != nullptr;
  // Groups by their best expert alone, without a bias: logits rank them too.
  const bool by_logit = !by_choice && (a.group_best == 1 || a.group_size == 1);
  uint32_t key[kPer];                              // expert 32 i + lane; 0: none
  float top = 0.f, inv = 1.f;
  // An error bound of every score (the bias adds half an ulp of the choice).
  // Sigmoid, in units of 2^-23: the exponential's relative error is 0.63 |l| (the
  // product with log2 e) + 1.41 (ex2.approx), which the score sees times e /
  // (1 + e)^2, 0.41 at most over all l; the sum adds 0.5, the reciprocal 0.5
  // (1 ulp of at most 2^-24), and what flushes to 0 is under 2^-126. Softmax,
  // in units of the largest score 1/sum and 2^-23: the exponential 1 (expf), the
  // same for the sum's terms, kPer + 5 half ulps of their additions, the
  // reciprocal and the product 1: at most 8 for kPer <= 4, 16 for 16, 32 for 32.
  float err = 0x1p-22f;
  auto in_range = [&](int i) { return kFull || 32 * i + lane < a.E; };
  auto choice_of = [&](float l, int e) {
    const float c = kSoftmax ? expf(l - top) * inv : rcp_approx(1.f + exp_approx(-l));
    return by_choice ? c + a.bias[e] : c;
  };
  {
    float l[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) l[i] = in_range(i) ? to_f32(row[32 * i + lane]) : -INFINITY;
    if constexpr (kSoftmax) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) m = max(m, order_key(l[i] + 0.f));
      m = __reduce_max_sync(kFullMask, m);
      top = key_value(m);
      if (!(fabsf(top) < INFINITY)) return false;  // infinite or NaN
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum += expf(l[i] - top);
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
      inv = 1.f / sum;
      err = inv * (kPer <= 4 ? 0x1p-20f : kPer <= 16 ? 0x1p-19f : 0x1p-18f);
    }
    if (by_choice) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float c = in_range(i) ? choice_of(l[i], 32 * i + lane) + 0.f : 0.f;
        if (a.groups > 1 && in_range(i)) scratch[32 * i + lane] = c;
        key[i] = in_range(i) ? order_key(c) : 0u;
      }
    } else {                                       // the logits' own order
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (a.groups > 1 && in_range(i))
          scratch[32 * i + lane] = by_logit ? l[i] + 0.f : choice_of(l[i], 32 * i + lane);
        key[i] = in_range(i) ? order_key(l[i] + 0.f) : 0u;
      }
    }
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = max(m, key[i]);
  if (__any_sync(kFullMask, m > kInfKey)) return false;      // a NaN among them
  if (a.groups > 1) {
    __syncwarp();
    bool sure = true;
    const unsigned kept =
        route_groups(a, scratch, by_logit, err, [&](float l) { return choice_of(l, 0); }, &sure);
    if (!sure) return false;
    // e / group_size by a multiplication: exact for e * group_size < 2^20.
    const uint32_t mul = ((1u << 20) + a.group_size - 1) / a.group_size;
    m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (!(kept >> ((32 * i + lane) * mul >> 20) & 1u)) key[i] = 0u;
      m = max(m, key[i]);
    }
    __syncwarp();
  }
  // The border: the (K+1)-th largest of the lanes' maxima (sorted, highest
  // first), or 1 where fewer lanes have one: every expert.
#pragma unroll
  for (int k = 2; k <= 32; k <<= 1) {
#pragma unroll
    for (int j = k >> 1; j >= 1; j >>= 1) {
      const uint32_t o = __shfl_xor_sync(kFullMask, m, j);
      const bool larger = ((lane & j) == 0) == ((lane & k) == 0);
      m = larger ? max(m, o) : min(m, o);
    }
  }
  uint32_t border = a.K < 32 ? __shfl_sync(kFullMask, m, a.K) : 0u;
  border = max(border, 1u);
  if (by_choice && border > 1u) {                  // what the error may hide
    const float c = key_value(border);
    if (!(fabsf(c) < 1e30f)) return false;
    border = order_key(c - 2.f * (err + fabsf(c) * 0x1p-23f) + 0.f);
  }
  // Candidates, one per lane: every lane hands over its own, one at a time.
  unsigned mine = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) mine |= key[i] >= border ? 1u << i : 0u;
  int* cid = reinterpret_cast<int*>(scratch);
  int n = 0;
  for (;;) {
    const unsigned b = __ballot_sync(kFullMask, mine != 0u);
    if (b == 0u) break;
    const int at = n + __popc(b & ((1u << lane) - 1u));
    n += __popc(b);
    if (n > 32) return false;
    if (mine != 0u) {
      cid[at] = 32 * (__ffs((int)mine) - 1) + lane;
      mine &= mine - 1u;
    }
  }
  __syncwarp();
  const int id = lane < n ? cid[lane] : 0x7fffffff;
  const float logit = lane < n ? to_f32(row[id]) : 0.f;
  uint32_t k = 0u;
  if (lane < n) k = order_key((by_choice ? choice_of(logit, id) : logit) + 0.f);
  __syncwarp();
  int rank = 0;
#pragma unroll 4
  for (int i = 0; i < n; ++i) rank += __shfl_sync(kFullMask, k, i) > k ? 1 : 0;
  const unsigned same = __match_any_sync(kFullMask, k);
  if (__any_sync(kFullMask, lane < n && same != 1u << lane)) {
    for (int i = 0; i < n; ++i) {                  // equal ones go by index
      const int ui = __shfl_sync(kFullMask, id, i);
      if ((same >> i & 1u) && ui < id) ++rank;
    }
  }
  if (by_choice) {
    // Neighbours in rank that are closer than the error, and not equal for
    // having the same logit and bias: rank the candidates in float64. The
    // neighbours to look at end at rank K, or, where equal ones share the border,
    // behind the last of those: any of them may stand at rank K - 1.
    if (lane < n) cid[rank] = lane;
    __syncwarp();
    const int at0 = cid[min(lane, max(n, 1) - 1)], at1 = cid[min(lane + 1, max(n, 1) - 1)];
    const float c = key_value(k);
    const float c0 = __shfl_sync(kFullMask, c, at0), c1 = __shfl_sync(kFullMask, c, at1);
    const bool close =
        lane + 1 < n && !(c0 - c1 > 2.f * err + (fabsf(c0) + fabsf(c1)) * 0x1p-23f);
    if (__any_sync(kFullMask, close && lane < a.K)) {
      const float b = lane < n ? a.bias[id] : 0.f;
      const float l0 = __shfl_sync(kFullMask, logit, at0), l1 = __shfl_sync(kFullMask, logit, at1);
      const float b0 = __shfl_sync(kFullMask, b, at0), b1 = __shfl_sync(kFullMask, b, at1);
      const bool equal = l0 == l1 && b0 == b1;
      // The first pair from rank K - 1 on that is no tie (lane 31 has no pair).
      const unsigned ties = __ballot_sync(kFullMask, close && equal) >> (a.K - 1);
      const int last = a.K - 2 + __ffs((int)~ties);
      if (__any_sync(kFullMask, close && !equal && lane <= last)) {
        if (kSoftmax) return false;                // the sum is needed in float64 too
        const double d = lane < n ? 1.0 / (1.0 + exp(-(double)logit)) + (double)b : 0.0;
        rank = 0;
        for (int i = 0; i < n; ++i) {
          const double u = __shfl_sync(kFullMask, d, i);
          const int ui = __shfl_sync(kFullMask, id, i);
          if (u > d || (u == d && ui < id)) ++rank;
        }
      }
    }
  }
  // Weights in float32: an exponential, the picks' sum and a quotient, 5.4e-8 off in
  // norm (2^-18 relative at most). Sum and quotient in float64 would give 4.5e-8,
  // the scores too 2.8e-8, half an ulp; but float64 instructions are so few a cycle
  // that 32768 x 384 would take 66 and 109 us for 28.
  const bool picked = lane < n && rank < a.K;
  float w = 0.f;
  if (picked) {
    if constexpr (kSoftmax) {
      // d + rest is logit - top exactly: d alone is off by half an ulp, which is
      // many of the exponential where d is large.
      const float d = logit - top, back = d - logit;
      const float rest = (logit - (d - back)) - (top + back);
      const float z = expf(d);
      w = z > 0.f ? fmaf(z, rest, z) * inv : 0.f;      // rest is NaN for a logit of -infinity
    } else {
      const float z = expf(-fabsf(logit));         // no overflow, and small scores keep their bits
      w = (logit >= 0.f ? 1.f : z) / (1.f + z);
    }
  }
  if (a.normalize) {
    float total = w;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(kFullMask, total, o);
    w /= total + 1e-20f;
  }
  if (picked) {
    a.sel[t * a.K + rank] = id;
    a.p[t * a.K + rank] = w * a.scaling;
  }
  if (lane >= n && lane < a.K) {                   // fewer experts than K
    a.sel[t * a.K + lane] = -1;
    a.p[t * a.K + lane] = 0.f;
  }
  return true;
}

// Bytes of shared memory per warp: E doubles for a token in float64, or the
// float32 choices and the candidates' ids.
__host__ __device__ __forceinline__ size_t scratch_bytes(int E) {
  return (size_t)(E > 33 ? E : 33) * sizeof(double);
}

template <int kPer, bool kFull, bool kSoftmax, typename Tok>
__global__ void __launch_bounds__(kThreads) route_experts_kernel(const RouteArgs a) {
  extern __shared__ double route_choice[];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5;
  double* scratch = route_choice + warp * (scratch_bytes(a.E) / sizeof(double));
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T;
       t += (int64_t)gridDim.x * kWarps) {
    const Tok* row = static_cast<const Tok*>(a.logits) + t * a.row_stride;
    const bool done = route_fast<kPer, kFull, kSoftmax>(a, row, reinterpret_cast<float*>(scratch), t);
    __syncwarp();
    if (!done) route_token(a, row, scratch, t);
    __syncwarp();
  }
}

// The fewest choices a lane that hold E experts, of the widths built; without the
// range checks where E fills them. 32768 tokens, sigmoid with a bias, 8 picks: 384
// experts 29 us without checks, 33 with them, 38 with 16 choices a lane and checks;
// 320 experts 32 us with 12 choices a lane, 37 with 16; 1024 experts 48 against 76.
template <int kPer, bool kSoftmax, typename Tok>
auto kernel_of_width(int E) {
  return E == 32 * kPer ? route_experts_kernel<kPer, true, kSoftmax, Tok>
                        : route_experts_kernel<kPer, false, kSoftmax, Tok>;
}
template <bool kSoftmax, typename Tok>
auto kernel_for(int E) {
  return E <= 32    ? kernel_of_width<1, kSoftmax, Tok>(E)
         : E <= 64  ? kernel_of_width<2, kSoftmax, Tok>(E)
         : E <= 128 ? kernel_of_width<4, kSoftmax, Tok>(E)
         : E <= 256 ? kernel_of_width<8, kSoftmax, Tok>(E)
         : E <= 384 ? kernel_of_width<12, kSoftmax, Tok>(E)
         : E <= 512 ? kernel_of_width<16, kSoftmax, Tok>(E)
                    : kernel_of_width<32, kSoftmax, Tok>(E);
}

}  // namespace

cudaError_t launch_route_experts(const RouteArgs& a, int dtype, cudaStream_t stream) {
  const unsigned blocks = (unsigned)std::min<int64_t>((a.T + kWarps - 1) / kWarps, 1 << 20);
  const size_t smem = kWarps * scratch_bytes(a.E);
  auto kernel = dtype == kTokenBF16
                    ? (a.softmax ? kernel_for<true, __nv_bfloat16>(a.E)
                                 : kernel_for<false, __nv_bfloat16>(a.E))
                    : (a.softmax ? kernel_for<true, float>(a.E) : kernel_for<false, float>(a.E));
  // Always the most that any call needs: a call of fewer experts on another thread
  // would otherwise take it back between this line and the launch.
  if (smem > 48 * 1024) {
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(kWarps * scratch_bytes(kRouteMaxExperts)));
    if (err != cudaSuccess) return err;
  }
  kernel<<<blocks, kThreads, smem, stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace mxfp4el

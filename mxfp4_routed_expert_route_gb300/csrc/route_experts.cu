// route_experts.cu -- experts and mixture weights from router logits
// (include/mxfp4el_quantized.h): softmax or sigmoid scores, a bias that only
// steers the choice, groups of experts, the K highest, normalised weights.
//
// One warp per token. The choice is decided in float64: float32 scores of
// different experts often fall together next to the border of the top K, and
// then the selection would depend on the last bit of an exponential.
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

// Lane and value of the highest value among lanes with `has`, ties to the lower
// index; index -1 where no lane has one.
struct Best {
  double value;
  int index;
};
__device__ __forceinline__ Best warp_best(Best b) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    const double v = __shfl_xor_sync(kFullMask, b.value, o);
    const int i = __shfl_xor_sync(kFullMask, b.index, o);
    if (i >= 0 && (b.index < 0 || v > b.value || (v == b.value && i < b.index))) b = {v, i};
  }
  return b;
}

// One token by one warp, in float64. choice: E doubles of shared memory.
template <typename Tok>
__device__ void route_token(const RouteArgs& a, const Tok* row, double* choice, int64_t t) {
  const int lane = threadIdx.x & 31;
  float top = -INFINITY;
  double sum = 0.0;
  if (a.softmax) {
    for (int e = lane; e < a.E; e += 32) top = fmaxf(top, to_f32(row[e]));   // NaN loses
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, o));
    for (int e = lane; e < a.E; e += 32) sum += softmax_term(to_f32(row[e]), top);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFullMask, sum, o);
  }
  auto score_of = [&](float logit) {
    return a.softmax ? softmax_term(logit, top) / sum : 1.0 / (1.0 + exp(-(double)logit));
  };
  // NaN marks an expert that cannot be taken (any more).
  for (int e = lane; e < a.E; e += 32) {
    const float l = to_f32(row[e]);
    const double c = score_of(l) + (a.bias != nullptr ? (double)a.bias[e] : 0.0);
    choice[e] = l == l ? c : (double)NAN;
  }
  __syncwarp();
  unsigned kept = ~0u;
  if (a.groups > 1) {
    Best mine = {0.0, -1};
    if (lane < a.groups) {
      double b0 = 0.0, b1 = 0.0;
      int n = 0;
      for (int j = 0; j < a.group_size; ++j) {
        const double c = choice[lane * a.group_size + j];
        if (!(c == c)) continue;
        if (n == 0 || c > b0) {
          b1 = b0;
          b0 = c;
        } else if (n == 1 || c > b1) {
          b1 = c;
        }
        ++n;
      }
      const double v = a.group_best > 1 && n > 1 ? b0 + b1 : b0;
      if (n > 0 && v == v) mine = {v, lane};
    }
    kept = 0u;
    for (int i = 0; i < a.top_groups; ++i) {
      const Best b = warp_best(mine);
      if (b.index < 0) break;
      kept |= 1u << b.index;
      if (lane == b.index) mine.index = -1;
    }
  }
  int pick = -1;                                   // lane k: the k-th pick
  for (int k = 0; k < a.K; ++k) {
    Best mine = {0.0, -1};
    for (int e = lane; e < a.E; e += 32) {
      double v = choice[e];
      if (!(v == v) || (a.groups > 1 && !(kept >> (e / a.group_size) & 1u))) continue;
      if (a.bias == nullptr) v = (double)to_f32(row[e]);
      if (mine.index < 0 || v > mine.value) mine = {v, e};
    }
    const Best b = warp_best(mine);
    if (b.index < 0) break;
    if (lane == k) pick = b.index;
    if (lane == (b.index & 31)) choice[b.index] = (double)NAN;
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

template <typename Tok>
__global__ void __launch_bounds__(kThreads) route_experts_kernel(const RouteArgs a) {
  extern __shared__ double route_choice[];
  pdl_launch_dependents();
  const int warp = threadIdx.x >> 5;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < a.T; t += (int64_t)gridDim.x * kWarps)
    route_token(a, static_cast<const Tok*>(a.logits) + t * a.row_stride,
                route_choice + (size_t)warp * a.E, t);
}

}  // namespace

cudaError_t launch_route_experts(const RouteArgs& a, int dtype, cudaStream_t stream) {
  const unsigned blocks = (unsigned)std::min<int64_t>((a.T + kWarps - 1) / kWarps, 152 * 16);
  const size_t smem = (size_t)kWarps * a.E * sizeof(double);
  auto kernel = dtype == kTokenBF16 ? route_experts_kernel<__nv_bfloat16>
                                    : route_experts_kernel<float>;
  if (smem > 48 * 1024) {
    const cudaError_t err =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
  }
  kernel<<<blocks, kThreads, smem, stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace mxfp4el

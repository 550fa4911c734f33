// quant.h -- declarations shared by the translation units of the operators
// on quantised tokens (include/mxfp4el_quantized.h).
#pragma once

#include "internal.h"

namespace mxfp4el {

constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxPicks = 32;     // one lane of a warp holds each pick
constexpr int kRouteMaxGroups = 32;    // one lane of a warp holds each group

struct RouteArgs {
  const void* logits;
  const float* bias;      // or null
  int64_t row_stride;     // elements
  int64_t T;
  int E, K;
  int groups, group_size, top_groups, group_best;
  bool softmax, normalize;
  float scaling;
  int32_t* sel;
  float* p;
};
cudaError_t launch_route_experts(const RouteArgs& a, int dtype, cudaStream_t stream);

cudaError_t launch_quantize(const void* x, int dtype, int64_t row_stride, int64_t rows, int64_t I,
                            uint8_t* packed, uint8_t* scales, cudaStream_t stream);
cudaError_t launch_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t rows,
                              int64_t I, void* out, int dtype, cudaStream_t stream);

// Products of MXFP4 tokens and MXFP4 weights (gemm_mx.cu). Experts with tokens
// that one call may have (their lists are kept in shared memory).
constexpr int64_t kMxMaxActive = 4096;
// Up to this many pairs the kernel makes its routing lists itself.
constexpr int kMxOwnPairs = 256;

// The shape of a call's units of work.
struct MxPlan {
  bool wide;              // blocks of up to 192 tokens, else 32
  int splits;             // units that share K
  int64_t blocks;         // dense: blocks of tokens; routed: at most this many
  int64_t units;          // blocks x 128-row tiles x splits
  size_t grouped_bytes;   // routed: the token rows in the lists' order (0: the kernel
                          // gathers them itself)
  bool own_lists;         // routed: the kernel routes for itself
};
MxPlan gemm_mx_plan(int64_t T, int64_t E, int64_t I, int64_t O, int64_t K, bool routed);

struct MxGemm {
  const uint8_t *x_packed, *x_scales;   // [T][I/2], [T][I/32]
  const uint8_t *w_packed, *w_scales;   // [E][O][I/2], [E][O][I/32]
  const RoutePlan* plan;                // routing lists, or null: dense (E = 1), or
  const void* sel;                      // shape.own_lists: the ids
  bool sel64;
  int64_t T, E, I, O, K;                // K: picks per token (routed)
  MxPlan shape;                         // gemm_mx_plan() of these sizes
  void* grouped;                        // shape.grouped_bytes of scratch (routed)
  float* part;                          // [pair or token][split][O] (routed, or splits > 1)
  void* out;                            // dense: [T][O] of out_dtype
  int out_dtype;
};
cudaError_t launch_gemm_mx(const MxGemm& g, cudaStream_t stream);

}  // namespace mxfp4el

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

}  // namespace mxfp4el

// quant_api.cu -- the C ABI of the operators on quantised tokens
// (include/mxfp4el_quantized.h): argument checks and launches.
#include <cmath>

#include "../../include/mxfp4_expert_linear.h"
#include "../../include/mxfp4el_quantized.h"
#include "quant.h"

namespace mxfp4el {
namespace {

constexpr int64_t kMaxDim = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxElements = (int64_t)1 << 50;

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  if (an == 0 || bn == 0 || a == nullptr || b == nullptr) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bn && b0 < a0 + an;
}

bool known_dtype(int d) { return d == MXFP4EL_DTYPE_F32 || d == MXFP4EL_DTYPE_BF16; }
size_t size_of(int dtype) { return dtype == MXFP4EL_DTYPE_BF16 ? 2 : 4; }

// Rows `stride` elements apart that span no more than kMaxElements: checked
// without overflow.
bool span_fits(int64_t rows, int64_t stride, int64_t width) {
  return rows <= 1 || (stride <= kMaxElements && (rows - 1) <= (kMaxElements - width) / (stride > 0 ? stride : 1));
}
size_t span_bytes(int64_t rows, int64_t stride, int64_t width, size_t esize) {
  return rows == 0 ? 0 : ((size_t)(rows - 1) * (size_t)stride + (size_t)width) * esize;
}

int status_of(cudaError_t err) { return err == cudaSuccess ? MXFP4EL_OK : MXFP4EL_ERR_CUDA; }

}  // namespace
}  // namespace mxfp4el

using namespace mxfp4el;

extern "C" int mxfp4_route_experts(const void* logits, int dtype, int64_t row_stride,
                                   const float* bias, int64_t T, int64_t E, int64_t K, int score,
                                   int64_t groups, int64_t top_groups, int64_t group_best,
                                   int normalize, float scaling, int32_t* selected_experts,
                                   float* mixture_weights, void* stream) {
  if (!known_dtype(dtype)) return MXFP4EL_ERR_UNSUPPORTED_DTYPE;
  if (T < 0 || E <= 0 || K < 0 || (score != MXFP4EL_SCORE_SOFTMAX && score != MXFP4EL_SCORE_SIGMOID) ||
      groups <= 0 || E % groups != 0 || top_groups <= 0 || top_groups > groups ||
      group_best < 1 || group_best > 2 || K > top_groups * (E / groups) ||
      !std::isfinite(scaling) || (T > 1 && row_stride < E))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (T > kMaxDim || E > kRouteMaxExperts || K > kRouteMaxPicks || groups > kRouteMaxGroups ||
      !span_fits(T, row_stride, E))
    return MXFP4EL_ERR_TOO_LARGE;
  if (T == 0 || K == 0) return MXFP4EL_OK;
  const size_t es = size_of(dtype);
  if (logits == nullptr || selected_experts == nullptr || mixture_weights == nullptr ||
      !aligned(logits, es) || !aligned(bias, 4) || !aligned(selected_experts, 4) ||
      !aligned(mixture_weights, 4))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  const size_t nl = span_bytes(T, row_stride, E, es), nb = (size_t)E * 4, no = (size_t)T * K * 4;
  if (overlaps(selected_experts, no, logits, nl) || overlaps(selected_experts, no, bias, nb) ||
      overlaps(mixture_weights, no, logits, nl) || overlaps(mixture_weights, no, bias, nb) ||
      overlaps(selected_experts, no, mixture_weights, no))
    return MXFP4EL_ERR_ALIAS;
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.row_stride = row_stride;
  a.T = T;
  a.E = (int)E;
  a.K = (int)K;
  a.groups = (int)groups;
  a.group_size = (int)(E / groups);
  a.top_groups = (int)top_groups;
  a.group_best = (int)group_best;
  a.softmax = score == MXFP4EL_SCORE_SOFTMAX;
  a.normalize = normalize != 0;
  a.scaling = scaling;
  a.sel = selected_experts;
  a.p = mixture_weights;
  return status_of(launch_route_experts(a, dtype, static_cast<cudaStream_t>(stream)));
}

extern "C" int mxfp4_quantize(const void* x, int dtype, int64_t row_stride, int64_t rows,
                              int64_t I, uint8_t* packed, uint8_t* scales, void* stream) {
  if (!known_dtype(dtype)) return MXFP4EL_ERR_UNSUPPORTED_DTYPE;
  if (rows < 0 || I <= 0 || I % 32 != 0 || (rows > 1 && row_stride < I))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (I > kMaxDim || rows > kMaxElements / I || !span_fits(rows, row_stride, I))
    return MXFP4EL_ERR_TOO_LARGE;
  if (rows == 0) return MXFP4EL_OK;
  const size_t es = size_of(dtype), G = (size_t)I / 32;
  if (x == nullptr || packed == nullptr || scales == nullptr || !aligned(x, es) ||
      !aligned(packed, 16))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  const size_t nx = span_bytes(rows, row_stride, I, es), np = rows * G * 16, ns = rows * G;
  if (overlaps(packed, np, x, nx) || overlaps(scales, ns, x, nx) ||
      overlaps(packed, np, scales, ns))
    return MXFP4EL_ERR_ALIAS;
  return status_of(launch_quantize(x, dtype, row_stride, rows, I, packed, scales,
                                   static_cast<cudaStream_t>(stream)));
}

extern "C" int mxfp4_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t rows,
                                int64_t I, void* out, int dtype, void* stream) {
  if (!known_dtype(dtype)) return MXFP4EL_ERR_UNSUPPORTED_DTYPE;
  if (rows < 0 || I <= 0 || I % 32 != 0) return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (I > kMaxDim || rows > kMaxElements / I) return MXFP4EL_ERR_TOO_LARGE;
  if (rows == 0) return MXFP4EL_OK;
  if (packed == nullptr || scales == nullptr || out == nullptr || !aligned(packed, 16) ||
      !aligned(out, 16))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  const size_t G = (size_t)I / 32, no = (size_t)rows * I * size_of(dtype);
  if (overlaps(out, no, packed, rows * G * 16) || overlaps(out, no, scales, rows * G))
    return MXFP4EL_ERR_ALIAS;
  return status_of(launch_dequantize(packed, scales, rows, I, out, dtype,
                                     static_cast<cudaStream_t>(stream)));
}

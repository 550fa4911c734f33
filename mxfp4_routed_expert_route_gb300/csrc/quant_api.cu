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

// Values of one expert's matrix: a tensor map's strides end before 2^40 bytes.
constexpr int64_t kMaxMatrix = (int64_t)1 << 40;

// Sizes of a product that every index in the kernels has room for.
bool product_fits(int64_t T, int64_t E, int64_t I, int64_t O, int64_t K) {
  if (T > (1 << 30) || E > kMaxDim || I > kMaxDim / 2 || O > kMaxDim / 2 || K > kMaxDim)
    return false;
  if (K > 0 && T > (1 << 30) / K) return false;         // pair ids are int32
  if (O > 0 && (E > kMaxElements / I / O || O > kMaxMatrix / I)) return false;
  return O == 0 || K == 0 || T * K <= kMaxElements / O;
}

// gemm_mx.cu numbers a call's units in 31 bits, with room for a grid past the last.
bool units_fit(const MxPlan& p) { return p.units <= kMaxDim - (1 << 20); }

constexpr size_t kAlign = 256;
size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

struct ExpertWorkspace {
  RoutePlan plan;
  int* wc_global;
  void* grouped;
  float* part;
  size_t bytes;
};

// The scratch of a routed call; base == nullptr only sizes.
ExpertWorkspace carve(void* base, int64_t T, int64_t E, int64_t O, int64_t K, const MxPlan& p) {
  ExpertWorkspace ws = {};
  size_t off = 0;
  auto take = [&](size_t bytes) -> void* {
    const size_t at = off;
    off = align_up(off + bytes);
    return base ? static_cast<char*>(base) + at : nullptr;
  };
  const size_t P = (size_t)T * K;
  if (!p.own_lists) {
    ws.plan.meta = static_cast<int*>(take(kMetaWords * sizeof(int)));
    ws.plan.counts = static_cast<int*>(take((size_t)E * sizeof(int)));
    ws.plan.offsets = static_cast<int*>(take((size_t)(E + 1) * sizeof(int)));
    ws.plan.active = static_cast<int*>(take((size_t)E * sizeof(int)));
    ws.plan.pair_list = static_cast<int*>(take(P * sizeof(int)));
    const size_t wc = route_global_counter_words(T, K, E, false);
    ws.wc_global = wc ? static_cast<int*>(take(wc * sizeof(int))) : nullptr;
  }
  ws.grouped = p.grouped_bytes ? take(p.grouped_bytes) : nullptr;
  ws.part = static_cast<float*>(take(P * p.splits * (size_t)O * sizeof(float)));
  ws.bytes = off;
  return ws;
}

// The units of a routed call; none without pairs or experts.
MxPlan routed_plan(int64_t T, int64_t E, int64_t I, int64_t O, int64_t K) {
  return K > 0 && E > 0 ? gemm_mx_plan(T, E, I, O, K, true) : MxPlan{false, 1, 0, 0, 0, false};
}

size_t linear_workspace(const MxPlan& p, int64_t T, int64_t O) {
  return p.splits > 1 ? align_up((size_t)T * O * p.splits * sizeof(float)) : 0;
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

extern "C" size_t mxfp4_linear_workspace_size(int64_t T, int64_t I, int64_t O) {
  if (T < 0 || O < 0 || I <= 0 || I % 32 != 0 || !product_fits(T, 1, I, O, 1)) return (size_t)-1;
  if (T == 0 || O == 0) return 0;
  return linear_workspace(gemm_mx_plan(T, 1, I, O, 1, false), T, O);
}

extern "C" int mxfp4_linear(const uint8_t* x_packed, const uint8_t* x_scales,
                            const uint8_t* packed_weights, const uint8_t* scale_bytes, void* out,
                            int64_t T, int64_t I, int64_t O, int out_dtype, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!known_dtype(out_dtype)) return MXFP4EL_ERR_UNSUPPORTED_DTYPE;
  if (T < 0 || O < 0 || I <= 0 || I % 32 != 0) return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (!product_fits(T, 1, I, O, 1)) return MXFP4EL_ERR_TOO_LARGE;
  if (T == 0 || O == 0) return MXFP4EL_OK;
  const MxPlan plan = gemm_mx_plan(T, 1, I, O, 1, false);
  if (!units_fit(plan)) return MXFP4EL_ERR_TOO_LARGE;
  const size_t es = size_of(out_dtype), G = (size_t)I / 32;
  if (x_packed == nullptr || x_scales == nullptr || packed_weights == nullptr ||
      scale_bytes == nullptr || out == nullptr || !aligned(x_packed, 16) ||
      !aligned(packed_weights, 16) || !aligned(out, es))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  const size_t no = (size_t)T * O * es;
  const size_t nw = linear_workspace(plan, T, O);
  const void* inputs[] = {x_packed, x_scales, packed_weights, scale_bytes};
  const size_t sizes[] = {T * G * 16, T * G, O * G * 16, O * G};
  for (int i = 0; i < 4; ++i)
    if (overlaps(out, no, inputs[i], sizes[i])) return MXFP4EL_ERR_ALIAS;
  if (nw > 0) {
    if (workspace == nullptr || workspace_bytes < nw || !aligned(workspace, kAlign))
      return MXFP4EL_ERR_WORKSPACE;
    if (overlaps(workspace, nw, out, no)) return MXFP4EL_ERR_ALIAS;
    for (int i = 0; i < 4; ++i)
      if (overlaps(workspace, nw, inputs[i], sizes[i])) return MXFP4EL_ERR_ALIAS;
  }
  MxGemm g = {};
  g.x_packed = x_packed;
  g.x_scales = x_scales;
  g.w_packed = packed_weights;
  g.w_scales = scale_bytes;
  g.T = T;
  g.E = 1;
  g.I = I;
  g.O = O;
  g.K = 1;
  g.shape = plan;
  g.part = static_cast<float*>(workspace);
  g.out = out;
  g.out_dtype = out_dtype;
  return status_of(launch_gemm_mx(g, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t mxfp4_expert_linear_quantized_workspace_size(int64_t T, int64_t E, int64_t I,
                                                               int64_t O, int64_t K) {
  if (T < 0 || E < 0 || O < 0 || K < 0 || I <= 0 || I % 32 != 0 || !product_fits(T, E, I, O, K))
    return (size_t)-1;
  if (T == 0 || O == 0) return 0;
  return carve(nullptr, T, E, O, K, routed_plan(T, E, I, O, K)).bytes;
}

extern "C" int mxfp4_expert_linear_quantized(
    const uint8_t* x_packed, const uint8_t* x_scales, const uint8_t* packed_weights,
    const uint8_t* scale_bytes, const void* selected_experts, const float* mixture_weights,
    const void* shared_output, void* out, int64_t T, int64_t E, int64_t I, int64_t O, int64_t K,
    int dtype, int index_dtype, void* workspace, size_t workspace_bytes, void* stream_) {
  if (!known_dtype(dtype) ||
      (index_dtype != MXFP4EL_INDEX_I32 && index_dtype != MXFP4EL_INDEX_I64))
    return MXFP4EL_ERR_UNSUPPORTED_DTYPE;
  if (T < 0 || E < 0 || O < 0 || K < 0 || I <= 0 || I % 32 != 0)
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (!product_fits(T, E, I, O, K)) return MXFP4EL_ERR_TOO_LARGE;
  if (T == 0 || O == 0) return MXFP4EL_OK;
  const bool product = K > 0 && E > 0;
  const MxPlan plan = routed_plan(T, E, I, O, K);
  if (product && ((E < T * K ? E : T * K) > kMxMaxActive || !units_fit(plan)))
    return MXFP4EL_ERR_TOO_LARGE;
  const size_t es = size_of(dtype), is = index_dtype == MXFP4EL_INDEX_I64 ? 8 : 4;
  const size_t G = (size_t)I / 32;
  if (shared_output == nullptr || out == nullptr || !aligned(shared_output, es) ||
      !aligned(out, es))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (K > 0 && (x_packed == nullptr || x_scales == nullptr || selected_experts == nullptr ||
                mixture_weights == nullptr || !aligned(x_packed, 16) ||
                !aligned(selected_experts, is) || !aligned(mixture_weights, 4)))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  if (product && (packed_weights == nullptr || scale_bytes == nullptr ||
                  !aligned(packed_weights, 16)))
    return MXFP4EL_ERR_INVALID_ARGUMENT;
  const size_t no = (size_t)T * O * es;
  const size_t nw = carve(nullptr, T, E, O, K, plan).bytes;
  const void* inputs[] = {x_packed,         x_scales,        packed_weights, scale_bytes,
                          selected_experts, mixture_weights, shared_output};
  const size_t sizes[] = {T * G * 16,         T * G,  (size_t)E * O * G * 16, (size_t)E * O * G,
                          (size_t)T * K * is, (size_t)T * K * 4, no};
  for (int i = 0; i < 7; ++i)
    if (overlaps(out, no, inputs[i], sizes[i])) return MXFP4EL_ERR_ALIAS;
  if (workspace == nullptr || workspace_bytes < nw || !aligned(workspace, kAlign))
    return MXFP4EL_ERR_WORKSPACE;
  if (overlaps(workspace, nw, out, no)) return MXFP4EL_ERR_ALIAS;
  for (int i = 0; i < 7; ++i)
    if (overlaps(workspace, nw, inputs[i], sizes[i])) return MXFP4EL_ERR_ALIAS;
  const ExpertWorkspace ws = carve(workspace, T, E, O, K, plan);
  const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  if (K > 0) {
    // With E == 0 every id is out of range: the bucketer counts them.
    if (!plan.own_lists &&
        launch_route(selected_experts, index_dtype, T, K, E, ws.wc_global, ws.plan,
                     TokenPrep{nullptr, nullptr, nullptr, I}, UnitSplit{0, 0, 0, 1000},
                     stream) != cudaSuccess)
      return MXFP4EL_ERR_CUDA;
    if (product) {
      MxGemm g = {};
      g.x_packed = x_packed;
      g.x_scales = x_scales;
      g.w_packed = packed_weights;
      g.w_scales = scale_bytes;
      if (plan.own_lists) {
        g.sel = selected_experts;
        g.sel64 = index_dtype == MXFP4EL_INDEX_I64;
      } else {
        g.plan = &ws.plan;
      }
      g.T = T;
      g.E = E;
      g.I = I;
      g.O = O;
      g.K = K;
      g.shape = plan;
      g.grouped = ws.grouped;
      g.part = ws.part;
      if (launch_gemm_mx(g, stream) != cudaSuccess) return MXFP4EL_ERR_CUDA;
    }
  }
  // The combine may read its other inputs before the product is done, unless the
  // product is the call's first kernel: that one starts, and lets the combine
  // start, while the kernel before the call may still be writing them.
  const bool early = product && !plan.own_lists;
  return status_of(launch_combine(shared_output, selected_experts, index_dtype, mixture_weights,
                                  ws.part, plan.splits, out, dtype, T, E, O, K, early, stream));
}

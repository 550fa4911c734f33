// quant.cu -- rows of values to MXFP4 and back (include/mxfp4el_quantized.h).
//
// Quantising. A group of 32 values with largest magnitude a has the scale
// byte s = clamp(floor(log2 a) - 2 + 127, 0, 252), so that a 2^(127-s) lies in
// [4, 8) and E2M1's largest value, 6, is at most a factor 4/3 away. floor(log2
// a) + 127 is the exponent field of a (0 for subnormals, which the clamp
// sends to s = 0 as it should), so no logarithm is taken; the scaling by a
// power of two is exact wherever a code other than 0 can come out, and the
// hardware conversion rounds to nearest, ties to the even code, and saturates.
// Largest magnitudes compare as integers, so a NaN or an infinity shows as a
// maximum of 0x7f800000 or more.
//
// Both directions only move bytes. A warp takes 1024 values at a time, eight
// per lane four times over, so that four loads per lane are in flight (one at a
// time, with a division for the row of every eight values: 37 us for 8192 x 7168
// bf16); the 32 scale bytes of a task are stored together. 8192 x 7168 bf16, from
// DRAM: 29 us, and 25 us back, against 22 us for the 149 MB of each at the rate
// of a copy.
#include <algorithm>

#include "common.cuh"
#include "quant.h"

namespace mxfp4el {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 8;                 // values per thread and step: four threads share a group
constexpr int kSteps = 4;                     // steps of a task
constexpr int kStep = 32 * kPerThread;        // values of a warp's step
constexpr int kTask = kStep * kSteps;
constexpr uint32_t kInfBits = 0x7f800000u;

// Eight float32 values to eight E2M1 codes, the first in the low nibble.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n"
      " .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n"
      "}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

template <bool kVec>
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  if constexpr (kVec) {
    const uint4 a = ld_stream_u4(p), b = ld_stream_u4(p + 4);
    v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y);
    v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
    v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y);
    v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[i];
  }
}
template <bool kVec>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  if constexpr (kVec) {
    const uint4 a = ld_stream_u4(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __bfloat162float(p[i]);
  }
}

// rows x I values as rows x segs tasks; a contiguous matrix is one row.
template <typename Tok, bool kVec>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const Tok* __restrict__ x, int64_t row_stride, int64_t rows, int64_t I,
                int64_t segs, uint8_t* __restrict__ packed, uint8_t* __restrict__ scales) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t tasks = rows * segs, step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t task = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); task < tasks;
       task += step) {
    const int64_t r = rows == 1 ? 0 : task / segs;
    const int64_t col = (task - r * segs) * kTask;         // first value of the task
    const Tok* from = x + r * row_stride + col + lane * kPerThread;
    const int left = (int)min((int64_t)kTask, I - col);    // its values, a multiple of 32
    float v[kSteps][8];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
      if (j * kStep + lane * kPerThread < left) load8<kVec>(from + j * kStep, v[j]);
    }
    uint32_t* to = reinterpret_cast<uint32_t*>(packed) + (r * I + col) / 8 + lane;
    int scale = 0;                                         // of group `lane` of the task
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[j][i]) & 0x7fffffffu);
      m = max(m, __shfl_xor_sync(kFullMask, m, 1));
      m = max(m, __shfl_xor_sync(kFullMask, m, 2));
      const bool finite = m < kInfBits;
      const int s = finite ? max((int)(m >> 23) - 2, 0) : 255;
      const float up = __uint_as_float((uint32_t)(254 - min(s, 252)) << 23);   // 2^(127 - s)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= up;
      const uint32_t q = finite ? f32x8_to_e2m1(v[j]) : 0u;
      if (j * kStep + lane * kPerThread < left) to[j * 32] = q;
      const int moved = __shfl_sync(kFullMask, s, 4 * (lane & 7));
      if (lane >> 3 == j) scale = moved;
    }
    if (lane * 32 < left) scales[(r * I + col) / 32 + lane] = (uint8_t)scale;
  }
}

__device__ __forceinline__ void store8(float* p, const float2 (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float2 (&v)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[i].x, v[i].y);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename Tok>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t* __restrict__ packed, const uint8_t* __restrict__ scales,
                  int64_t n, Tok* __restrict__ out) {
  pdl_launch_dependents();
  pdl_wait();                                 // the codes may come from the kernel before
  const int64_t step = (int64_t)gridDim.x * kThreads;
  for (int64_t at0 = (int64_t)blockIdx.x * kThreads + threadIdx.x; at0 < n; at0 += kSteps * step) {
    uint32_t q[kSteps], s[kSteps];
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int64_t at = at0 + j * step;
      q[j] = at < n ? reinterpret_cast<const uint32_t*>(packed)[at] : 0u;
      s[j] = at < n ? scales[at >> 2] : 0u;
    }
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int64_t at = at0 + j * step;
      if (at >= n) break;
      uint32_t f = s[j] << 23;                // 2^(s - 127)
      if (s[j] == 0) f = 0x00400000u;         // a subnormal float32
      if (s[j] == 255) f = 0x7fc00000u;       // NaN
      const float by = __uint_as_float(f);
      uint32_t h[4];
      e2m1x8_to_f16x2x4(q[j], h);
      float2 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = f16x2_to_f32x2(h[i]);
        v[i].x *= by;
        v[i].y *= by;
      }
      store8(out + at * kPerThread, v);
    }
  }
}

// Blocks for n threads' first steps: few enough for a second round where there
// is work for the whole GPU.
unsigned grid_for(int64_t n) {
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>((n + kThreads - 1) / kThreads, 152 * 8));
}

template <typename Tok>
cudaError_t quantize_typed(const Tok* x, int64_t row_stride, int64_t rows, int64_t I,
                           uint8_t* packed, uint8_t* scales, cudaStream_t stream) {
  if (rows > 1 && row_stride == I) {
    I *= rows;
    rows = 1;
  }
  const int64_t segs = (I + kTask - 1) / kTask, tasks = rows * segs;
  const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
                   (rows == 1 || row_stride * (int64_t)sizeof(Tok) % 16 == 0);
  const unsigned grid =
      (unsigned)std::min<int64_t>((tasks + kThreads / 32 - 1) / (kThreads / 32), 1 << 20);
  if (vec)
    quantize_kernel<Tok, true><<<grid, kThreads, 0, stream>>>(x, row_stride, rows, I, segs, packed,
                                                              scales);
  else
    quantize_kernel<Tok, false><<<grid, kThreads, 0, stream>>>(x, row_stride, rows, I, segs,
                                                               packed, scales);
  const cudaError_t err = cudaGetLastError();
  if (err == cudaSuccess) note_launch();
  return err;
}

}  // namespace

cudaError_t launch_quantize(const void* x, int dtype, int64_t row_stride, int64_t rows, int64_t I,
                            uint8_t* packed, uint8_t* scales, cudaStream_t stream) {
  if (dtype == kTokenBF16)
    return quantize_typed(static_cast<const __nv_bfloat16*>(x), row_stride, rows, I, packed,
                          scales, stream);
  return quantize_typed(static_cast<const float*>(x), row_stride, rows, I, packed, scales, stream);
}

cudaError_t launch_dequantize(const uint8_t* packed, const uint8_t* scales, int64_t rows,
                              int64_t I, void* out, int dtype, cudaStream_t stream) {
  const int64_t n = rows * (I / kPerThread);
  if (dtype == kTokenBF16)
    return launch_after_previous(dequantize_kernel<__nv_bfloat16>, dim3(grid_for(n)),
                                 dim3(kThreads), 0, stream, packed, scales, n,
                                 static_cast<__nv_bfloat16*>(out));
  return launch_after_previous(dequantize_kernel<float>, dim3(grid_for(n)), dim3(kThreads), 0,
                               stream, packed, scales, n, static_cast<float*>(out));
}

}  // namespace mxfp4el

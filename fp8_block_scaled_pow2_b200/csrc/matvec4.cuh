// Matrix-vector products with 4-bit weights and group scales:
//   y[m, n] = sum_k x[m, k] * w[n, k],  M <= 16 rows of x
// for the three weight forms of this library: MXFP4 (E2M1, E8M0 scale per 32),
// NVFP4 (E2M1, E4M3 scale per 16, one float32 factor per matrix) and symmetric
// INT4 (float32 scale per 128).  x keeps its own type (no quantisation), sums
// are float32, y is rounded once.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {
namespace matvec {

constexpr int kMaxRows = 16;      // rows of x per call

enum Format { kMxfp4 = 0, kNvfp4 = 1, kInt4 = 2 };

struct Args {
  const void* x;
  int64_t ldx;
  int x_type, M;
  const uint8_t* w;
  const void* scale;
  const float* global;
  int N, K;
  void* out;
  int64_t ldout;
  int out_type;
};

__device__ __forceinline__ float load_x(const void* x, int type, int64_t i) {
  if (type == MOE_TYPE_F32) return __ldg(static_cast<const float*>(x) + i);
  if (type == MOE_TYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(x)[i]);
  return __half2float(static_cast<const __half*>(x)[i]);
}

__device__ __forceinline__ void store_y(void* out, int type, int64_t i, float v) {
  if (type == MOE_TYPE_F32) static_cast<float*>(out)[i] = v;
  else if (type == MOE_TYPE_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

// E2M1 code -> value: magnitude from the exponent and mantissa bits.
__device__ __forceinline__ float e2m1_to_float(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e == 0 ? 0.5f * (float)m : __uint_as_float(((e + 126u) << 23) | (m << 22));
  return (c & 8u) ? -v : v;
}

// E8M0 byte -> 2^(b - 127); 255 is NaN.
__device__ __forceinline__ float e8m0_to_float(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7FC00000u) : exp2_int((int)b - 127);
}

// One warp per output; a lane takes every 32nd 32-wide group of the row.
template <int FMT>
__global__ void __launch_bounds__(256) matvec_kernel(const Args a) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int groups = a.K / 32;
  float acc[kMaxRows];
#pragma unroll
  for (int m = 0; m < kMaxRows; ++m) acc[m] = 0.f;
  for (int g = lane; g < groups; g += 32) {
    const uint4 wv = __ldg(reinterpret_cast<const uint4*>(a.w + n * (a.K / 2)) + g);
    const uint32_t u[4] = {wv.x, wv.y, wv.z, wv.w};
    float s0, s1;
    if (FMT == kMxfp4) {
      s0 = s1 = e8m0_to_float(static_cast<const uint8_t*>(a.scale)[n * groups + g]);
    } else if (FMT == kNvfp4) {
      const uint8_t* sp = static_cast<const uint8_t*>(a.scale) + n * (a.K / 16) + 2 * g;
      s0 = e4m3_to_float(sp[0]);
      s1 = e4m3_to_float(sp[1]);
    } else {
      s0 = s1 = static_cast<const float*>(a.scale)[n * (a.K / 128) + g / 4];
    }
    float v[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint32_t c = (u[j / 8] >> (4 * (j % 8))) & 15u;
      v[j] = FMT == kInt4 ? (float)((int)(c ^ 8u) - 8) : e2m1_to_float(c);
    }
#pragma unroll
    for (int m = 0; m < kMaxRows; ++m) {
      if (m < a.M) {
        float p0 = 0.f, p1 = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) p0 = fmaf(v[j], load_x(a.x, a.x_type, m * a.ldx + 32 * g + j), p0);
#pragma unroll
        for (int j = 16; j < 32; ++j) p1 = fmaf(v[j], load_x(a.x, a.x_type, m * a.ldx + 32 * g + j), p1);
        acc[m] = fmaf(p0, s0, fmaf(p1, s1, acc[m]));
      }
    }
  }
  const float f = FMT == kNvfp4 ? __ldg(a.global) : 1.0f;
#pragma unroll
  for (int m = 0; m < kMaxRows; ++m) {
    float v = acc[m];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (m < a.M && lane == 0) store_y(a.out, a.out_type, m * a.ldout + n, v * f);
  }
}

}  // namespace matvec
}  // namespace moe

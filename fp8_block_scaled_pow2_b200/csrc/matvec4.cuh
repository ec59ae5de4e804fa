// Matrix-vector products with 4-bit weights and group scales:
//   y[m, n] = sum_k x[m, k] * w[n, k],  M <= 16 rows of x
// for the three weight forms of this library: MXFP4 (E2M1, E8M0 scale per 32),
// NVFP4 (E2M1, E4M3 scale per 16, one float32 factor per matrix) and symmetric
// INT4 (float32 scale per 128).  x keeps its own type (no quantisation), sums
// are float32, y is rounded once.
//
// Bound: the stream of weights (0.53 to 0.56 bytes each, 188 cycles of an SM
// sub-partition per 2048 weights at the copy rate), so conversions have to be
// cheap and the products go to half-precision mma.sync m16n8k16 (8 cycles; its
// FP8 form is emulated here, 26 cycles):
//   x      float16 times a power of two per row of x.  bfloat16 and float16 values
//          are exact there down to 2^-29 of the row's largest value (2^-39 of
//          it is lost at most); a float32 value becomes two columns, a float16
//          and the next 11 bits of it.
//   MXFP4  the hardware conversion of E2M1 pairs to float16; each group of 32 is
//          two MMAs from zero whose sums take the E8M0 scale in float32.
//   NVFP4  the same values times the E4M3 scale, exact in float16 (2 + 4
//          significant bits, 2^-10 .. 2688), so sums run over all of K.
//   INT4   the code with its top bit flipped, u = q + 8, left where it lies in
//          the low mantissa bits of a float16: the subnormal u * 2^-24 (u * 2^-20
//          for every second nibble, whose x is divided by 16): one logic
//          operation per two weights.  sum x q = sum x u - 8 sum x, the second sum
//          taken once per (row of x, group of 128).
//
// A tile is 16 rows of w.  The warps of a block split a tile's K, 256 columns a
// step, and add their sums in shared memory.  Each warp has a ring of its own:
// one TMA copy a step brings the 16 x 128 bytes, swizzled so that ldmatrix
// reads the 4-byte words of 8 rows without bank conflicts (a matrix row is a
// scale group of 32 weights, a lane's word is its part of an MMA operand).
// With copies by the lanes and word loads a step took 220 instructions per
// 2048 weights and the kernel ran at half the copy rate.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "sm100.cuh"

namespace moe {
namespace matvec {

constexpr int kMaxRows = 16;      // rows of x per call
constexpr int kMaxK = 32768;      // one float32 row of x in a block's shared memory
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxStages = 4;
constexpr int kStep = 256;        // columns of a step
constexpr int kTile = 16 * 128;   // bytes of a step's weights
constexpr int kTileSf = 16 * 16;  // and of its scales (16 a row: NVFP4 all, the others the first 8)

enum Format { kMxfp4 = 0, kNvfp4 = 1, kInt4 = 2 };

struct Args {
  const void* x;
  int64_t ldx;
  int x_type, M;
  const uint8_t* scale;
  const float* global;
  int N, K;
  void* out;
  int64_t ldout;
  int out_type;
  int warps_per_tile;             // 8, 4, 2 or 1
  int scale_vec;                  // scales can be copied as 4-byte words
  int x_vec;                      // rows of x are 16-byte aligned
};

struct Smem {
  // ring of weights (1024-byte aligned) | of scales | barriers | x [cols][stride] float16 | 8 x sums of x per 128
  // columns (INT4) [K / 128][cols] | sums [2][warps][cols][16] | exponents [16], abort flag
  __host__ __device__ static int steps(int K) { return (K + kStep - 1) / kStep; }
  __host__ __device__ static int x_stride(int K) { return steps(K) * kStep * 2 + 64; }   // bytes; rows 64 mod 128 apart
  __host__ __device__ static int sf_off(int stages) { return kWarps * stages * kTile; }
  __host__ __device__ static int bar_off(int stages) { return sf_off(stages) + kWarps * stages * kTileSf; }
  __host__ __device__ static int x_off(int stages) { return bar_off(stages) + kWarps * kMaxStages * 8; }
  __host__ __device__ static int corr_off(int stages, int cols, int K) { return x_off(stages) + cols * x_stride(K); }
  __host__ __device__ static int red_off(int stages, int cols, int K) {
    return corr_off(stages, cols, K) + (2 * steps(K) * cols * 4 + 15) / 16 * 16;
  }
  __host__ __device__ static int fac_off(int stages, int cols, int K) {
    return red_off(stages, cols, K) + 2 * kWarps * cols * 16 * 4;
  }
  __host__ __device__ static int total(int stages, int cols, int K) { return fac_off(stages, cols, K) + 17 * 4 + 1024; }
};

__device__ __forceinline__ void store_y(void* out, int type, int64_t i, float v) {
  if (type == MOE_TYPE_F32) static_cast<float*>(out)[i] = v;
  else if (type == MOE_TYPE_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(out)[i] = __float2half_rn(v);
}

// v * 2^s, |s| <= 254, by two exact factors (one rounding where the result is subnormal).
__device__ __forceinline__ float scale_pow2(float v, int s) {
  const int h = s / 2;
  return v * exp2_int(h) * exp2_int(s - h);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
// This lane's earlier cp.async copies arrive on the barrier (counted in its expected arrivals).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(bar)) : "memory");
}

// Four 8-row matrices of 16-byte rows: lane (g, q) gets word q of row g of each.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// As mma_f16 with zero in place of the old sums.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 E2M1 nibbles -> four float16 pairs in order.
__device__ __forceinline__ void e2m1_pairs(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// 8 two's complement nibbles n0..n7 -> u = n + 8 as float16 subnormals: pairs
// (u0, u4) 2^-24, (u1, u5) 2^-20, (u2, u6) 2^-24, (u3, u7) 2^-20.
__device__ __forceinline__ void int4_pairs(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t v = w >> 8;
  r[0] = (w & 0x000F000Fu) ^ 0x00080008u;
  r[1] = (w & 0x00F000F0u) ^ 0x00800080u;
  r[2] = (v & 0x000F000Fu) ^ 0x00080008u;
  r[3] = (v & 0x00F000F0u) ^ 0x00800080u;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 s) {
  const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// NT: groups of 8 columns (a column is a row of x, or one of the two halves of a
// float32 row).
template <int FMT, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    matvec_kernel(const __grid_constant__ CUtensorMap tmW, const Args a, int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const int g = lane >> 2, q = lane & 3;
  const int P = a.x_type == MOE_TYPE_F32 ? 2 : 1, cols = a.M * P, steps = Smem::steps(a.K);
  const int xs_stride = Smem::x_stride(a.K);
  uint8_t* xs = smem + Smem::x_off(stages);
  float* corr = reinterpret_cast<float*>(smem + Smem::corr_off(stages, cols, a.K));
  float* red = reinterpret_cast<float*>(smem + Smem::red_off(stages, cols, a.K));
  int* fac = reinterpret_cast<int*>(smem + Smem::fac_off(stages, cols, a.K));      // exponent of each row's factor
  int* abort_word = fac + kMaxRows;
  volatile int* abort_flag = abort_word;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Smem::bar_off(stages)) + warp * kMaxStages;
  pdl_trigger();
  if (lane == 0) {
    for (int i = 0; i < stages; ++i) sm100::mbar_init(&bars[i], 1 + 32);   // the TMA copy, the lanes' scales
    sm100::fence_mbar_init();
  }
  if (tid < kMaxRows) fac[tid] = 0;
  if (tid == kMaxRows) *abort_word = 0;
  __syncthreads();
  pdl_wait();

  // ---- this warp's tiles and steps ----
  const int wpt = a.warps_per_tile, groups = kWarps / wpt, tg = warp / wpt, wk = warp % wpt;
  const int tiles = (a.N + 15) / 16, rounds_total = (tiles + groups - 1) / groups;      // rounds over all blocks
  uint8_t* ring = smem + warp * stages * kTile;
  uint8_t* ring_sf = smem + Smem::sf_off(stages) + warp * stages * kTileSf;
  constexpr int kSfBytes = FMT == kNvfp4 ? 16 : 8;      // scale bytes of a row and step
  const int srow = FMT == kNvfp4 ? a.K / 16 : a.K / 32; // scale bytes of a row (INT4: K / 128 floats)
  // the lane's scale words: row lane / 2, word lane % 2 (NVFP4: and + 2)
  const int sf_r = lane >> 1, sf_o = (lane & 1) * 4;
  const uint8_t* sf_src = nullptr;
  bool sf_row = false;
  int fround = blockIdx.x, fstep = wk, fslot = 0, in_flight = 0;
  auto fetch_round = [&]() {
    const int64_t n = ((int64_t)fround * groups + tg) * 16 + sf_r;
    sf_row = n < a.N;
    sf_src = a.scale + (sf_row ? n * srow : 0);
  };
  fetch_round();
  auto fetch = [&]() {
    if (fround < rounds_total) {
      const int64_t n0 = ((int64_t)fround * groups + tg) * 16;
      if (n0 < a.N) {
        ++in_flight;
        uint64_t* bar = &bars[fslot];
        if (sm100::elect_one()) {
          sm100::mbar_arrive_expect_tx(bar, kTile);
          sm100::tma_load_2d(ring + fslot * kTile, &tmW, fstep * 128, (int)n0, bar);
        }
        __syncwarp();
        uint8_t* sd = ring_sf + fslot * kTileSf;
        if (a.scale_vec) {
#pragma unroll
          for (int i = 0; i < kSfBytes / 8; ++i) {
            const int o = fstep * kSfBytes + sf_o + 8 * i;
            const bool in = sf_row && o < srow;
            cp_async4(sm100::smem_u32(sd + sf_r * 16 + sf_o + 8 * i), in ? sf_src + o : a.scale, in);
          }
          cp_async_arrive(bar);
        } else {
          // rows of scales that start at any byte (K not a multiple of 128, or an odd base address)
          for (int i = lane; i < 16 * kSfBytes; i += 32) {
            const int r = i / kSfBytes, b = i % kSfBytes, o = fstep * kSfBytes + b;
            sd[r * 16 + b] = n0 + r < a.N && o < srow ? a.scale[(n0 + r) * srow + o] : 0;
          }
          sm100::mbar_arrive(bar);
        }
      }
      fstep += wpt;
      if (fstep >= steps) {
        fstep = wk;
        fround += gridDim.x;
        fetch_round();
      }
    }
    fslot = fslot + 1 == stages ? 0 : fslot + 1;
  };
  for (int s = 0; s < stages; ++s) fetch();

  // ---- x: float16 columns; a warp takes 256 columns of a row, 8 a lane, four
  // such tasks at a time (their loads in flight together) ----
  const int tasks = a.M * steps;
  auto load_tasks = [&](int t0, float (&v)[4][8]) {
    uint4 raw[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j * kWarps, m = t / steps, k = (t - m * steps) * kStep + lane * 8;
      const bool in = t < tasks && k < a.K;
      const int64_t at = m * a.ldx + k;
      raw[j][0] = raw[j][1] = make_uint4(0u, 0u, 0u, 0u);
      if (in && a.x_vec) {
        if (P == 2) {
          raw[j][0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(a.x) + at));
          raw[j][1] = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(a.x) + at) + 1);
        } else {
          raw[j][0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + at));
        }
      } else if (in) {
        if (P == 2) {
          const uint32_t* p = static_cast<const uint32_t*>(a.x) + at;
          raw[j][0] = make_uint4(__ldg(p), __ldg(p + 1), __ldg(p + 2), __ldg(p + 3));
          raw[j][1] = make_uint4(__ldg(p + 4), __ldg(p + 5), __ldg(p + 6), __ldg(p + 7));
        } else {
          const uint16_t* p = static_cast<const uint16_t*>(a.x) + at;
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = __ldg(p + 2 * i) | ((uint32_t)__ldg(p + 2 * i + 1) << 16);
          raw[j][0] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t w[8] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w,
                             raw[j][1].x, raw[j][1].y, raw[j][1].z, raw[j][1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (a.x_type == MOE_TYPE_F32) {
          v[j][i] = __uint_as_float(w[i]);
          v[j][i + 4] = __uint_as_float(w[i + 4]);
        } else if (a.x_type == MOE_TYPE_BF16) {
          v[j][2 * i] = bf16_lo(w[i]);
          v[j][2 * i + 1] = bf16_hi(w[i]);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          v[j][2 * i] = f.x;
          v[j][2 * i + 1] = f.y;
        }
      }
    }
  };
  // the power of two of a row takes its largest value to [2^14, 2^15); float16
  // stays as it is, unless half of its values are to be divided by 16
  const bool once = tasks <= 4 * kWarps;  // every task in one batch: x is read once
  float v4[4][8];
  if (a.x_type != MOE_TYPE_F16 || FMT == kInt4) {
    for (int t0 = warp; t0 < tasks; t0 += 4 * kWarps) {
      load_tasks(t0, v4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v4[j][i]));
        mx = warp_max_nonneg(mx);
        if (lane == 0 && t0 + j * kWarps < tasks) atomicMax(fac + (t0 + j * kWarps) / steps, (int)__float_as_uint(mx));
      }
    }
    __syncthreads();
    if (tid < a.M) {
      const int mx = fac[tid];
      fac[tid] = mx > 0 ? max(mx >> 23, 1) - 127 - 14 : 0;      // exponent of the factor of y
    }
    __syncthreads();
  }
  for (int t0 = warp; t0 < tasks; t0 += 4 * kWarps) {
    if (!once || (a.x_type == MOE_TYPE_F16 && FMT != kInt4)) load_tasks(t0, v4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j * kWarps;
      if (t >= tasks) break;
      const int m = t / steps, k0 = (t - m * steps) * kStep, k = k0 + lane * 8, s = -fac[m];
      float hi[8], lo[8], sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = scale_pow2(v4[j][i], s);
        hi[i] = __half2float(__float2half_rn(v));
        sum0 += hi[i];
        lo[i] = P == 2 ? __half2float(__float2half_rn((v - hi[i]) * 2048.0f)) : 0.f;
        sum1 += lo[i];
      }
      auto put = [&](int col, const float (&f)[8]) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 h = FMT == kInt4 ? __floats2half2_rn(i & 1 ? f[i] * 0.0625f : f[i], i & 1 ? f[i + 4] * 0.0625f : f[i + 4])
                                         : __floats2half2_rn(f[2 * i], f[2 * i + 1]);
          p[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(xs + col * xs_stride + k * 2) = make_uint4(p[0], p[1], p[2], p[3]);
      };
      put(m * P, hi);
      if (P == 2) put(m * P + 1, lo);
      if (FMT == kInt4) {
        // 128 columns = a half-warp
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          sum0 += __shfl_xor_sync(0xFFFFFFFFu, sum0, o);
          sum1 += __shfl_xor_sync(0xFFFFFFFFu, sum1, o);
        }
        if ((lane & 15) == 0) {
          float* c = corr + (k0 / 128 + (lane >> 4)) * cols + m * P;
          c[0] = 8.0f * sum0;
          if (P == 2) c[1] = 8.0f * sum1;
        }
      }
    }
  }
  __syncthreads();

  const float glob = FMT == kNvfp4 ? __ldg(a.global) : 1.0f;
  // E8M0 scales reach 2^127, and rows of x below 2^14 were scaled up: sums are
  // kept 2^shift times smaller, so that they overflow only where y does (rows
  // of x below 2^-10, whose factor is larger than that, excepted).
  int shift = 0;
  if (FMT == kMxfp4)
    for (int m = 0; m < a.M; ++m) shift = max(shift, min(24, -fac[m]));
  const float unit = exp2_int(-shift);
  int col_b[NT];                          // the lane's column of the token operand (past the last one: any)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) col_b[nt] = min(nt * 8 + g, cols - 1) * xs_stride + q * 16;
  // ldmatrix: lane l names row l % 8 of matrix l / 8, a 16-byte chunk of the swizzled tile
  const int lr = lane & 7;
  const uint32_t ld0 = lr * 128 + (((lane >> 3) ^ lr) << 4), ld1 = lr * 128 + (((4 + (lane >> 3)) ^ lr) << 4);
  const uint32_t ring_u = sm100::smem_u32(ring);
  const uint32_t sel16 = q >= 2 ? 0x3232u : 0x1010u;     // NVFP4: the lane's half of a pair of scales, twice
  int slot = 0, buf = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int round = blockIdx.x; round < rounds_total; round += gridDim.x) {
    const int64_t n0 = ((int64_t)round * groups + tg) * 16;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
    for (int step = wk; step < steps; step += wpt) {
      if (n0 < a.N && ok) ok = sm100::mbar_wait_warp(&bars[slot], phase, abort_flag);
      if (n0 < a.N && ok) {
        --in_flight;
        const uint32_t wt = ring_u + slot * kTile;
        const uint8_t* s0 = ring_sf + slot * kTileSf + g * 16;
        const uint8_t* s8 = s0 + 8 * 16;
        const uint8_t* xk = xs + step * kStep * 2;
#pragma unroll
        for (int half = 0; half < 2; ++half) {           // 128 columns each
          uint32_t u0[4], u8[4];
          ldmatrix4(u0, wt + (half ? ld1 : ld0));
          ldmatrix4(u8, wt + 1024 + (half ? ld1 : ld0));
          float c[NT][4];
          float f0[4], f8[4];                            // MXFP4: scales of the four groups
          __half2 h0[4], h8[4];                          // NVFP4: scales of the lane's columns in each group
          if (FMT == kMxfp4) {
            const uint32_t m0 = *reinterpret_cast<const uint32_t*>(s0 + half * 4);
            const uint32_t m8 = *reinterpret_cast<const uint32_t*>(s8 + half * 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t t0, t8;
              asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(t0) : "h"((uint16_t)(m0 >> (16 * i))));
              asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(t8) : "h"((uint16_t)(m8 >> (16 * i))));
              f0[2 * i] = bf16_lo(t0) * unit;
              f0[2 * i + 1] = bf16_hi(t0) * unit;
              f8[2 * i] = bf16_lo(t8) * unit;
              f8[2 * i + 1] = bf16_hi(t8) * unit;
            }
          }
          if (FMT == kNvfp4) {
            const uint2 m0 = *reinterpret_cast<const uint2*>(s0 + half * 8), m8 = *reinterpret_cast<const uint2*>(s8 + half * 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {                // the two scales of group i
              const uint32_t p0 = (i < 2 ? m0.x : m0.y) >> (16 * (i & 1)), p8 = (i < 2 ? m8.x : m8.y) >> (16 * (i & 1));
              const __half2_raw c0 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)p0, __NV_E4M3);
              const __half2_raw c8 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)p8, __NV_E4M3);
              const uint32_t d0 = __byte_perm(*reinterpret_cast<const uint32_t*>(&c0), 0u, sel16);
              const uint32_t d8 = __byte_perm(*reinterpret_cast<const uint32_t*>(&c8), 0u, sel16);
              h0[i] = *reinterpret_cast<const __half2*>(&d0);
              h8[i] = *reinterpret_cast<const __half2*>(&d8);
            }
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {                  // groups of 32 columns
            uint32_t r0[4], r8[4];
            if (FMT == kInt4) {
              int4_pairs(u0[s], r0);
              int4_pairs(u8[s], r8);
            } else {
              e2m1_pairs(u0[s], r0);
              e2m1_pairs(u8[s], r8);
            }
            if (FMT == kNvfp4) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                r0[i] = mul_f16x2(r0[i], h0[s]);
                r8[i] = mul_f16x2(r8[i], h8[s]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 b = *reinterpret_cast<const uint4*>(xk + col_b[nt] + half * 256 + s * 64);
              if (FMT == kNvfp4) {
                mma_f16(acc[nt], r0[0], r8[0], r0[1], r8[1], b.x, b.y);
                mma_f16(acc[nt], r0[2], r8[2], r0[3], r8[3], b.z, b.w);
              } else if (FMT == kInt4 && s > 0) {
                mma_f16(c[nt], r0[0], r8[0], r0[1], r8[1], b.x, b.y);
                mma_f16(c[nt], r0[2], r8[2], r0[3], r8[3], b.z, b.w);
              } else {
                mma_f16_first(c[nt], r0[0], r8[0], r0[1], r8[1], b.x, b.y);
                mma_f16(c[nt], r0[2], r8[2], r0[3], r8[3], b.z, b.w);
              }
              if (FMT == kMxfp4) {
                acc[nt][0] = fmaf(c[nt][0], f0[s], acc[nt][0]);
                acc[nt][1] = fmaf(c[nt][1], f0[s], acc[nt][1]);
                acc[nt][2] = fmaf(c[nt][2], f8[s], acc[nt][2]);
                acc[nt][3] = fmaf(c[nt][3], f8[s], acc[nt][3]);
              }
            }
          }
          if (FMT == kInt4) {
            const float i0 = *reinterpret_cast<const float*>(s0 + half * 4), i8 = *reinterpret_cast<const float*>(s8 + half * 4);
            const float* cr = corr + (step * 2 + half) * cols;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float k0 = cr[min(nt * 8 + 2 * q, cols - 1)], k1 = cr[min(nt * 8 + 2 * q + 1, cols - 1)];
              acc[nt][0] = fmaf(fmaf(c[nt][0], 16777216.0f, -k0), i0, acc[nt][0]);
              acc[nt][1] = fmaf(fmaf(c[nt][1], 16777216.0f, -k1), i0, acc[nt][1]);
              acc[nt][2] = fmaf(fmaf(c[nt][2], 16777216.0f, -k0), i8, acc[nt][2]);
              acc[nt][3] = fmaf(fmaf(c[nt][3], 16777216.0f, -k1), i8, acc[nt][3]);
            }
          }
        }
      }
      if (!ok) continue;                  // the ring stays where it gave up
      __syncwarp();                       // every lane has read the slot
      fetch();
      if (++slot == stages) {
        slot = 0;
        phase ^= 1u;
      }
    }
    // ---- sum over the tile's warps; two buffers in turn, so one barrier of these warps a round ----
    float* rb = red + (buf * kWarps + tg * wpt) * cols * 16;
    buf ^= 1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = nt * 8 + 2 * q + (i & 1);
        if (col < cols) rb[(wk * cols + col) * 16 + g + 8 * (i >> 1)] = acc[nt][i];
      }
    }
    if (wpt > 1) sm100::named_bar_sync(1 + tg, wpt * 32);
    else __syncwarp();
    for (int i = wk * 32 + lane; i < a.M * 16; i += wpt * 32) {
      const int r = i & 15, m = i >> 4;
      if (n0 + r >= a.N) continue;
      const float* p = rb + m * P * 16 + r;
      float v = 0.f, lo = 0.f;
      for (int w = 0; w < wpt; ++w, p += cols * 16) {
        v += p[0];
        if (P == 2) lo += p[16];
      }
      if (P == 2) v = fmaf(lo, 1.0f / 2048.0f, v);
      if (FMT == kNvfp4) v *= glob;
      store_y(a.out, a.out_type, m * a.ldout + n0 + r, scale_pow2(v, fac[m] + shift));
    }
  }
  // after a wait has given up: the copies still on their way (bounded)
  const uint64_t t0 = globaltimer_ns();
  for (; in_flight > 0 && globaltimer_ns() - t0 < sm100::kWaitTimeoutNs; --in_flight) {
    while (!sm100::mbar_try_wait(sm100::smem_u32(&bars[slot]), phase) && globaltimer_ns() - t0 < sm100::kWaitTimeoutNs) {
    }
    if (++slot == stages) {
      slot = 0;
      phase ^= 1u;
    }
  }
}

}  // namespace matvec
}  // namespace moe

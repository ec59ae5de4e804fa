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
//   x      float16 times a power of two per row of x (for float16 too: its
//          subnormals would lose bits as above).  bfloat16 and float16 values are
//          exact there down to 2^-29 of the row's largest value (2^-39 of it is
//          lost at most); a float32 value becomes two columns, a float16 and
//          the next 11 bits of it (one value in four loses its last bit, 2^-23;
//          a third column would cost half as much again for it).
//   MXFP4  the hardware conversion of E2M1 pairs to float16; each group of 32 is
//          two MMAs from zero whose sums take the row's power of two back and
//          then the E8M0 scale, in float32.
//   NVFP4  the same values times the E4M3 scale, exact in float16 (2 + 4
//          significant bits, 2^-10 .. 2688), so that MMAs sum a whole step (256
//          columns; over 32768 their truncation came to 2^-18).
//   INT4   the code with its top bit flipped, u = q + 8, or'ed under the exponent of
//          1024: the float16 1024 + u (1024 + 16 u for every second nibble), from
//          which one packed addition (multiply-add) leaves q.  (Y. J. Kim, R.
//          Henry, R. Fahim, H. Hassan Awadalla, "Who Says Elephants Can't Run",
//          2022, describe this conversion for unsigned codes.  u itself, as the
//          float16 subnormal u * 2^-24 that its bits are, saves that operation
//          and is wrong by 2^-18: the tensor core aligns products by their
//          exponent fields, and a subnormal's has up to 10 leading zeros.)
//
// A block takes sets of 16-row tiles, K split over its 16 compute warps, 256
// columns each, so that whole rows stream in at a time (with warps on tiles of
// their own, 128-byte pieces 2 KB apart were in flight, and memory gave 4.5
// instead of 6.1 TB/s).  One warp issues the copies: a single TMA instruction
// brings a set's tiles, another one their scales, swizzled so that ldmatrix
// reads the 4-byte words of 8 rows without bank conflicts (a matrix row is a
// scale group of 32 weights, a lane's word its part of an MMA operand).  A
// warp's part of x never changes where K <= 4096 and stays in registers (up to 8
// columns; 8 rows read from shared memory took as long as the weights' stream).
// Three more warps add the compute warps' sums and store y, so these never wait
// for one another.
// Measured (one B200, captured): 1 x 131072 x 4096 NVFP4 73 us (302 MB: 4.1 TB/s;
// 50 us without conversions and products), INT4 70, MXFP4 66; 65536 x 4096 MXFP4
// with 1 row of x 36 us, with 8 rows 42, with 16 rows 53 (INT4 54, NVFP4 54);
// 4096 x 2048 MXFP4 5.3 us.  Issue-bound: 180 to 190 instructions per 2048
// weights, 120 of them conversions, scale products and MMAs.  16 rows of float32
// are 32 columns, which at K = 4096 do not fit beside two ring slots: two passes
// over the weights, 99 us for 65536 x 4096.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "sm100.cuh"

namespace moe {
namespace matvec {

constexpr int kMaxRows = 16;      // rows of x per call
constexpr int kMaxN = 0x7FFF0000; // rows of w: row numbers of a last set stay 32-bit
constexpr int kMaxK = 32768;      // one float32 row of x in a block's shared memory
constexpr int kWarps = 16;        // compute warps; then the copies' and the sums' warp
constexpr int kProducer = kWarps, kReducers = 3;
constexpr int kThreads = 32 * (kWarps + 1 + kReducers);
constexpr int kRedPitch = 20;     // floats of 16 sums, 4 banks apart from the next column's
constexpr int kMaxStages = 6;
constexpr int kStep = 256;        // columns of a step
constexpr int kTile = 16 * 128;   // bytes of a tile's step

enum Format { kMxfp4 = 0, kNvfp4 = 1, kInt4 = 2 };

__host__ __device__ __forceinline__ int scale_row_bytes(int fmt, int K) { return fmt == kNvfp4 ? K / 16 : K / 32; }
__host__ __device__ __forceinline__ int scale_step_bytes(int fmt) { return fmt == kNvfp4 ? 16 : 8; }

// How a launch cuts the work and its shared memory: ring of weights [stages][chunk steps][set rows][128], of scales
// [stages][1 or 2][set rows][128], both swizzled | x [cols][stride] float16 |
// sums [reds][set][chunk steps][cols][20] | barriers | exponents [16], abort flag
struct Layout {
  int steps, chunk, chunks;       // steps of K, of a copy (16 at most), copies of a set
  int set;                        // tiles of a set: set * chunk compute warps have work
  int x_stride;                   // rows of x, 64 mod 128 bytes apart
  int w_bytes, sf_bytes;          // of a ring slot
  int reds;                       // buffers of sums: two, or one where they are large
  int sf, x, red, bars, fac, total;
  __host__ __device__ Layout(int fmt, int stages, int cols, int K, int64_t tiles, int sms) {
    steps = (K + kStep - 1) / kStep;
    chunks = (steps + kWarps - 1) / kWarps;
    chunk = (steps + chunks - 1) / chunks;
    if (chunks > 1) chunk = (chunk + 1) / 2 * 2;         // so that a copy of scales starts on 16 bytes
    // as many tiles as there are warps for, but not more than leave every SM a set
    const int64_t per_sm = (tiles + sms - 1) / sms;
    set = kWarps / chunk < per_sm ? kWarps / chunk : (int)per_sm;
    x_stride = steps * kStep * 2 + 64;
    w_bytes = set * chunk * kTile;
    sf_bytes = set * kTile * ((chunk * scale_step_bytes(fmt) + 127) / 128);
    sf = stages * w_bytes;
    x = sf + stages * sf_bytes;
    red = x + cols * x_stride;
    reds = cols <= 8 ? 2 : 1;
    bars = red + reds * set * chunk * cols * kRedPitch * 4;
    fac = bars + (2 * kMaxStages + 4) * 8;
    total = fac + (kMaxRows + 1) * 4 + 1024;
  }
};

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
  int stages, sms;                // for the Layout
  int whole;                      // K is whole steps: a set's chunk is one three-dimensional copy
  int scale_tma;                  // scales come by tensor copies too, else by the lanes
  int scale_words;                // which may read 4 bytes at a time
  int x_vec;                      // rows of x are 16-byte aligned
};

// v * 2^s, |s| <= 254, by two exact factors (one rounding where the result is subnormal).
__device__ __forceinline__ float scale_pow2(float v, int s) {
  const int h = s / 2;
  return v * exp2_int(h) * exp2_int(s - h);
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// Arrives on the barrier when the thread's earlier cp.async are done (one of the arrivals that it expects).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sm100::smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts_f32(uint32_t addr, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
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
// (a & mask) ^ c in one operation.
template <uint32_t kMask>
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(r) : "r"(a), "n"(kMask), "r"(c));
  return r;
}
// 8 two's complement nibbles n0..n7 -> float16 pairs (n0, n4), (n1, n5), (n2, n6), (n3, n7).
__device__ __forceinline__ void int4_pairs(uint32_t w, uint32_t (&r)[4]) {
  const uint32_t v = w >> 8, lo = 0x64086408u, hi = 0x64806480u;        // 1024 + (n ^ 8), 1024 + 16 (n ^ 8)
  const uint32_t p[4] = {and_xor<0x000F000Fu>(w, lo), and_xor<0x00F000F0u>(w, hi), and_xor<0x000F000Fu>(v, lo),
                         and_xor<0x00F000F0u>(v, hi)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = *reinterpret_cast<const __half2*>(&p[i]);
    const __half2 q = i & 1 ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-72.0f)) : __hadd2(h, __float2half2_rn(-1032.0f));
    r[i] = *reinterpret_cast<const uint32_t*>(&q);
  }
}

// Two float32 in one register pair, for the packed operations (one instruction for both).
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
// acc += c * unit * scale, two sums at a time; the first product is exact (a power of two).
__device__ __forceinline__ void add_scaled(float& acc0, float& acc1, float c0, float c1, const float (&unit)[2],
                                           float scale) {
  uint64_t c, a = pair(acc0, acc1);
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c) : "l"(pair(c0, c1)), "l"(pair(unit[0], unit[1])));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(c), "l"(pair(scale, scale)));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(acc0), "=f"(acc1) : "l"(a));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, __half2 s) {
  const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&a), s);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// sm100::mbar_wait_warp with a time for the hardware to suspend the warp: without one a waiting warp polls, and 20
// of them took a third of the SM's issue slots.
__device__ __forceinline__ bool wait_warp(uint32_t addr, uint32_t parity, volatile int* abort_flag) {
  uint64_t t0 = 0;
  uint32_t ok = 0;
  while (true) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity), "r"(20000u)
        : "memory");
    if (__all_sync(0xFFFFFFFFu, ok)) return true;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    const bool late = t - t0 > sm100::kWaitTimeoutNs;
    if (late) {
      record_error(MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    if (__any_sync(0xFFFFFFFFu, late || *abort_flag)) return false;
  }
}

// NT: groups of 8 columns (a column is a row of x, or one of the two halves of a
// float32 row).
template <int FMT, int NT>
__global__ void __launch_bounds__(kThreads, 1) matvec_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmS,
                                                              const Args a) {
  extern __shared__ uint8_t smem_raw[];
  // by an offset, so that the compiler still knows that it is shared memory (generic 64-bit addresses cost a third of
  // the loop's instructions)
  uint8_t* smem = smem_raw + (-sm100::smem_u32(smem_raw) & 1023u);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = threadIdx.x;
  const int P = a.x_type == MOE_TYPE_F32 ? 2 : 1, cols = a.M * P;
  const int tiles = (a.N + 15) / 16;
  const Layout lay(FMT, a.stages, cols, a.K, tiles, a.sms);
  const int steps = lay.steps, stages = a.stages, workers = lay.set * lay.chunk, sets = (tiles + lay.set - 1) / lay.set;
  const int srow = scale_row_bytes(FMT, a.K);             // scale bytes of a row (INT4: K / 128 floats)
  constexpr int kSfStep = FMT == kNvfp4 ? 16 : 8;         // of a row and step
  const int xs_stride = lay.x_stride;
  uint8_t* xs = smem + lay.x;
  float* red = reinterpret_cast<float*>(smem + lay.red);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + lay.bars);
  uint64_t* empty = full + kMaxStages;
  uint64_t* red_full = empty + kMaxStages;
  uint64_t* red_empty = red_full + 2;
  int* fac = reinterpret_cast<int*>(smem + lay.fac);      // exponent of each row's factor
  volatile int* abort_flag = fac + kMaxRows;
  pdl_trigger();
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      sm100::mbar_init(&full[i], a.scale_tma ? 1 : 33);
      sm100::mbar_init(&empty[i], workers);
    }
    for (int i = 0; i < lay.reds; ++i) {
      sm100::mbar_init(&red_full[i], workers);
      sm100::mbar_init(&red_empty[i], kReducers);
    }
    sm100::fence_mbar_init();
  }
  if (tid <= kMaxRows) fac[tid] = 0;      // and the abort flag
  __syncthreads();
  pdl_wait();

  // ---- copies: one chunk of a set a slot ----
  int fset = blockIdx.x, fchunk = 0, issued = 0;
  uint32_t fslot = 0, fphase = 0;         // the copies' warp; of its next slot
  auto fetch = [&]() {                    // the slot is free; whole warp
    uint64_t* bar = &full[fslot];
    uint8_t* wdst = smem + fslot * lay.w_bytes;
    uint8_t* sdst = smem + lay.sf + fslot * lay.sf_bytes;
    const int n0 = fset * lay.set * 16, rows = min(lay.set * 16, a.N - n0), step0 = fchunk * lay.chunk;
    const int todo = min(lay.chunk, steps - step0), sf0 = step0 * kSfStep;
    if (!a.scale_tma) {
      // the same swizzled rows by the lanes, zeros past K (plain stores are
      // released by the elected thread's arrival)
      const int words = todo * kSfStep / 4, have = min(todo * kSfStep, srow - sf0);
      const int lanes = 32 >> max(__clz(words - 1) - 27, 0), dr = 32 / lanes;      // lanes of a row: 2^n >= words
      for (int c = (lane & (lanes - 1)) * 4; c < words * 4; c += 128) {
        const uint8_t* p = a.scale + (int64_t)(n0 + lane / lanes) * srow + sf0 + c;
        uint8_t* dst = sdst + (c >> 7) * lay.set * kTile;
        if (a.scale_words) {
#pragma unroll 4
          for (int r = lane / lanes; r < rows; r += dr, p += dr * srow) {
            uint8_t* d = dst + r * 128 + ((c & 127) ^ ((r & 7) << 4));
            if (c < have) cp_async4(sm100::smem_u32(d), p);
            else *reinterpret_cast<uint32_t*>(d) = 0u;
          }
        } else {
#pragma unroll 4
          for (int r = lane / lanes; r < rows; r += dr, p += dr * srow) {
            uint32_t w = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) w |= (c + j < have ? (uint32_t)__ldg(p + j) : 0u) << (8 * j);
            *reinterpret_cast<uint32_t*>(dst + r * 128 + ((c & 127) ^ ((r & 7) << 4))) = w;
          }
        }
      }
      cp_async_arrive(bar);
    }
    __syncwarp();
    if (sm100::elect_one()) {
      sm100::mbar_arrive_expect_tx(bar, (a.whole ? lay.chunk : todo) * lay.set * kTile + (a.scale_tma ? lay.sf_bytes : 0));
      if (a.whole) {
        sm100::tma_load_3d(wdst, &tmW, 0, n0, step0, bar);
      } else {
        for (int s = 0; s < todo; ++s)
          sm100::tma_load_2d(wdst + s * lay.set * kTile, &tmW, (step0 + s) * 128, n0, bar);
      }
      if (a.scale_tma)
        for (int b = 0; b * lay.set * kTile < lay.sf_bytes; ++b)
          sm100::tma_load_2d(sdst + b * lay.set * kTile, &tmS, sf0 + b * 128, n0, bar);
    }
    __syncwarp();
    ++issued;
    if (++fchunk == lay.chunks) {
      fchunk = 0;
      fset += gridDim.x;
    }
    if (++fslot == (uint32_t)stages) {
      fslot = 0;
      fphase ^= 1u;
    }
  };
  if (warp == kProducer)
    for (int s = 0; s < stages && fset < sets; ++s) fetch();

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
  // the power of two of a row takes its largest value to [2^14, 2^15)
  const bool once = tasks <= 4 * kWarps;  // every task in one batch: x is read once
  float v4[4][8];
  for (int t0 = warp; warp < kWarps && t0 < tasks; t0 += 4 * kWarps) {
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
    fac[tid] = mx > 0 ? max(mx >> 23, 1) - 127 - 14 : 0;        // exponent of the factor of y
  }
  __syncthreads();
  for (int t0 = warp; warp < kWarps && t0 < tasks; t0 += 4 * kWarps) {
    if (!once) load_tasks(t0, v4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + j * kWarps;
      if (t >= tasks) break;
      const int m = t / steps, k = (t - m * steps) * kStep + lane * 8, s = -fac[m];
      float hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = scale_pow2(v4[j][i], s);
        hi[i] = __half2float(__float2half_rn(v));
        lo[i] = P == 2 ? __half2float(__float2half_rn((v - hi[i]) * 2048.0f)) : 0.f;
      }
      auto put = [&](int col, const float (&f)[8]) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __half2 h = FMT == kInt4 ? __floats2half2_rn(f[i], f[i + 4])
                                         : __floats2half2_rn(f[2 * i], f[2 * i + 1]);
          p[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(xs + col * xs_stride + k * 2) = make_uint4(p[0], p[1], p[2], p[3]);
      };
      put(m * P, hi);
      if (P == 2) put(m * P + 1, lo);
    }
  }
  __syncthreads();

  const float glob = FMT == kNvfp4 ? __ldg(a.global) : 1.0f;
  // Rows of x below 2^14 were scaled up.  MXFP4 and INT4 take that back from
  // the sums of a group before its scale (row by row: 2^sum_exponent, exact, as
  // sums of products are at least 2^-25 or zero), so that they overflow only
  // where y does; what is left of the row's factor comes at the end.
  auto sum_exponent = [&](int m) { return FMT == kNvfp4 ? 0 : max(-100, min(0, fac[m])); };
  if (warp == kProducer) {
    while (fset < sets) {
      if (!wait_warp(sm100::smem_u32(&empty[fslot]), fphase ^ 1u, abort_flag)) break;
      fetch();
    }
  } else if (warp > kProducer) {
    // ---- y of a set: the sums of its tiles' warps; a lane takes four rows of a column ----
    uint32_t buf = 0, phase = 0;
    const int items = lay.set * cols * 4, inv = 65536 / cols + 1, chunk = lay.chunk, pitch = cols * (kRedPitch / 4);
    for (int set = blockIdx.x; set < sets; set += gridDim.x) {
      if (!wait_warp(sm100::smem_u32(&red_full[buf]), phase, abort_flag)) break;
      const float4* rb = reinterpret_cast<const float4*>(red) + buf * workers * pitch;
#pragma unroll 1
      for (int i0 = 32 * (warp - kProducer - 1); i0 < items; i0 += 32 * kReducers) {
        const int i = min(i0 + lane, items - 1), j = i >> 2;
        const int t = j * inv >> 16, col = j - t * cols, m = P == 2 ? col >> 1 : col;       // j / cols: j < 512, cols <= 32
        const float4* p = rb + t * chunk * pitch + col * (kRedPitch / 4) + (i & 3);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = 0; w < chunk; ++w, p += pitch) {
          const float4 f = *p;
          v = make_float4(v.x + f.x, v.y + f.y, v.z + f.z, v.w + f.w);
        }
        if (P == 2) {                     // the row's low parts are the next column
          v.x = fmaf(__shfl_down_sync(0xFFFFFFFFu, v.x, 4), 1.0f / 2048.0f, v.x);
          v.y = fmaf(__shfl_down_sync(0xFFFFFFFFu, v.y, 4), 1.0f / 2048.0f, v.y);
          v.z = fmaf(__shfl_down_sync(0xFFFFFFFFu, v.z, 4), 1.0f / 2048.0f, v.z);
          v.w = fmaf(__shfl_down_sync(0xFFFFFFFFu, v.w, 4), 1.0f / 2048.0f, v.w);
        }
        // NVFP4 (sums below 2^43, and at least 2^-34 or zero): the global factor between two parts of the row's, of
        // which neither overflows nor loses bits unless y does
        const int n = (set * lay.set + t) * 16 + (i & 3) * 4, s = fac[m] - sum_exponent(m);
        const int first = FMT == kNvfp4 ? max(-80, min(80, s)) : 0;
        const float s0 = exp2_int(first), s1 = exp2_int(s - first);
        auto result = [&](float f) { return FMT == kNvfp4 ? f * s0 * glob * s1 : f * s1; };
        const float y[4] = {result(v.x), result(v.y), result(v.z), result(v.w)};
        const int left = i0 + lane < items && (P == 1 || (col & 1) == 0) ? a.N - n : 0;
        const int64_t at = m * a.ldout + n;
        if (a.out_type == MOE_TYPE_F32) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (r < left) static_cast<float*>(a.out)[at + r] = y[r];
        } else if (a.out_type == MOE_TYPE_BF16) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (r < left) static_cast<__nv_bfloat16*>(a.out)[at + r] = __float2bfloat16_rn(y[r]);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (r < left) static_cast<__half*>(a.out)[at + r] = __float2half_rn(y[r]);
        }
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(&red_empty[buf]);
      if (++buf == (uint32_t)lay.reds) {
        buf = 0;
        phase ^= 1u;
      }
    }
  } else if (warp < workers) {
    // the loop below is issue-bound: its addresses are kept, not computed
    const int g = lane >> 2, q = lane & 3, tg = warp / lay.chunk, st = warp - tg * lay.chunk, chunks = lay.chunks;
    uint32_t x_lane[NT];                  // the lane's column of the token operand (past the last one: any)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      x_lane[nt] = sm100::smem_u32(xs) + min(nt * 8 + g, cols - 1) * xs_stride + q * 16 + st * kStep * 2;
    // ldmatrix: lane l names row l % 8 of matrix l / 8, a 16-byte chunk of the swizzled tile (the second half's: ^ 64)
    const uint32_t w_bytes = lay.w_bytes, sf_bytes = lay.sf_bytes, bar0 = sm100::smem_u32(full);
    const uint32_t w_first = sm100::smem_u32(smem) + (st * lay.set + tg) * kTile + (lane & 7) * 128 +
                             (((lane >> 3) ^ (lane & 7)) << 4);
    const uint32_t s_first = sm100::smem_u32(smem + lay.sf) + ((st * kSfStep) >> 7) * lay.set * kTile + (tg * 16 + g) * 128 +
                             (((st * kSfStep) & 127) ^ (g << 4));
    const uint32_t r_first = sm100::smem_u32(red) + (warp * cols + 2 * q) * kRedPitch * 4 + g * 4;
    const uint32_t r_bytes = workers * cols * kRedPitch * 4, rbar0 = sm100::smem_u32(red_full);
    const uint32_t sel16 = q >= 2 ? 0x3232u : 0x1010u;   // NVFP4: the lane's half of a pair of scales, twice
    const bool two = lay.reds == 2;
    float unit[NT][2];                    // of the lane's two columns in each group of 8
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) unit[nt][i] = exp2_int(sum_exponent(min(nt * 8 + 2 * q + i, cols - 1) / P));
    // one step of 8 columns: kept where a warp's step is always the same
    uint4 xr[8];
    uint32_t w_lane = w_first, s_lane = s_first, bar = bar0, slots = stages, phase = 0, buf = 0, red_phase = 0;
    bool ok = true;
    int tile = blockIdx.x * lay.set + tg;
    for (int set = blockIdx.x; set < sets && ok; set += gridDim.x, tile += gridDim.x * lay.set) {
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.f;
      for (int ch = 0; ch < chunks; ++ch) {
        ok = wait_warp(bar, phase, abort_flag);
        if (!ok) break;
        const int step0 = ch * lay.chunk;
        const bool mine = tile < tiles && step0 + st < steps;
        if (NT == 1 && mine && (chunks > 1 || set == (int)blockIdx.x)) {
#pragma unroll
          for (int s = 0; s < 8; ++s) xr[s] = lds128(x_lane[0] + step0 * kStep * 2 + s * 64);
        }
        uint32_t ua[2][4], ub[2][4];
        uint4 ma = make_uint4(0u, 0u, 0u, 0u), mb = ma;
        if (mine) {
          ldmatrix4(ua[0], w_lane);
          ldmatrix4(ub[0], w_lane + 1024);
          ldmatrix4(ua[1], w_lane ^ 64u);
          ldmatrix4(ub[1], (w_lane ^ 64u) + 1024);
          if (FMT == kNvfp4) {
            ma = lds128(s_lane);
            mb = lds128(s_lane + 1024);
          } else {
            const uint2 t0 = lds64(s_lane), t8 = lds64(s_lane + 1024);
            ma.x = t0.x, ma.y = t0.y, mb.x = t8.x, mb.y = t8.y;
          }
        }
        __syncwarp();                     // every lane has read the slot
        if (lane == 0) arrive(bar + 8 * kMaxStages);
        bar += 8;
        w_lane += w_bytes;
        s_lane += sf_bytes;
        if (--slots == 0) {
          slots = stages;
          bar = bar0;
          w_lane = w_first;
          s_lane = s_first;
          phase ^= 1u;
        }
        if (!mine) continue;
        float c[NT][4];                                  // sums of a group (MXFP4), a half (INT4) or the step
#pragma unroll
        for (int half = 0; half < 2; ++half) {           // 128 columns each
          const uint32_t* u0 = ua[half];
          const uint32_t* u8 = ub[half];
          float f0[4], f8[4];                            // MXFP4: scales of the four groups
          __half2 h0[4], h8[4];                          // NVFP4: scales of the lane's columns in each group
          if (FMT == kMxfp4) {
            const uint32_t m0 = half ? ma.y : ma.x, m8 = half ? mb.y : mb.x;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t t0, t8;
              asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(t0) : "h"((uint16_t)(m0 >> (16 * i))));
              asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(t8) : "h"((uint16_t)(m8 >> (16 * i))));
              f0[2 * i] = bf16_lo(t0);
              f0[2 * i + 1] = bf16_hi(t0);
              f8[2 * i] = bf16_lo(t8);
              f8[2 * i + 1] = bf16_hi(t8);
            }
          }
          if (FMT == kNvfp4) {
            const uint2 m0 = half ? make_uint2(ma.z, ma.w) : make_uint2(ma.x, ma.y);
            const uint2 m8 = half ? make_uint2(mb.z, mb.w) : make_uint2(mb.x, mb.y);
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
              const uint4 b = NT == 1 ? xr[half * 4 + s] : lds128(x_lane[nt] + step0 * kStep * 2 + half * 256 + s * 64);
              if ((FMT == kInt4 && s > 0) || (FMT == kNvfp4 && half + s > 0)) {
                mma_f16(c[nt], r0[0], r8[0], r0[1], r8[1], b.x, b.y);
                mma_f16(c[nt], r0[2], r8[2], r0[3], r8[3], b.z, b.w);
              } else {
                mma_f16_first(c[nt], r0[0], r8[0], r0[1], r8[1], b.x, b.y);
                mma_f16(c[nt], r0[2], r8[2], r0[3], r8[3], b.z, b.w);
              }
              if (FMT == kMxfp4) {
                add_scaled(acc[nt][0], acc[nt][1], c[nt][0], c[nt][1], unit[nt], f0[s]);
                add_scaled(acc[nt][2], acc[nt][3], c[nt][2], c[nt][3], unit[nt], f8[s]);
              }
            }
          }
          if (FMT == kInt4) {
            const float i0 = __uint_as_float(half ? ma.y : ma.x), i8 = __uint_as_float(half ? mb.y : mb.x);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              acc[nt][0] = fmaf(c[nt][0] * unit[nt][0], i0, acc[nt][0]);
              acc[nt][1] = fmaf(c[nt][1] * unit[nt][1], i0, acc[nt][1]);
              acc[nt][2] = fmaf(c[nt][2] * unit[nt][0], i8, acc[nt][2]);
              acc[nt][3] = fmaf(c[nt][3] * unit[nt][1], i8, acc[nt][3]);
            }
          }
        }
        if (FMT == kNvfp4) {              // the tensor core truncates: steps are added here, rounded to nearest
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] += c[nt][i];
        }
      }
      if (!ok || !wait_warp(rbar0 + 16 + buf * 8, red_phase ^ 1u, abort_flag)) break;
      const uint32_t r_lane = r_first + (buf ? r_bytes : 0u);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (nt * 8 + 2 * q + (i & 1) < cols) sts_f32(r_lane + ((nt * 8 + (i & 1)) * kRedPitch + 8 * (i >> 1)) * 4, acc[nt][i]);
      }
      __syncwarp();
      if (lane == 0) arrive(rbar0 + buf * 8);
      if (two) buf ^= 1u;
      if (buf == 0) red_phase ^= 1u;
    }
  }
  // after a wait has given up: the copies still on their way (bounded)
  __syncthreads();
  if (warp == kProducer && *abort_flag) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    const uint64_t t0 = globaltimer_ns();
    for (int i = min(issued, stages); i > 0; --i) {
      if (fslot == 0) {
        fslot = stages;
        fphase ^= 1u;
      }
      --fslot;
      while (!sm100::mbar_try_wait(sm100::smem_u32(&full[fslot]), fphase) &&
             globaltimer_ns() - t0 < sm100::kWaitTimeoutNs) {
      }
    }
  }
}

}  // namespace matvec
}  // namespace moe

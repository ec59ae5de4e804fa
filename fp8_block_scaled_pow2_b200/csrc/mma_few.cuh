// Tensor-core inner step of the kernels for a few tokens: a tile of 16 weight
// rows times the E4M3 values of a few tokens, by mma.sync m16n8k32 on FP8.
//
// These kernels are bound by the stream of 4-bit weights, so what counts is
// the work per weight.  Only a handful of the instruction's 8 columns are
// needed for tokens; the others separate the scale groups.  A lane (g = lane
// / 4, q = lane % 4) holds 16 bytes of row g: the 32 weights of scale group q
// of a 128-wide K step (and the same of row g + 8).  They are used as the
// lane's k slots of four MMAs, so one MMA sums over all four groups at once;
// column n of the token operand is the token of column set n / 4, zero outside
// group n % 4, so that the four groups end in four columns: two column sets an
// MMA.  Weights then go from one 16-byte shared-memory read to the MMA with a
// conversion between (7 logic operations per 8 weights), no transposition,
// and the group scales are applied to 4 accumulators per 64 weights of a lane
// rather than to 16.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace moe {
namespace fewmma {

// Token operand: 128 columns of one token as E4M3, 128 bytes: for group c and
// j = 0..3 the 8 bytes at 32 c + 8 j are elements 32 c + 8 j + {0, 2, 4, 6}
// then {1, 3, 5, 7}: the order in which a word's nibbles come apart.
__device__ __forceinline__ uint2 pack_evens_odds(const float (&v)[8]) {
  return make_uint2(e4m3x4(v[0], v[2], v[4], v[6]), e4m3x4(v[1], v[3], v[5], v[7]));
}

// 8 E2M1 nibbles -> E4M3 bytes worth 2^-6 of their value (E2M1's exponent and
// mantissa bits are E4M3's low exponent and high mantissa bits, subnormals
// included): even elements in lo, odd ones in hi.
constexpr float kE2m1Unit = 64.0f;
__device__ __forceinline__ void e2m1_words(uint32_t w, uint32_t& lo, uint32_t& hi) {
  lo = ((w << 4) & 0x80808080u) | ((w << 2) & 0x1C1C1C1Cu);
  hi = (w & 0x80808080u) | ((w >> 2) & 0x1C1C1C1Cu);
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two E8M0 bytes -> two floats 2^(b - 127) (exact; 255 is NaN).
__device__ __forceinline__ float2 e8m0x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return make_float2(bf16_lo(r), bf16_hi(r));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A converted 16-row tile of one K step: a lane's weights of rows g and g + 8
// as MMA operands, and the scales of the two groups whose sums it receives.
struct TileA {
  uint32_t a[4][4];
};
__device__ __forceinline__ void load_tile(TileA& t, const uint8_t* row0, const uint8_t* row8) {
  const uint4 u = *reinterpret_cast<const uint4*>(row0), v = *reinterpret_cast<const uint4*>(row8);
  const uint32_t uw[4] = {u.x, u.y, u.z, u.w}, vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    e2m1_words(uw[j], t.a[j][0], t.a[j][2]);
    e2m1_words(vw[j], t.a[j][1], t.a[j][3]);
  }
}

struct TokB {
  uint32_t b[8];
};
// p: the lane's 32 bytes of its column set's token, nullptr for zeros.
__device__ __forceinline__ void load_tok(TokB& t, const uint8_t* p) {
  uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
  if (p) {
    u = *reinterpret_cast<const uint4*>(p);
    v = *reinterpret_cast<const uint4*>(p + 16);
  }
  t.b[0] = u.x; t.b[1] = u.y; t.b[2] = u.z; t.b[3] = u.w;
  t.b[4] = v.x; t.b[5] = v.y; t.b[6] = v.z; t.b[7] = v.w;
}

__device__ __forceinline__ void tile_mma(float (&c)[4], const TileA& a, const TokB& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) mma_e4m3(c, a.a[j][0], a.a[j][1], a.a[j][2], a.a[j][3], b.b[2 * j], b.b[2 * j + 1]);
}

}  // namespace fewmma
}  // namespace moe

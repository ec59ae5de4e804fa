// The whole MoE layer for a few tokens (T <= 16) with MXFP4 experts.
//
// A step for a few tokens is a stream of weights: one token of the 256-expert
// layer reads 7 experts (94 MB) and multiplies each weight once, so the time
// goes to launches and hand-overs between the grouped calls rather than to
// work.
#pragma once

#include "common.cuh"
#include "elementwise.cuh"
#include "matvec4.cuh"

namespace moe {
namespace few {

constexpr int kMaxTokens = 16;
constexpr int kMaxWidth = 8192;         // H and I: one row in a block's shared memory
constexpr int kWBlock = 8192 + 512;     // prepared weight block (moe_prepare_weights)

struct Args {
  const uint16_t* x;            // bf16 [T, H]
  const float* logits;          // [T, E]
  const uint8_t* w13;           // prepared, paired order
  const uint8_t* w2;            // prepared, plain order
  int T, H, I, E, k, has_shared;
  float limit;
  int32_t* idx;                 // [T, k]
  float* w;                     // [T, k]
  uint16_t* y;                  // bf16 [T, H]
  float* h;                     // workspace: float32 [T * k + (shared) T][I]
};

// ------------------------------- routing ----------------------------------
// The order of a2 (value descending, ties to the lower index) as unsigned
// keys; 0 stands for a NaN or an expert already taken.  -0 counts as +0.
__device__ __forceinline__ uint32_t logit_key(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key >> 31) ? (key & 0x7FFFFFFFu) : ~key);
}

// Scored routing of one token by one warp: lane j < k gets slot j's expert
// and logit (expert -1 when fewer than k logits are numbers).
template <int V>
__device__ __forceinline__ void select_topk(const float* row, int E, int k, int& e_sel, float& z_sel) {
  const int lane = threadIdx.x & 31;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < E ? logit_key(__ldg(row + lane + 32 * i)) : 0u;
  e_sel = -1;
  z_sel = 0.f;
  for (int r = 0; r < k; ++r) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < V; ++i) best = max(best, key[i]);
    best = __reduce_max_sync(0xFFFFFFFFu, best);
    if (best == 0u) break;
    int e = 0x7FFFFFFF;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (key[i] == best) e = lane + 32 * i;
    e = __reduce_min_sync(0xFFFFFFFFu, e);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e == lane + 32 * i) key[i] = 0u;
    if (lane == r) {
      e_sel = e;
      z_sel = key_logit(best);
    }
  }
}

// Routing of token t by one warp, the arithmetic of route_topk_kernel and
// route_hash_kernel: lane j < k gets expert and weight of slot j.  Returns
// whether every slot has an expert (the same in all lanes).
__device__ __forceinline__ bool route_token(const float* logits, const int32_t* token_ids, const int32_t* tid2eid,
                                            int vocab, int E, int k, float route_scale, int route_norm, int t,
                                            int& e_sel, float& w_sel) {
  const int lane = threadIdx.x & 31;
  const float* row = logits + (int64_t)t * E;
  float z = 0.f;
  e_sel = -1;
  if (tid2eid) {
    const int id = __ldg(token_ids + t);
    if (id >= 0 && id < vocab && lane < k) {
      const int e = __ldg(tid2eid + (int64_t)id * k + lane);
      if (e >= 0 && e < E) {
        e_sel = e;
        z = __ldg(row + e);
      }
    }
  } else if (E <= 256) {
    select_topk<8>(row, E, k, e_sel, z);
  } else if (E <= 512) {
    select_topk<16>(row, E, k, e_sel, z);
  } else {
    select_topk<32>(row, E, k, e_sel, z);
  }
  const float s = lane < k && e_sel >= 0 ? sqrtf(softplus_f(z)) : 0.f;
  float sum = 0.f;
  for (int j = 0; j < k; ++j) sum += __shfl_sync(0xFFFFFFFFu, s, j);     // slot order
  w_sel = e_sel < 0 ? 0.f : (route_norm ? route_scale * __fdiv_rn(s, sum) : route_scale * s);
  return __all_sync(0xFFFFFFFFu, lane >= k || e_sel >= 0);
}

struct Routing {
  const int32_t* token_ids;
  const int32_t* tid2eid;
  int vocab;
  float route_scale;
  int route_norm;
};

// One warp per token.
__global__ void __launch_bounds__(32) route_kernel(const Args a, const Routing r) {
  pdl_trigger();
  pdl_wait();
  int e;
  float w;
  const int t = blockIdx.x, lane = threadIdx.x;
  const bool ok = route_token(a.logits, r.token_ids, r.tid2eid, r.vocab, a.E, a.k, r.route_scale, r.route_norm, t, e, w);
  if (!ok && lane == 0) record_error(MOE_ERR_INVALID);
  if (lane < a.k) {
    a.idx[t * a.k + lane] = e;
    a.w[t * a.k + lane] = w;
  }
}

// Quantise-dequantise 128 columns held 4 per lane (the a1 rule): returns the
// values the tensor path sees, exact in float32.
__device__ __forceinline__ void quant_dequant4(float (&v)[4]) {
  const float m = warp_max_nonneg(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
  const int k = pow2_scale_exponent(m);
  const float sc = exp2_int(-k), inv = exp2_int(k);
  const uint32_t q = e4m3x4(__fmul_rn(v[0], sc), __fmul_rn(v[1], sc), __fmul_rn(v[2], sc), __fmul_rn(v[3], sc));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = matvec::e4m3_to_float((uint8_t)(q >> (8 * i))) * inv;
}

// sum_k row[k] * weight(row m of the prepared blocks `blk`, block stride `bs`)
// by one warp: lane l holds columns 4 l .. 4 l + 3 of each 128-wide step.
__device__ __forceinline__ float prepared_dot(const uint8_t* blk, int64_t bs, int m, int KT, const float* row) {
  const int lane = threadIdx.x & 31;
  float acc = 0.f;
  for (int kt = 0; kt < KT; ++kt) {
    const uint8_t* b = blk + kt * bs;
    const uint32_t n = *reinterpret_cast<const uint16_t*>(b + m * 64 + 2 * lane);
    const float s = matvec::e8m0_to_float(b[8192 + (m & 31) * 16 + (m >> 5) * 4 + (lane >> 3)]);
    const float* r = row + kt * 128 + 4 * lane;
    float p = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) p = fmaf(matvec::e2m1_to_float((n >> (4 * j)) & 15u), r[j], p);
    acc = fmaf(p, s, acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, o);
  return acc;
}

// h of one pair (routed pair t * k + j, or T * k + t for the shared expert)
// and 64 features.
__global__ void __launch_bounds__(256) gate_up_kernel(const Args a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ float row[];
  const int p = blockIdx.x, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int P = a.T * a.k;
  const int t = p < P ? p / a.k : p - P;
  const int e = p < P ? a.idx[p] : a.E;
  if (e < 0) return;
  const int KT = a.H / 128;
  for (int kt = wid; kt < KT; kt += 8) {
    float v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float((uint32_t)a.x[(int64_t)t * a.H + kt * 128 + 4 * lane + i] << 16);
    quant_dequant4(v);
#pragma unroll
    for (int i = 0; i < 4; ++i) row[kt * 128 + 4 * lane + i] = v[i];
  }
  __syncthreads();
  for (int j = wid; j < 64; j += 8) {
    const int f = blockIdx.y * 64 + j;
    const uint8_t* blk = a.w13 + ((int64_t)e * (a.I / 128) + f / 128) * KT * 2 * kWBlock;
    const float g = prepared_dot(blk, 2 * kWBlock, f % 128, KT, row);
    const float u = prepared_dot(blk + kWBlock, 2 * kWBlock, f % 128, KT, row);
    if (lane == 0) a.h[(int64_t)p * a.I + f] = swiglu_clamped(g, u, a.limit);
  }
}

// y of one token and 64 output columns: slots in order, then the shared expert.
__global__ void __launch_bounds__(256) down_kernel(const Args a) {
  pdl_trigger();
  pdl_wait();
  extern __shared__ float row[];
  const int t = blockIdx.x, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int KT = a.I / 128;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  for (int j = 0; j < a.k + (a.has_shared ? 1 : 0); ++j) {
    const int p = j < a.k ? t * a.k + j : a.T * a.k + t;
    const int e = j < a.k ? a.idx[p] : a.E;
    if (e < 0) continue;
    const float wt = j < a.k ? a.w[p] : 1.0f;
    __syncthreads();
    for (int kt = wid; kt < KT; kt += 8) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = a.h[(int64_t)p * a.I + kt * 128 + 4 * lane + i];
      quant_dequant4(v);
#pragma unroll
      for (int i = 0; i < 4; ++i) row[kt * 128 + 4 * lane + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = blockIdx.y * 64 + i * 8 + wid;
      const uint8_t* blk = a.w2 + ((int64_t)e * (a.H / 128) + n / 128) * KT * kWBlock;
      acc[i] = fmaf(wt, prepared_dot(blk, kWBlock, n % 128, KT, row), acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (lane == 0)
      reinterpret_cast<__nv_bfloat16*>(a.y)[(int64_t)t * a.H + blockIdx.y * 64 + i * 8 + wid] =
          __float2bfloat16_rn(acc[i]);
  }
}

}  // namespace few
}  // namespace moe

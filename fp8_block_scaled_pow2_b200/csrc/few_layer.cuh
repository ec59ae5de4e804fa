// The whole MoE layer for a few tokens (T <= 16) with MXFP4 experts, in two
// kernels.
//
// A step for a few tokens is a stream of weights: one token of the 256-expert
// layer reads 7 experts (94 MB, 14.3 us at the copy rate) and multiplies each
// weight once.  The grouped path (quantise, route, group, two plans and GEMMs,
// combine) spends 53 us on it, most of it in launches and hand-overs.  Here
//   gate_up_kernel   every block routes all tokens and quantises x for itself
//                    (cheaper than waiting for another kernel to do it), then
//                    computes 128-feature blocks of the chosen experts' gate
//                    and up projections, SwiGLU and the requantised h;
//   down_kernel      a cluster of blocks owns 128 output columns, splits the
//                    (expert, K) range, weights each expert's sums with the
//                    router's weights and adds the blocks' parts over
//                    distributed shared memory: y in one pass, no atomics.
// Both use the block-scaled tensor-core MMA on the prepared weights, as the
// grouped GEMM does (weight tile = the 128-row operand, tokens = 16 columns):
// the 4-bit weights are unpacked by TMA and scaled by the tensor core, so no
// instruction is spent per weight.  (A first version with FP8 mma.sync in
// registers took 60 us for one token: that instruction is emulated here, 26
// cycles a step, and the conversions alone cost 60 % of the stream's time.)
//
// The weights of down_kernel are prefetched into L2 by gate_up_kernel's blocks
// as these run out of work, so the stream from memory does not stop between
// the two.
#pragma once

#include "common.cuh"
#include "elementwise.cuh"
#include "sm100.cuh"

namespace moe {
namespace few {

using namespace sm100;

constexpr int kMaxTokens = 16;          // the MMA's N: one column per token
constexpr int kMaxWidth = 8192;         // H and I
constexpr int kWBlock = 8192 + 512;     // prepared weight block (moe_prepare_weights)
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxList = kMaxTokens * 16 + 1;     // distinct experts of a step

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
  uint8_t* hq;                  // workspace: E4M3 h, row base[d] + c: entry d's c-th token
  uint8_t* h_sf;                // workspace: scales of h as tensor-memory blocks [entry][K step / 4][512]
  int down_blocks, cluster;     // down_kernel's grid and cluster size
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

// ------------------------- experts of the step -----------------------------
// The distinct experts that the tokens chose, the same in every block: entry 0
// is the shared expert (when there is one), then the routed ones in ascending
// order.  Rows of h: entry d's tokens (set bits of mask[d], ascending) have
// rows base[d], base[d] + 1, ...
struct List {
  int expert[kMaxList];
  uint32_t mask[kMaxList];
  int base[kMaxList + 1];
  int n;                                  // entries
  uint32_t chosen[32];                    // bit e % 32 of word e / 32
  int word_at[32];                        // entry of word's first expert
  int32_t idx[kMaxTokens * 16];           // routing of the step
  float w[kMaxTokens * 16];
};

// Routing of all tokens and the list, by the whole block (the high warps
// first: the low ones have other work at that point).  `emit`: this block also
// writes the routing outputs and records errors.
__device__ __forceinline__ void build_list(List& L, const Args& a, const Routing& r, bool emit) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, tid = threadIdx.x;
  // L.chosen was cleared before a barrier
  const int t = kWarps - 1 - wid;
  if (t < a.T) {
    int e;
    float w;
    const bool ok = route_token(a.logits, r.token_ids, r.tid2eid, r.vocab, a.E, a.k, r.route_scale, r.route_norm, t, e, w);
    if (lane < a.k) {
      L.idx[t * a.k + lane] = e;
      L.w[t * a.k + lane] = w;
      if (e >= 0) atomicOr(&L.chosen[e >> 5], 1u << (e & 31));
      if (emit) {
        a.idx[t * a.k + lane] = e;
        a.w[t * a.k + lane] = w;
      }
    }
    if (emit && !ok && lane == 0) record_error(MOE_ERR_INVALID);
  }
  __syncthreads();
  const int sh = a.has_shared;
  if (tid < 32) {
    // entries before word `lane` of the bitmap, then this word's experts
    uint32_t m = L.chosen[lane];
    const int c = __popc(m);
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    int at = sh + x - c;
    L.word_at[lane] = at;
    for (; m; m &= m - 1u) {
      L.expert[at] = 32 * lane + __ffs(m) - 1;
      L.mask[at++] = 0u;
    }
    if (lane == 31) L.n = sh + x;
    if (lane == 0 && sh) {
      L.expert[0] = a.E;
      L.mask[0] = (1u << a.T) - 1u;
    }
  }
  __syncthreads();
  if (tid < a.T * a.k) {
    const int e = L.idx[tid];
    if (e >= 0)
      atomicOr(&L.mask[L.word_at[e >> 5] + __popc(L.chosen[e >> 5] & ((1u << (e & 31)) - 1u))], 1u << (tid / a.k));
  }
  __syncthreads();
  if (tid < 32) {
    int run = 0;
    for (int d0 = 0; d0 < L.n; d0 += 32) {
      const int c = d0 + lane < L.n ? __popc(L.mask[d0 + lane]) : 0;
      int x = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      if (d0 + lane < L.n) L.base[d0 + lane] = run + x - c;
      run += __shfl_sync(0xFFFFFFFFu, x, 31);
    }
    if (lane == 0) L.base[L.n] = run;
  }
  __syncthreads();
}
static_assert(kWarps == kMaxTokens && kThreads >= kMaxTokens * 16, "one warp per token, one thread per pair");

// Barriers and flags of a block.
struct Sync {
  uint64_t full[8], empty[8], acc_full[2], acc_empty[2], sf;
  uint32_t tmem;
  int abort_flag;
  int produced;                           // steps whose copies are issued
};

// After a wait has given up: the producer waits (bounded) for the copies it
// issued into the ring's last `n` slots before the block ends.  `stage` and
// `phase` are those of its next step.
__device__ __forceinline__ void drain_ring(Sync& s, int stages, int n, uint32_t stage, uint32_t phase) {
  const uint64_t t0 = globaltimer_ns();
  for (int i = 0; i < n; ++i) {
    if (stage == 0) {
      stage = stages;
      phase ^= 1u;
    }
    --stage;
    while (!mbar_try_wait(smem_u32(&s.full[stage]), phase) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
    }
  }
}

// The K steps [s0, s1) of the flattened (entry, K step) range that block
// `rank` of a cluster of `size` takes in down_kernel.
__host__ __device__ __forceinline__ int down_first(int total, int rank, int size) {
  return (int)((int64_t)total * rank / size);
}

// --------------------------- gate / up kernel -------------------------------
// Work item: (list entry, block of 128 features): the gate and the up tile of
// all K steps.  Ring slot: both tiles unpacked (2 x 16 KB) and their scale
// blocks.  All tokens' rows of x (E4M3, zero rows past T) stay in shared
// memory in the MMA's layout, their scales in tensor memory, for the whole
// kernel: every expert multiplies all 16 columns and the epilogue takes those
// of the tokens that chose it (the MMA's N is 16 at least).
constexpr int kUpStage = 2 * 16384 + 2 * 512;

struct UpSmem {
  // ring (1024-byte aligned) | x tiles [KT][2048] | x scale blocks [KG][512] | Sync | red | List
  __host__ __device__ static int x_off(int stages) { return stages * kUpStage; }
  __host__ __device__ static int sf_off(int stages, int KT) { return x_off(stages) + KT * 2048; }
  __host__ __device__ static int sync_off(int stages, int KT) { return sf_off(stages, KT) + (KT + 3) / 4 * 512; }
  __host__ __device__ static int red_off(int stages, int KT) { return sync_off(stages, KT) + (int)sizeof(Sync); }
  __host__ __device__ static int list_off(int stages, int KT) { return red_off(stages, KT) + 5 * 16 * 4; }
  __host__ __device__ static int total(int stages, int KT) {
    return list_off(stages, KT) + (int)sizeof(List) + 1024;
  }
};

__device__ __forceinline__ void init_sync(Sync& s, int stages, int consumers, int epi_threads) {
  for (int i = 0; i < stages; ++i) {
    mbar_init(&s.full[i], 1);
    mbar_init(&s.empty[i], consumers);
  }
  for (int b = 0; b < 2; ++b) {
    mbar_init(&s.acc_full[b], 2);
    mbar_init(&s.acc_empty[b], epi_threads);
  }
  mbar_init(&s.sf, 1);
  s.abort_flag = 0;
  s.produced = 0;
  fence_mbar_init();
}

__global__ void __launch_bounds__(kThreads, 1)
    gate_up_kernel(const __grid_constant__ CUtensorMap tmW, const Args a, const Routing r, int stages, int tmem_cols) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int KT = a.H / 128, KG = (KT + 3) / 4, FB = a.I / 128, sh = a.has_shared;
  uint8_t* xt = smem + UpSmem::x_off(stages);
  uint8_t* xsf = smem + UpSmem::sf_off(stages, KT);
  Sync& sy = *reinterpret_cast<Sync*>(smem + UpSmem::sync_off(stages, KT));
  float* red = reinterpret_cast<float*>(smem + UpSmem::red_off(stages, KT));     // [4][16] maxima, [16] 2^-k
  List& L = *reinterpret_cast<List*>(smem + UpSmem::list_off(stages, KT));
  volatile int* abort_flag = &sy.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;

  if (tid == 0) {
    init_sync(sy, stages, 2, 128);
    prefetch_tensormap(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(&sy.tmem, tmem_cols);
    tmem_relinquish();
  }
  if (tid < 32) L.chosen[tid] = 0u;
  for (int i = tid; i < (KT * 2048 + KG * 512) / 16; i += kThreads)
    reinterpret_cast<uint4*>(xt)[i] = make_uint4(0u, 0u, 0u, 0u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sy.tmem;
  pdl_wait();
  pdl_trigger();                          // only now: down_kernel reads the inputs before its own wait

  // ---- weights that need no routing: the shared expert's ----
  uint32_t stage = 0, phase = 0;          // the producer's
  int pre = 0;
  auto load_step = [&](int e, int pb, int kt) {
    uint8_t* st = smem + stage * kUpStage;
    const int p = (e * FB + pb) * KT + kt;
    mbar_arrive_expect_tx(&sy.full[stage], 2 * kWBlock);
    tma_load_4d(st, &tmW, 0, 0, 0, p, &sy.full[stage]);
    const uint8_t* s = a.w13 + (int64_t)p * 2 * kWBlock + 8192;
    bulk_load(st + 32768, s, 512, &sy.full[stage]);
    bulk_load(st + 32768 + 512, s + kWBlock, 512, &sy.full[stage]);
    sy.produced = sy.produced + 1;
  };
  if (warp == 0 && sh && (int)blockIdx.x < FB) {
    for (; pre < min(stages, KT); ++pre) {
      if (elect_one()) load_step(a.E, blockIdx.x, pre);
      __syncwarp();
      if (++stage == (uint32_t)stages) { stage = 0; phase ^= 1u; }
    }
  }
  if (warp == 3 && lane == 0 && sh) {
    // this block's slice of the shared expert into L2
    const int n13 = FB * KT, n2 = (a.H / 128) * FB, n = n13 + n2;
    for (int i = (int)((int64_t)blockIdx.x * n / gridDim.x); i < (int)((int64_t)(blockIdx.x + 1) * n / gridDim.x); ++i) {
      if (i < n13) bulk_prefetch(a.w13 + ((int64_t)a.E * n13 + i) * 2 * kWBlock, 2 * kWBlock);
      else bulk_prefetch(a.w2 + ((int64_t)a.E * n2 + i - n13) * kWBlock, kWBlock);
    }
  }

  // ---- x: E4M3 tiles and scale blocks; half-warps of 128 columns ----
  {
    const int groups = a.T * KT, hl = lane & 15;
    for (int p0 = warp * 2; p0 < groups; p0 += 2 * kWarps) {
      const int p = p0 + (lane >> 4);
      const bool in = p < groups;
      const int t = in ? p / KT : 0, kt = in ? p - t * KT : 0;
      const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H + kt * 128) + hl)
                         : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t wv[4] = {u.x, u.y, u.z, u.w};
      float f[8], m = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(wv[i]);
        f[2 * i + 1] = bf16_hi(wv[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const int k = pow2_scale_exponent(m);
      const float sc = exp2_int(-k);
      if (in) {
        // 128-byte swizzle: 16-byte chunk c of row t is at chunk c ^ (t % 8)
        uint8_t* dst = xt + kt * 2048 + (t >> 3) * 1024 + (t & 7) * 128 + (((hl >> 1) ^ (t & 7)) << 4) + (hl & 1) * 8;
        *reinterpret_cast<uint2*>(dst) =
            make_uint2(e4m3x4(__fmul_rn(f[0], sc), __fmul_rn(f[1], sc), __fmul_rn(f[2], sc), __fmul_rn(f[3], sc)),
                       e4m3x4(__fmul_rn(f[4], sc), __fmul_rn(f[5], sc), __fmul_rn(f[6], sc), __fmul_rn(f[7], sc)));
        if (hl == 0) xsf[(kt >> 2) * 512 + t * 16 + (kt & 3)] = (uint8_t)(k + 127);
      }
    }
  }
  fence_async_smem();                     // the tiles are read by the tensor core
  build_list(L, a, r, blockIdx.x == 0);   // ends with a barrier

  const int n_items = L.n * FB;
  constexpr int kAcc = 0, kSfa = 64, kSfb = 72;       // tensor-memory columns: 2 x (gate 16, up 16), 2 x 4, KT
  if (warp == 0) {
    // ------------------------------ producer ------------------------------
    bool ok = true;
    int issued = pre;
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
      const int d = item / FB, pb = item - d * FB, e = L.expert[d];
      for (int kt = item == (int)blockIdx.x ? pre : 0; kt < KT; ++kt) {
        if (!mbar_wait_warp(&sy.empty[stage], phase ^ 1u, abort_flag)) { ok = false; break; }
        if (elect_one()) load_step(e, pb, kt);
        __syncwarp();
        ++issued;
        if (++stage == (uint32_t)stages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok) drain_ring(sy, stages, min(issued, stages), stage, phase);
  } else if (warp == 3) {
    // ------------------------------ L2 prefetcher --------------------------
    // down_kernel's first K steps, one of its blocks per block of this
    // kernel, once this block's own copies are issued.
    if (lane == 0 && (int)blockIdx.x < a.down_blocks) {
      const int mine = n_items > (int)blockIdx.x ? ((n_items - 1 - (int)blockIdx.x) / (int)gridDim.x + 1) * KT : 0;
      const uint64_t t0 = globaltimer_ns();
      bool go = true;
      while (*reinterpret_cast<volatile int*>(&sy.produced) < mine) {
        if (*abort_flag || globaltimer_ns() - t0 > kWaitTimeoutNs) { go = false; break; }
        __nanosleep(100);
      }
      const int rb = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster, KT2 = FB, RB = a.H / 128;
      const int s0 = down_first(L.n * KT2, rank, a.cluster), s1 = down_first(L.n * KT2, rank + 1, a.cluster);
      for (int s = s0; go && s < min(s1, s0 + 32); ++s) {
        const int d = s / KT2;
        if (d < sh) continue;             // already asked for
        bulk_prefetch(a.w2 + (((int64_t)L.expert[d] * RB + rb) * KT2 + (s - d * KT2)) * kWBlock, kWBlock);
      }
    }
  } else if (warp == 1 || warp == 2) {
    // ---------------- MMA issuers: gate tile, up tile ----------------
    const int iss = warp - 1;
    if (iss == 0) {
      if (elect_one()) {
        for (int g = 0; g < KG; ++g) tmem_cp_32x128b_warpx4(tmem + kSfb + 4 * g, sdesc_sf(smem_u32(xsf + g * 512)));
        tc_commit(&sy.sf);
      }
      __syncwarp();
    }
    const uint32_t idesc = idesc_mxf8f6f4(5u /*E2M1*/, 0u /*E4M3*/, 128, 16);
    const uint32_t sfa = tmem + kSfa + 4 * iss;
    uint32_t ab = 0, acc_bits = 0, st_i = 0, ph = 0;
    bool ok = mbar_wait_warp(&sy.sf, 0, abort_flag);
    tc_fence_after();
    for (int item = blockIdx.x; item < n_items && ok; item += gridDim.x) {
      if (!mbar_wait_warp(&sy.acc_empty[ab], ((acc_bits >> ab) & 1u) ^ 1u, abort_flag)) break;
      tc_fence_after();
      const uint32_t dcol = tmem + kAcc + ab * 32 + iss * 16;
      for (int kt = 0; kt < KT; ++kt) {
        if (!mbar_wait_warp(&sy.full[st_i], ph, abort_flag)) { ok = false; break; }
        const uint32_t st = smem_u32(smem + st_i * kUpStage);
        const uint64_t da = sdesc_kmajor_sw128(st + iss * 16384), db = sdesc_kmajor_sw128(smem_u32(xt + kt * 2048));
        const uint32_t bsel = kt & 3, sfb = (tmem + kSfb + (kt >> 2) * 4) | (bsel << 30);
        if (elect_one()) {
          tmem_cp_32x128b_warpx4(sfa, sdesc_sf(st + 32768 + iss * 512));
#pragma unroll
          for (int kb = 0; kb < 4; ++kb)
            mma_mxf8f6f4(dcol, da + 2 * kb, db + 2 * kb, idesc_with_sf_ids(idesc, kb, 0) | (bsel << 4),
                         sfa | ((uint32_t)kb << 30), sfb, (kb || kt) ? 1u : 0u);
          tc_commit(&sy.empty[st_i]);
        }
        __syncwarp();
        if (++st_i == (uint32_t)stages) { st_i = 0; ph ^= 1u; }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(&sy.acc_full[ab]);
      __syncwarp();
      acc_bits ^= 1u << ab;
      ab ^= 1u;
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------- epilogue: SwiGLU and the a1 rule per token -------------
    const int q = warp & 3, f = q * 32 + lane;
    const uint32_t lane_addr = tmem + kAcc + ((uint32_t)(q * 32) << 16);
    const int KG2 = (FB + 3) / 4;
    uint32_t ab = 0, acc_bits = 0;
    for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
      const int d = item / FB, pb = item - d * FB;
      const uint32_t mask = L.mask[d];
      bool ok = mbar_wait(&sy.acc_full[ab], (acc_bits >> ab) & 1u, abort_flag);
      ok = named_bar_and(1, 128, ok);     // the four warps go on or stop together
      if (!ok) break;
      tc_fence_after();
      uint32_t g[16], u[16];
      tmem_ld16(lane_addr + ab * 32, g);
      tmem_ld16(lane_addr + ab * 32 + 16, u);
      tmem_wait_ld(g, u);
      tc_fence_before();
      mbar_arrive(&sy.acc_empty[ab]);
      float h[16];
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        if ((mask >> t) & 1u) {
          h[t] = swiglu_clamped(__uint_as_float(g[t]), __uint_as_float(u[t]), a.limit);
          const float m = warp_max_nonneg(fabsf(h[t]));
          if (lane == 0) red[q * 16 + t] = m;
        }
      }
      named_bar_sync(1, 128);
      if (f < 16 && ((mask >> f) & 1u)) {
        const float amax = fmaxf(fmaxf(red[f], red[16 + f]), fmaxf(red[32 + f], red[48 + f]));
        const int k = pow2_scale_exponent(amax);
        red[64 + f] = exp2_int(-k);
        const int c = __popc(mask & ((1u << f) - 1u));
        a.h_sf[((size_t)d * KG2 + (pb >> 2)) * 512 + c * 16 + (pb & 3)] = (uint8_t)(k + 127);
      }
      named_bar_sync(1, 128);
      uint8_t* row = a.hq + (size_t)L.base[d] * a.I + pb * 128 + f;
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        if ((mask >> t) & 1u) {
          *row = (uint8_t)(e4m3x2(__fmul_rn(h[t], red[64 + t]), 0.0f) & 0xFFu);
          row += a.I;
        }
      }
      named_bar_sync(1, 128);             // red is free again
      acc_bits ^= 1u << ab;
      ab ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, tmem_cols);
  }
}

// ------------------------------ down kernel ---------------------------------
// Block (row block rb, rank) of a cluster: K steps [s0, s1) of the flattened
// (entry, K step) range, one weight tile each.  The steps of one entry form a
// segment with its own accumulators, which the epilogue multiplies with the
// router weights of the entry's tokens and adds to the block's y (float32 in
// shared memory).  Two issuers take alternate steps (one is bound by its own
// issue latency).
constexpr int kDnStage = 16384 + 2048 + 512 + 512;     // weight tile, h tile, weight and h scales

struct DownSmem {
  // ring | y part [16][128] float32 | Sync | List
  __host__ __device__ static int y_off(int stages) { return stages * kDnStage; }
  __host__ __device__ static int sync_off(int stages) { return y_off(stages) + 16 * 128 * 4; }
  __host__ __device__ static int list_off(int stages) { return sync_off(stages) + (int)sizeof(Sync); }
  __host__ __device__ static int total(int stages) { return list_off(stages) + (int)sizeof(List) + 1024; }
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kThreads, 1)
    down_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmH, const Args a,
                const Routing r, int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  float* ys = reinterpret_cast<float*>(smem + DownSmem::y_off(stages));
  Sync& sy = *reinterpret_cast<Sync*>(smem + DownSmem::sync_off(stages));
  List& L = *reinterpret_cast<List*>(smem + DownSmem::list_off(stages));
  volatile int* abort_flag = &sy.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int KT = a.I / 128, KG = (KT + 3) / 4, RB = a.H / 128;
  const int rb = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster;
  pdl_trigger();
  if (tid == 0) {
    init_sync(sy, stages, 1, 128);
    prefetch_tensormap(&tmW);
    prefetch_tensormap(&tmH);
  }
  if (warp == 1) {
    tmem_alloc(&sy.tmem, 128);
    tmem_relinquish();
  }
  if (tid < 32) L.chosen[tid] = 0u;
  for (int i = tid; i < 16 * 128; i += kThreads) ys[i] = 0.f;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sy.tmem;
  // Routing and weights are inputs of the call, complete before gate_up_kernel
  // let this kernel start (it does so after its own wait): read before the wait.
  build_list(L, a, r, false);
  const int total = L.n * KT;
  const int s0 = down_first(total, rank, a.cluster), s1 = down_first(total, rank + 1, a.cluster);
  constexpr int kAcc = 0, kSf = 64;       // tensor-memory columns: 2 x 2 partial sums of 16; per issuer 4 + 4 of scales

  if (warp == 0) {
    // ------------------------------ producer ------------------------------
    auto load_w = [&](int s, uint32_t stage) {
      const int d = s / KT, kt = s - d * KT, blk = L.expert[d] * RB + rb;
      uint8_t* st = smem + stage * kDnStage;
      mbar_arrive_expect_tx(&sy.full[stage], kWBlock + 2048 + 512);
      tma_load_4d(st, &tmW, 0, 0, kt, blk, &sy.full[stage]);
      bulk_load(st + 18432, a.w2 + ((int64_t)blk * KT + kt) * kWBlock + 8192, 512, &sy.full[stage]);
    };
    auto load_h = [&](int s, uint32_t stage) {
      const int d = s / KT, kt = s - d * KT;
      uint8_t* st = smem + stage * kDnStage;
      tma_load_2d(st + 16384, &tmH, kt * 128, L.base[d], &sy.full[stage]);
      bulk_load(st + 18944, a.h_sf + ((size_t)d * KG + (kt >> 2)) * 512, 512, &sy.full[stage]);
    };
    // the first weights before gate_up_kernel has ended, h after it
    const int pre = min(stages, s1 - s0);
    for (int i = 0; i < pre; ++i) {
      if (elect_one()) load_w(s0 + i, i);
      __syncwarp();
    }
    pdl_wait();
    for (int i = 0; i < pre; ++i) {
      if (elect_one()) load_h(s0 + i, i);
      __syncwarp();
    }
    uint32_t stage = pre == stages ? 0 : pre, phase = pre == stages ? 1 : 0;
    for (int s = s0 + pre; s < s1; ++s) {
      if (!mbar_wait_warp(&sy.empty[stage], phase ^ 1u, abort_flag)) {
        drain_ring(sy, stages, stages, stage, phase);
        break;
      }
      if (elect_one()) {
        load_w(s, stage);
        load_h(s, stage);
      }
      __syncwarp();
      if (++stage == (uint32_t)stages) { stage = 0; phase ^= 1u; }
    }
  } else if (warp == 1 || warp == 2) {
    // ---------------- MMA issuers: alternate steps of a segment ----------------
    const int iss = warp - 1;
    const uint32_t idesc = idesc_mxf8f6f4(5u /*E2M1*/, 0u /*E4M3*/, 128, 16);
    const uint32_t sfa = tmem + kSf + 8 * iss, sfb_t = sfa + 4;
    uint32_t ab = 0, acc_bits = 0, st_i = 0, ph = 0;
    bool ok = true;
    for (int s = s0; s < s1 && ok;) {
      const int d = s / KT, e = min(s1, (d + 1) * KT);
      if (!mbar_wait_warp(&sy.acc_empty[ab], ((acc_bits >> ab) & 1u) ^ 1u, abort_flag)) break;
      tc_fence_after();
      const uint32_t dcol = tmem + kAcc + ab * 32 + iss * 16;
      for (int j = 0; s < e; ++s, ++j) {
        if ((j & 1) == iss) {
          if (!mbar_wait_warp(&sy.full[st_i], ph, abort_flag)) { ok = false; break; }
          const uint32_t st = smem_u32(smem + st_i * kDnStage);
          const uint64_t da = sdesc_kmajor_sw128(st), db = sdesc_kmajor_sw128(st + 16384);
          const uint32_t bsel = (s - d * KT) & 3, sfb = sfb_t | (bsel << 30);
          if (elect_one()) {
            tmem_cp_32x128b_warpx4(sfa, sdesc_sf(st + 18432));
            tmem_cp_32x128b_warpx4(sfb_t, sdesc_sf(st + 18944));
#pragma unroll
            for (int kb = 0; kb < 4; ++kb)
              mma_mxf8f6f4(dcol, da + 2 * kb, db + 2 * kb, idesc_with_sf_ids(idesc, kb, 0) | (bsel << 4),
                           sfa | ((uint32_t)kb << 30), sfb, (kb || j > 1) ? 1u : 0u);
            tc_commit(&sy.empty[st_i]);
          }
          __syncwarp();
        }
        if (++st_i == (uint32_t)stages) { st_i = 0; ph ^= 1u; }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(&sy.acc_full[ab]);
      __syncwarp();
      acc_bits ^= 1u << ab;
      ab ^= 1u;
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------- epilogue: router weights, the block's part of y ----------
    const int q = warp & 3, f = q * 32 + lane;
    const uint32_t lane_addr = tmem + kAcc + ((uint32_t)(q * 32) << 16);
    uint32_t ab = 0, acc_bits = 0;
    for (int s = s0; s < s1;) {
      const int d = s / KT, e = min(s1, (d + 1) * KT);
      const int expert = L.expert[d];
      const bool two = e - s > 1;
      s = e;
      if (!mbar_wait_warp(&sy.acc_full[ab], (acc_bits >> ab) & 1u, abort_flag)) break;
      tc_fence_after();
      uint32_t v[16], u[16];
      tmem_ld16(lane_addr + ab * 32, v);
      tmem_ld16(lane_addr + ab * 32 + 16, u);
      tmem_wait_ld(v, u);
      tc_fence_before();
      mbar_arrive(&sy.acc_empty[ab]);
      uint32_t m = L.mask[d];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        if (m) {
          const int t = __ffs(m) - 1;
          m &= m - 1u;
          float w = 1.0f;
          if (expert != a.E) {
            w = 0.f;
            for (int j = 0; j < a.k; ++j)
              if (L.idx[t * a.k + j] == expert) w += L.w[t * a.k + j];
          }
          const float o = two ? __uint_as_float(v[c]) + __uint_as_float(u[c]) : __uint_as_float(v[c]);
          ys[t * 128 + f] = fmaf(w, o, ys[t * 128 + f]);
        }
      }
      acc_bits ^= 1u << ab;
      ab ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
  // ---- the cluster's parts, in rank order ----
  cluster_sync();
  for (int i = rank * kThreads + tid; i < a.T * 64; i += a.cluster * kThreads) {
    const int t = i >> 6, c2 = (i & 63) * 2;
    float v0 = 0.f, v1 = 0.f;
    for (int p = 0; p < a.cluster; ++p) {
      const uint32_t src = cluster_addr(ys + t * 128 + c2, p);
      v0 += ld_cluster_f32(src);
      v1 += ld_cluster_f32(src + 4);
    }
    *reinterpret_cast<__nv_bfloat162*>(a.y + (int64_t)t * a.H + rb * 128 + c2) = __floats2bfloat162_rn(v0, v1);
  }
  cluster_sync();                         // the parts stay until every block has read them
}

}  // namespace few
}  // namespace moe

// The whole MoE layer for a few tokens (T <= 16) with MXFP4 experts, in two
// kernels.
//
// A step for a few tokens is a stream of weights: one token of the 256-expert
// layer reads 7 experts (94 MB, 14.3 us at the copy rate) and multiplies each
// weight once.  The grouped path (quantise, route, group, two plans and GEMMs,
// combine) spends 53 us on it, most of it in launches and hand-overs.  Here
//   quant_rows_kernel  quantises x (a1) and clears the counters below;
//   few_layer_kernel   one cooperative launch for the rest.  Every block routes
//                      all tokens for itself (cheaper than waiting for another
//                      kernel to do it) and then runs two phases through one
//                      ring of weight tiles: 128-feature blocks of the chosen
//                      experts' gate and up projections with SwiGLU and the
//                      requantisation of h, then its share of the down
//                      projection's (row blocks, expert, K) range.
// The copies of the second phase follow those of the first without a pause;
// only the rows of h wait, per expert, for a counter that the first phase's
// epilogues advance.  (As two kernels with programmatic launch the hand-over
// left memory idle for 5 to 7 us.)  The parts of y that different blocks hold
// are summed in block order by the last one to finish (a second counter), so
// the result does not depend on timing and needs no third kernel.
//
// The products run on the block-scaled tensor-core MMA as in the grouped GEMM
// (weight tile = the 128-row operand, tokens = 16 columns): TMA unpacks the
// 4-bit weights and the tensor core scales them, so no instruction is spent
// per weight.  (Register MMAs were tried first, 60 us for one token: FP8
// mma.sync is emulated on this target, 26 cycles a step, and the conversions
// alone took 60 % of the stream's time.)
//
// Measured (one B200, captured in a graph, 256 experts of 4096 x 2048, top-6 and
// the shared one): 1 token 30.6 us, 2 43.7, 4 63.7, 8 104, 16 180; the grouped
// path takes 55, 71, 89, 127 and 204.  16 tokens through 384 experts: 194 us on
// one layer's weights (6.0 TB/s), 203 to 213 over three layers' in turn (5.4 to
// 5.7).  From 8 tokens on the stream of weights is the bound; below, what one
// after another cannot overlap: launch and routing, the first tiles' latency,
// the last rows of h between the phases, the sum of y's parts (a layer with
// almost no weights takes 20 us).
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
  // workspace
  uint8_t* xq;                  // E4M3 x [T, H]
  uint8_t* x_sf;                // its scales as tensor-memory blocks [K step / 4][256]
  uint8_t* hq;                  // E4M3 h, row base[d] + c: entry d's c-th token
  uint8_t* h_sf;                // its scales [entry][K step / 4][256]
  int* done;                    // counters: feature blocks of each entry, then parts of each row pair
  float* part;                  // parts of y [block][2][T][256]
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
// and logit (expert -1 when fewer than k logits are numbers).  V: logits of a
// lane (experts lane, lane + 32, ...), in registers: a round over 256 experts
// is two warp reductions and 24 compares (rescanning only the winner's lane
// from memory instead took 1 us a round).
template <int V>
__device__ __forceinline__ void select_topk(const float* row, int E, int k, int& e_sel, float& z_sel) {
  const int lane = threadIdx.x & 31;
  uint32_t key[V];
#pragma unroll
  for (int i = 0; i < V; ++i) key[i] = lane + 32 * i < E ? logit_key(__ldg(row + lane + 32 * i)) : 0u;
  e_sel = -1;
  z_sel = 0.f;
#pragma unroll 1
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

struct Routing {
  const int32_t* token_ids;
  const int32_t* tid2eid;
  int vocab;
  float route_scale;
  int route_norm;
};

// Routing of token t by one warp: lane j < k gets slot j's expert (-1: none)
// and logit ...
__device__ __forceinline__ void route_experts(const Args& a, const Routing& r, int t, int& e_sel, float& z) {
  const int lane = threadIdx.x & 31;
  const float* row = a.logits + (int64_t)t * a.E;
  z = 0.f;
  e_sel = -1;
  if (r.tid2eid) {
    const int id = __ldg(r.token_ids + t);
    if (id >= 0 && id < r.vocab && lane < a.k) {
      const int e = __ldg(r.tid2eid + (int64_t)id * a.k + lane);
      if (e >= 0 && e < a.E) {
        e_sel = e;
        z = __ldg(row + e);
      }
    }
  } else if (a.E <= 256) {
    select_topk<8>(row, a.E, a.k, e_sel, z);
  } else if (a.E <= 512) {
    select_topk<16>(row, a.E, a.k, e_sel, z);
  } else {
    select_topk<32>(row, a.E, a.k, e_sel, z);
  }
}
// ... and its weight, by the arithmetic of route_topk_kernel and
// route_hash_kernel (sums in slot order).
__device__ __forceinline__ float route_weight(const Args& a, const Routing& r, int e_sel, float z) {
  const float s = (int)(threadIdx.x & 31) < a.k && e_sel >= 0 ? sqrtf(softplus_f(z)) : 0.f;
  float sum = 0.f;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xFFFFFFFFu, s, j);
  return e_sel < 0 ? 0.f : (r.route_norm ? r.route_scale * __fdiv_rn(s, sum) : r.route_scale * s);
}

// L2 prefetch of `bytes` bytes by one warp, through the load/store unit: bulk
// prefetches would queue with the block's own TMA copies (they held x back by
// 3 us).
__device__ __forceinline__ void warp_prefetch(const uint8_t* p, int bytes) {
  for (int o = (threadIdx.x & 31) * 128; o < bytes; o += 32 * 128)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p + o) : "memory");
}

// ------------------------- experts of the step -----------------------------
// The distinct experts that the tokens chose, the same in every block: entry 0
// is the shared expert (when there is one), then the routed ones in ascending
// order.  Rows of h: entry d's tokens (set bits of mask[d], ascending) have
// rows base[d], base[d] + 1, ...
struct List {
  int expert[kMaxList];
  uint32_t mask[kMaxList];                // zero before build_list
  int base[kMaxList + 1];
  int n;                                  // entries
  uint32_t chosen[32];                    // bit e % 32 of word e / 32; zero before build_list
  int32_t idx[kMaxTokens * 16];           // routing of the step
  float w[kMaxTokens * 16];
  float weight[kMaxTokens * 17];          // router weight of each row of h
};

// Routing of all tokens and the list without `base` and `weight`, by all warps
// but kXWarp, which waits for x meanwhile (it joins with wait_list): one warp
// per token, the high warps first, as the low ones have other work at that
// point.  The router weights are needed last, so they are computed after the
// list is there.  `emit`: this block also writes the routing outputs and
// records errors.
constexpr int kXWarp = 3, kListThreads = kThreads - 32;
constexpr int kBarList = 3, kBarListX = 4;          // named barriers
__device__ __forceinline__ void bar_arrive(int id, int nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}
// A warp's place in the deal of tokens: warp 15 is 0, kXWarp has none.
__device__ __forceinline__ int route_turn() {
  const int wid = threadIdx.x >> 5;
  return wid > kXWarp ? kWarps - 1 - wid : kWarps - 2 - wid;
}
__device__ __forceinline__ void build_list(List& L, const Args& a, const Routing& r, bool emit) {
  const int lane = threadIdx.x & 31, turn = route_turn();
  // at most two tokens a warp (kMaxTokens = kListThreads / 32 + 1)
  int e0 = -1, e1 = -1;
  float z0 = 0.f, z1 = 0.f;
#pragma unroll 1
  for (int t = turn; t < a.T; t += kWarps - 1) {
    int e;
    float z;
    route_experts(a, r, t, e, z);
    if (lane < a.k) {
      L.idx[t * a.k + lane] = e;
      if (e >= 0) atomicOr(&L.chosen[e >> 5], 1u << (e & 31));
    }
    if (t == turn) {
      e0 = e;
      z0 = z;
    } else {
      e1 = e;
      z1 = z;
    }
  }
  named_bar_sync(kBarList, kListThreads);
  const int sh = a.has_shared, P = a.T * a.k;
  if (turn * 32 < P) {
    // entry of a word's first expert: a scan over the bitmap in every warp
    const uint32_t word = L.chosen[lane];
    int x = __popc(word);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    const int p = turn * 32 + lane;
    const int e = p < P ? L.idx[p] : -1;
    const int src = e >= 0 ? e >> 5 : 0;
    const uint32_t ew = __shfl_sync(0xFFFFFFFFu, word, src);
    const int first = __shfl_sync(0xFFFFFFFFu, x, src) - __popc(ew);
    if (e >= 0) {
      const int d = sh + first + __popc(ew & ((1u << (e & 31)) - 1u));
      L.expert[d] = e;                    // the same value from every token that chose e
      atomicOr(&L.mask[d], 1u << (p / a.k));
    }
    if (turn == 0 && lane == 31) L.n = sh + x;
    if (turn == 0 && lane == 0 && sh) {
      L.expert[0] = a.E;
      L.mask[0] = (1u << a.T) - 1u;
    }
  }
  named_bar_sync(kBarList, kListThreads);
#pragma unroll 1
  for (int t = turn; t < a.T; t += kWarps - 1) {
    const int e = t == turn ? e0 : e1;
    const float w = route_weight(a, r, e, t == turn ? z0 : z1);
    if (lane < a.k) {
      L.w[t * a.k + lane] = w;
      if (emit) {
        a.idx[t * a.k + lane] = e;
        a.w[t * a.k + lane] = w;
        if (e < 0) record_error(MOE_ERR_INVALID);
      }
    }
    __syncwarp();
  }
  bar_arrive(kBarListX, kThreads);
}
__device__ __forceinline__ void wait_list() { named_bar_sync(kBarListX, kThreads); }
static_assert(kListThreads >= kMaxTokens * 16 && kMaxTokens <= 2 * (kListThreads / 32), "a thread per pair, two tokens a warp");

// base, by one warp.
__device__ __forceinline__ void list_rows(List& L) {
  const int lane = threadIdx.x & 31;
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
  __syncwarp();
}

// Router weights of the rows, by one warp (after base): an entry's tokens add
// up the slots that name its expert, the shared expert weighs 1.
__device__ __forceinline__ void list_weights(List& L, const Args& a) {
  for (int d = threadIdx.x & 31; d < L.n; d += 32) {
    const int e = L.expert[d];
    int row = L.base[d];
    for (uint32_t m = L.mask[d]; m; m &= m - 1u, ++row) {
      const int t = __ffs(m) - 1;
      float w = e == a.E ? 1.0f : 0.0f;
      if (e != a.E)
        for (int j = 0; j < a.k; ++j)
          if (L.idx[t * a.k + j] == e) w += L.w[t * a.k + j];
      L.weight[row] = w;
    }
  }
  __syncwarp();                           // lanes part over the loops; the next barrier takes whole warps
}

__device__ __forceinline__ void clear_list(List& L) {
  if (threadIdx.x < 32) L.chosen[threadIdx.x] = 0u;
  for (int i = threadIdx.x; i < kMaxList; i += kThreads) L.mask[i] = 0u;
}

// Scale blocks in tensor-memory order have 32 rows of 16 bytes; tokens take 16
// rows at most, so blocks are stored (and copied) as 256 bytes.
constexpr int kSfBlock = 256;

// ------------------------------ x (a1) --------------------------------------
// Block t quantises row t, a half-warp per 128 columns; block 0 also clears
// the counters.
__global__ void __launch_bounds__(256) quant_rows_kernel(const Args a, int n_counters) {
  pdl_wait();
  pdl_trigger();                          // only now: few_layer_kernel reads inputs and writes idx, w before its own wait
  const int t = blockIdx.x, KT = a.H / 128, lane = threadIdx.x & 31, hl = lane & 15;
  if (t == 0)
    for (int i = threadIdx.x; i < n_counters; i += 256) a.done[i] = 0;
  for (int k0 = 2 * (threadIdx.x >> 5); k0 < KT; k0 += 16) {
    const int kt = k0 + (lane >> 4);
    const bool in = kt < KT;
    const uint4 v = in ? __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H + kt * 128) + hl)
                       : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t wv[4] = {v.x, v.y, v.z, v.w};
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
      reinterpret_cast<uint2*>(a.xq + (int64_t)t * a.H + kt * 128)[hl] =
          make_uint2(e4m3x4(__fmul_rn(f[0], sc), __fmul_rn(f[1], sc), __fmul_rn(f[2], sc), __fmul_rn(f[3], sc)),
                     e4m3x4(__fmul_rn(f[4], sc), __fmul_rn(f[5], sc), __fmul_rn(f[6], sc), __fmul_rn(f[7], sc)));
      if (hl == 0) a.x_sf[(kt >> 2) * kSfBlock + t * 16 + (kt & 3)] = (uint8_t)(k + 127);
    }
  }
}

// ------------------------------ main kernel ---------------------------------
// Ring slot: two unpacked weight tiles (gate and up of a feature block, or two
// row blocks of w2), their scale blocks, and in the second phase a K step of h
// with its scales.  The rows of x stay in shared memory for the first phase;
// the block's part of y takes their place in the second.  With at most 8
// tokens a K step of x has 8 rows only: the MMA's columns 8..15 are then the
// next step's rows (h: what the slot held before), which nothing reads.
constexpr int kTileBytes = 32768, kSlotSf = 1024 + 512, kSlotH = 2048;
constexpr int kMaxStages = 5;
constexpr int kMaxGrid = 160;             // blocks at most (the parts of y are sized for it)
constexpr int kTmemCols = 256;
constexpr int kAhead = 4;                 // steps the L2 prefetcher runs ahead of the copies

struct Sync {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], x_full, x_scales, up_done;
  uint32_t tmem;
  int abort_flag;
  int produced;                           // steps whose weight copies are issued
  int last[2];                            // row pair + 1 whose parts this block sums, for its first and second piece
};

struct Smem {
  // tiles | h | x or y | scale blocks | x scale blocks | Sync | red | List
  __host__ __device__ static int rows(int T) { return T <= 8 ? 8 : 16; }
  __host__ __device__ static int h_off(int stages) { return stages * kTileBytes; }
  __host__ __device__ static int x_off(int stages) { return h_off(stages) + stages * kSlotH; }
  __host__ __device__ static int x_bytes(int T, int KT) {
    const int x = (KT + 3) / 4 * 4 * rows(T) * 128 + 1024, y = (T * 1024 + 1023) / 1024 * 1024;
    return x > y ? x : y;
  }
  __host__ __device__ static int sf_off(int stages, int T, int KT) { return x_off(stages) + x_bytes(T, KT); }
  __host__ __device__ static int xsf_off(int stages, int T, int KT) { return sf_off(stages, T, KT) + stages * kSlotSf; }
  __host__ __device__ static int sync_off(int stages, int T, int KT) {
    return xsf_off(stages, T, KT) + (KT + 3) / 4 * kSfBlock + kSfBlock;
  }
  __host__ __device__ static int red_off(int stages, int T, int KT) {
    return sync_off(stages, T, KT) + (int)(sizeof(Sync) + 15) / 16 * 16;
  }
  __host__ __device__ static int list_off(int stages, int T, int KT) { return red_off(stages, T, KT) + 2 * 16 * 4; }
  __host__ __device__ static int total(int stages, int T, int KT) {
    return list_off(stages, T, KT) + (int)sizeof(List) + 1024;
  }
};

// Ring position.
struct Slot {
  uint32_t i = 0, phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++i == (uint32_t)stages) {
      i = 0;
      phase ^= 1u;
    }
  }
};

// After a wait has given up: the weight producer waits (bounded) for the copies
// of its last `n` steps before the block ends.
__device__ __forceinline__ void drain_ring(Sync& s, int stages, int n, Slot at) {
  const uint64_t t0 = globaltimer_ns();
  for (int k = 0; k < n; ++k) {
    if (at.i == 0) {
      at.i = stages;
      at.phase ^= 1u;
    }
    --at.i;
    while (!mbar_try_wait(smem_u32(&s.full[at.i]), at.phase) && globaltimer_ns() - t0 < kWaitTimeoutNs) {
    }
  }
}

// The second phase's steps in order: (row pair, entry, K step).  Block c of
// `blocks` takes [first(c), first(c + 1)): at most two row pairs, as there are
// at least as many blocks as row pairs (the launch refuses devices where there
// are not).
struct Down {
  int z, z1, rp, d, kt;
  // (Z <= 32 * 257 * 64 steps and 160 blocks: products stay below 2^31)
  __device__ static int first(int Z, int c, int blocks) { return Z * c / blocks; }
  // the block whose range holds z
  __device__ static int owner(int Z, int z, int blocks) { return ((z + 1) * blocks - 1) / Z; }
  __device__ __forceinline__ Down(int Z, int c, int blocks, int n, int KT) {
    z = c < blocks ? first(Z, c, blocks) : Z;
    z1 = c < blocks ? first(Z, c + 1, blocks) : Z;
    const int total = n * KT;
    rp = total > 0 ? z / total : 0;
    const int s = z - rp * total;
    d = s / KT;
    kt = s - d * KT;
  }
  __device__ __forceinline__ bool more() const { return z < z1; }
  __device__ __forceinline__ void next(int n, int KT) {
    ++z;
    if (++kt == KT) {
      kt = 0;
      if (++d == n) {
        d = 0;
        ++rp;
      }
    }
  }
};

__device__ __forceinline__ int ld_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
// Global memory written through the generic proxy and read by TMA (or the
// other way round), on both sides of the hand-over.
__device__ __forceinline__ void fence_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// One 32-bit column per lane of the warp's sub-partition.
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t& r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld1(uint32_t& r0, uint32_t& r1) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r0), "+r"(r1)::"memory");
}

struct Maps {
  CUtensorMap w13, w13_sf, w2, w2_sf, x, h;
};

__global__ void __launch_bounds__(kThreads, 1)
    few_layer_kernel(const __grid_constant__ Maps m, const Args a, const Routing r, int stages) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (-sm100::smem_u32(smem_raw) & 1023u);      // by an offset: shared addresses stay 32-bit
  const int KT = a.H / 128, KG = (KT + 3) / 4, FB = a.I / 128, KG2 = (FB + 3) / 4, sh = a.has_shared;
  const int RB = a.H / 128, RP = (RB + 1) / 2, xtile = Smem::rows(a.T) * 128;
  uint8_t* hts = smem + Smem::h_off(stages);
  uint8_t* xt = smem + Smem::x_off(stages);
  float* ys = reinterpret_cast<float*>(xt);               // [T][256], second phase
  uint8_t* sfs = smem + Smem::sf_off(stages, a.T, KT);
  uint8_t* xsf = smem + Smem::xsf_off(stages, a.T, KT);
  Sync& sy = *reinterpret_cast<Sync*>(smem + Smem::sync_off(stages, a.T, KT));
  float* red = reinterpret_cast<float*>(smem + Smem::red_off(stages, a.T, KT));     // maxima [2][4 tokens][4 warps]
  List& L = *reinterpret_cast<List*>(smem + Smem::list_off(stages, a.T, KT));
  volatile int* abort_flag = &sy.abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const int c = blockIdx.x, G = gridDim.x;

  pdl_trigger();
  // the logits first, before weights fill the memory queues
  if (warp != kXWarp && !r.tid2eid)
    for (int t = route_turn(); t < a.T; t += kWarps - 1)
      warp_prefetch(reinterpret_cast<const uint8_t*>(a.logits + (int64_t)t * a.E), a.E * 4);
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(&sy.full[i], 2);          // the two producers
      mbar_init(&sy.empty[i], 2);         // the two issuers
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sy.acc_full[b], 2);
      mbar_init(&sy.acc_empty[b], 128);
    }
    mbar_init(&sy.x_full, 1);
    mbar_init(&sy.x_scales, 1);
    mbar_init(&sy.up_done, 2);
    sy.abort_flag = 0;
    sy.produced = 0;
    sy.last[0] = sy.last[1] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sy.tmem, kTmemCols);
    tmem_relinquish();
  }
  clear_list(L);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sy.tmem;

  // Everything up to pdl_wait touches only the call's inputs (logits, token ids,
  // weights) and idx and w: quant_rows_kernel lets this kernel start after its
  // own wait, when all earlier work on the stream is complete.
  // ---- weights that need no routing: the shared expert's ----
  Slot slot;                              // of the weight producer
  int pre = 0, issued = 0;
  auto load_up = [&](int p) {             // p: pair of blocks of w13
    uint64_t* bar = &sy.full[slot.i];
    mbar_arrive_expect_tx(bar, 2 * kWBlock);
    mbar_arrive(bar);                     // no second operand in this phase
    tma_load_4d(smem + slot.i * kTileBytes, &m.w13, 0, 0, 0, p, bar);
    tma_load_3d(sfs + slot.i * kSlotSf, &m.w13_sf, 0, 0, p, bar);
    sy.produced = sy.produced + 1;
  };
  if (warp == 0 && sh && c < FB) {
    for (; pre < min(stages, KT); ++pre) {
      if (elect_one()) load_up((a.E * FB + c) * KT + pre);
      __syncwarp();
      slot.next(stages);
    }
  }
  if (warp == 8 && sh) {
    // this block's slice of the shared expert into L2
    const int n13 = FB * KT, n2 = RB * FB, n = n13 + n2;
    for (int i = c * n / G; i < (c + 1) * n / G; ++i) {
      if (i < n13) warp_prefetch(a.w13 + ((int64_t)a.E * n13 + i) * 2 * kWBlock, 2 * kWBlock);
      else warp_prefetch(a.w2 + ((int64_t)a.E * n2 + i - n13) * kWBlock, kWBlock);
    }
  }
  __syncwarp();
  if (warp == kXWarp) {
    // ---- x, four K steps a copy (with steps past the row as zeros) ----
    pdl_wait();                           // x is quantised, the counters are clear
    if (elect_one()) {
      mbar_arrive_expect_tx(&sy.x_full, KG * (4 * xtile + kSfBlock));
      bulk_load(xsf, a.x_sf, KG * kSfBlock, &sy.x_full);
      for (int g = 0; g < KG; ++g) tma_load_3d(xt + g * 4 * xtile, &m.x, 0, 0, 4 * g, &sy.x_full);
    }
    __syncwarp();
    wait_list();
  } else {
    build_list(L, a, r, c == 0);
  }

  const int n = L.n, n_items = n * FB, Z = RP * n * FB;
  const int blocks2 = min(G, Z);          // blocks of the second phase
  // tensor-memory columns: accumulators 2 x (tile 0: 16, tile 1: 16), weight
  // scales 4 per issuer, h scales 4 per issuer, x scales KT
  constexpr int kAcc = 0, kSfa = 64, kSfh = 72, kSfx = 80;
  static_assert(kSfx + kMaxWidth / 128 <= kTmemCols, "tensor memory overflow");
  if (warp == 0) {
    // ------------------------- producer of weights -------------------------
    issued = pre;
    bool ok = true;
    for (int item = c; item < n_items && ok; item += G) {
      const int d = item / FB, p = (L.expert[d] * FB + item - d * FB) * KT;
      for (int kt = item == c ? pre : 0; kt < KT; ++kt) {
        if (!mbar_wait_warp(&sy.empty[slot.i], slot.phase ^ 1u, abort_flag)) { ok = false; break; }
        if (elect_one()) load_up(p + kt);
        __syncwarp();
        ++issued;
        slot.next(stages);
      }
    }
    for (Down w(Z, c, blocks2, n, FB); w.more() && ok; w.next(n, FB)) {
      if (!mbar_wait_warp(&sy.empty[slot.i], slot.phase ^ 1u, abort_flag)) { ok = false; break; }
      const int blk = L.expert[w.d] * RB + 2 * w.rp;
      if (elect_one()) {
        uint64_t* bar = &sy.full[slot.i];
        mbar_arrive_expect_tx(bar, 2 * kWBlock);
        tma_load_4d(smem + slot.i * kTileBytes, &m.w2, 0, 0, w.kt, blk, bar);
        tma_load_3d(sfs + slot.i * kSlotSf, &m.w2_sf, 0, w.kt, blk, bar);
        sy.produced = sy.produced + 1;
      }
      __syncwarp();
      ++issued;
      slot.next(stages);
    }
  } else if (warp == kXWarp) {
    // ---------------------------- producer of h ----------------------------
    list_rows(L);
    list_weights(L, a);
    named_bar_sync(2, 160);               // the epilogue warps read both
    // Slots pass to the second phase once the first phase's products are done.
    // From there on no slot is used again before this warp has filled it, so
    // the parity of `empty` cannot run ahead of it.
    const int steps = c < n_items ? ((n_items - 1 - c) / G + 1) * KT : 0;      // of the first phase
    const bool follow = mbar_wait_warp(&sy.up_done, 0, abort_flag);
    Slot hs;
    hs.i = steps % stages;
    hs.phase = (steps / stages) & 1;
    int filled = 0;
    int ready = -1;                       // entry whose h is known to be complete
    bool first = true;
    for (Down w(Z, c, blocks2, n, FB); w.more() && follow; w.next(n, FB)) {
      bool ok = filled++ < stages || mbar_wait_warp(&sy.empty[hs.i], hs.phase ^ 1u, abort_flag);
      if (ok && w.d != ready) {
        const uint64_t t0 = globaltimer_ns();
        while (ld_acquire(a.done + w.d) < FB) {
          if (*abort_flag) { ok = false; break; }
          if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
            record_error(MOE_ERR_TIMEOUT);
            *abort_flag = 1;
            ok = false;
            break;
          }
        }
        ok = __all_sync(0xFFFFFFFFu, ok);
        fence_async_global();
        ready = w.d;
      }
      if (!ok) break;
      // scales of four K steps a block: at a group's first step
      const bool sf = first || (w.kt & 3) == 0;
      if (elect_one()) {
        uint64_t* bar = &sy.full[hs.i];
        mbar_arrive_expect_tx(bar, xtile + (sf ? kSfBlock : 0));
        tma_load_2d(hts + hs.i * kSlotH, &m.h, w.kt * 128, L.base[w.d], bar);
        if (sf) bulk_load(sfs + hs.i * kSlotSf + 1024, a.h_sf + ((size_t)w.d * KG2 + (w.kt >> 2)) * kSfBlock, kSfBlock, bar);
      }
      __syncwarp();
      first = false;
      hs.next(stages);
    }
  } else if (warp == 8) {
    // ---------------------------- L2 prefetcher ----------------------------
    // kAhead steps ahead of the copies, through both phases.  A hint only: it
    // gives up quietly when the block aborts or after the wait bound.
    const uint64_t t0 = globaltimer_ns();
    int at = 0;
    auto wait_turn = [&]() {              // false: stop
      while (*reinterpret_cast<volatile int*>(&sy.produced) + kAhead <= at) {
        if (*abort_flag || globaltimer_ns() - t0 > kWaitTimeoutNs) return false;
        __nanosleep(64);
      }
      ++at;
      return true;
    };
    bool go = true;
    for (int item = c; item < n_items && go; item += G) {
      const int d = item / FB;
      const uint8_t* src = a.w13 + (int64_t)(L.expert[d] * FB + item - d * FB) * KT * 2 * kWBlock;
      for (int kt = 0; kt < KT; ++kt) {
        go = __all_sync(0xFFFFFFFFu, wait_turn());
        if (!go) break;
        if (d >= sh && at > stages) warp_prefetch(src + (int64_t)kt * 2 * kWBlock, 2 * kWBlock);
      }
    }
    for (Down w(Z, c, blocks2, n, FB); w.more() && go; w.next(n, FB)) {
      go = __all_sync(0xFFFFFFFFu, wait_turn());
      if (!go) break;
      if (w.d < sh) continue;             // already asked for
      const uint8_t* src = a.w2 + (((int64_t)L.expert[w.d] * RB + 2 * w.rp) * FB + w.kt) * kWBlock;
      warp_prefetch(src, kWBlock);
      if (2 * w.rp + 1 < RB) warp_prefetch(src + (int64_t)FB * kWBlock, kWBlock);
    }
  } else if (warp == 1 || warp == 2) {
    // --------------------- MMA issuers: one tile each ---------------------
    const int iss = warp - 1;
    const uint32_t idesc = idesc_mxf8f6f4(5u /*E2M1*/, 0u /*E4M3*/, 128, 16);
    const uint32_t sfa = tmem + kSfa + 4 * iss, sfh = tmem + kSfh + 4 * iss, sfx = tmem + kSfx;
    uint32_t ab = 0, acc_bits = 0;
    Slot in;
    bool ok = true;
    auto step = [&](uint64_t db, uint32_t sfb, uint32_t dcol, uint32_t accumulate) {   // one elected lane
      const uint64_t da = sdesc_kmajor_sw128(smem_u32(smem + in.i * kTileBytes + iss * 16384));
      const uint32_t bsel = sfb >> 30;
      tmem_cp_32x128b_warpx4(sfa, sdesc_sf(smem_u32(sfs + in.i * kSlotSf + iss * 512)));
#pragma unroll
      for (int kb = 0; kb < 4; ++kb)
        mma_mxf8f6f4(dcol, da + 2 * kb, db + 2 * kb, idesc_with_sf_ids(idesc, kb, 0) | (bsel << 4),
                     sfa | ((uint32_t)kb << 30), sfb, kb ? 1u : accumulate);
      tc_commit(&sy.empty[in.i]);
    };
    ok = mbar_wait_warp(&sy.x_full, 0, abort_flag);
    if (c < n_items) {
      if (ok && iss == 0) {
        if (elect_one()) {
          for (int g = 0; g < KG; ++g) tmem_cp_32x128b_warpx4(sfx + 4 * g, sdesc_sf(smem_u32(xsf + g * kSfBlock)));
          tc_commit(&sy.x_scales);
        }
        __syncwarp();
      }
      ok = ok && mbar_wait_warp(&sy.x_scales, 0, abort_flag);
      tc_fence_after();
    }
    for (int item = c; item < n_items && ok; item += G) {
      if (!mbar_wait_warp(&sy.acc_empty[ab], ((acc_bits >> ab) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
      tc_fence_after();
      const uint32_t dcol = tmem + kAcc + ab * 32 + iss * 16;
      for (int kt = 0; kt < KT; ++kt) {
        if (!mbar_wait_warp(&sy.full[in.i], in.phase, abort_flag)) { ok = false; break; }
        const uint64_t db = sdesc_kmajor_sw128(smem_u32(xt + kt * xtile));
        if (elect_one()) step(db, (sfx + (kt >> 2) * 4) | ((uint32_t)(kt & 3) << 30), dcol, kt ? 1u : 0u);
        __syncwarp();
        in.next(stages);
      }
      if (!ok) break;
      if (elect_one()) tc_commit(&sy.acc_full[ab]);
      __syncwarp();
      acc_bits ^= 1u << ab;
      ab ^= 1u;
    }
    if (elect_one()) tc_commit(&sy.up_done);
    __syncwarp();
    bool fresh = true;                    // the next step starts a segment
    bool first = true;
    for (Down w(Z, c, blocks2, n, FB); w.more() && ok;) {
      if (fresh) {
        if (!mbar_wait_warp(&sy.acc_empty[ab], ((acc_bits >> ab) & 1u) ^ 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
      }
      if (!mbar_wait_warp(&sy.full[in.i], in.phase, abort_flag)) { ok = false; break; }
      const uint32_t dcol = tmem + kAcc + ab * 32 + iss * 16;
      const uint64_t db = sdesc_kmajor_sw128(smem_u32(hts + in.i * kSlotH));
      if (elect_one()) {
        if (first || (w.kt & 3) == 0) tmem_cp_32x128b_warpx4(sfh, sdesc_sf(smem_u32(sfs + in.i * kSlotSf + 1024)));
        step(db, sfh | ((uint32_t)(w.kt & 3) << 30), dcol, fresh ? 0u : 1u);
      }
      __syncwarp();
      in.next(stages);
      first = false;
      const int d = w.d, rp = w.rp;
      w.next(n, FB);
      fresh = !w.more() || w.d != d || w.rp != rp;
      if (fresh) {
        if (elect_one()) tc_commit(&sy.acc_full[ab]);
        __syncwarp();
        acc_bits ^= 1u << ab;
        ab ^= 1u;
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------ epilogue ------------------------------
    const int q = warp & 3, f = q * 32 + lane;
    const uint32_t lane_addr = tmem + kAcc + ((uint32_t)(q * 32) << 16);
    uint32_t ab = 0, acc_bits = 0;
    bool ok = true;
    // Waits for the next accumulators; the four warps go on or stop together.
    auto take = [&]() {
      ok = named_bar_and(1, 128, mbar_wait(&sy.acc_full[ab], (acc_bits >> ab) & 1u, abort_flag));
      if (ok) tc_fence_after();
    };
    // One column of both tiles.  Columns are read one by one, in rolled loops:
    // most experts have one or two of the 16 tokens, and unrolled over all
    // columns this code was 4 us of instruction misses a pass.
    auto column = [&](int t, float& v0, float& v1) {
      uint32_t r0, r1;
      tmem_ld1(lane_addr + ab * 32 + t, r0);
      tmem_ld1(lane_addr + ab * 32 + 16 + t, r1);
      tmem_wait_ld1(r0, r1);
      v0 = __uint_as_float(r0);
      v1 = __uint_as_float(r1);
    };
    auto release = [&]() {
      tc_fence_before();
      mbar_arrive(&sy.acc_empty[ab]);
      acc_bits ^= 1u << ab;
      ab ^= 1u;
    };
    named_bar_sync(2, 160);               // L.base (warp 3)
    pdl_wait();                           // the counters are clear
    ok = named_bar_and(1, 128, mbar_wait(&sy.x_full, 0, abort_flag));        // y takes x's place later
    // first phase: SwiGLU and the a1 rule per token
    int rb = 0;                           // two sets of maxima in turn
    for (int item = c; item < n_items && ok; item += G) {
      const int d = item / FB, pb = item - d * FB;
      take();
      if (!ok) break;
      uint8_t* hq = a.hq + (size_t)L.base[d] * a.I + pb * 128 + f;
      uint8_t* sf = a.h_sf + ((size_t)d * KG2 + (pb >> 2)) * kSfBlock + (pb & 3);
#pragma unroll 1
      for (uint32_t mask = L.mask[d]; mask;) {
        // up to four tokens a round: their maxima cross the warps together
        float h[4];
        int cnt = 0;
        float* rd = red + rb * 16;
        rb ^= 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (mask) {
            float gate, up;
            column(__ffs(mask) - 1, gate, up);
            mask &= mask - 1u;
            h[j] = swiglu_clamped(gate, up, a.limit);
            const float mx = warp_max_nonneg(fabsf(h[j]));
            if (lane == 0) rd[j * 4 + q] = mx;
            cnt = j + 1;
          }
        }
        named_bar_sync(1, 128);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j < cnt) {
            const float4 w4 = *reinterpret_cast<const float4*>(rd + j * 4);
            const int k = pow2_scale_exponent(fmaxf(fmaxf(w4.x, w4.y), fmaxf(w4.z, w4.w)));
            *hq = (uint8_t)(e4m3x2(__fmul_rn(h[j], exp2_int(-k)), 0.0f) & 0xFFu);
            if (f == 0) *sf = (uint8_t)(k + 127);
            hq += a.I;
            sf += 16;
          }
        }
      }
      release();
      fence_async_global();               // read by TMA
      named_bar_sync(1, 128);
      if (f == 0) {
        __threadfence();                  // after the barrier: covers the four warps' writes
        atomicAdd(a.done + d, 1);
      }
    }
    // second phase: router weights, the block's parts of y
    int piece = 0;
    Down w(Z, c, blocks2, n, FB);
    bool fresh = true;
    while (ok && w.more()) {
      const int d = w.d, rp = w.rp;
      const int left = min(FB - w.kt, w.z1 - w.z);     // steps of the segment
      take();
      if (!ok) break;
      if (fresh) {
#pragma unroll 1
        for (int t = 0; t < a.T; ++t) ys[t * 256 + f] = ys[t * 256 + 128 + f] = 0.f;
      }
      int col = 0;
#pragma unroll 1
      for (uint32_t mask = L.mask[d]; mask; mask &= mask - 1u, ++col) {
        const int t = __ffs(mask) - 1;
        const float wt = L.weight[L.base[d] + col];
        float v0, v1;
        column(col, v0, v1);
        float* y = ys + t * 256 + f;
        y[0] = fmaf(wt, v0, y[0]);
        y[128] = fmaf(wt, v1, y[128]);
      }
      release();
      w.z += left - 1;                    // to the segment's last step, then past it
      w.kt += left - 1;
      w.next(n, FB);
      fresh = !w.more() || w.rp != rp;
      if (fresh) {
        // the piece of this row pair is complete
        float* part = a.part + (size_t)(c * 2 + piece) * a.T * 256;
#pragma unroll 1
        for (int t = 0; t < a.T; ++t) {
          __stcg(part + t * 256 + f, ys[t * 256 + f]);
          __stcg(part + t * 256 + 128 + f, ys[t * 256 + 128 + f]);
        }
        named_bar_sync(1, 128);
        if (f == 0) {
          const int total = n * FB, lo = Down::owner(Z, rp * total, blocks2);
          const int hi = Down::owner(Z, (rp + 1) * total - 1, blocks2);
          __threadfence();
          if (atomicAdd(a.done + n + rp, 1) == hi - lo) {
            __threadfence();
            sy.last[piece] = rp + 1;
          }
        }
        ++piece;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && sy.abort_flag) drain_ring(sy, stages, min(issued, stages), slot);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  // ---- y of the row pairs whose last part this block added: the parts in block order ----
#pragma unroll 1
  for (int piece = 0; piece < 2; ++piece) {
    if (sy.last[piece] == 0) continue;
    const int rp = sy.last[piece] - 1, total = n * FB, cols = min(256, a.H - rp * 256);
    const int lo = Down::owner(Z, rp * total, blocks2), hi = Down::owner(Z, (rp + 1) * total - 1, blocks2);
    // only the first block can have started in an earlier row pair: this one is its second piece then
    const int skip = Down::first(Z, lo, blocks2) < rp * total ? 1 : 0;
    const int64_t stride = (int64_t)a.T * 256;
    for (int i = tid; i < a.T * 64; i += kThreads) {
      const int t = i >> 6, c4 = (i & 63) * 4;
      if (c4 >= cols) continue;
      const float* src = a.part + ((int64_t)lo * 2 * a.T + t) * 256 + c4;
      float4 v = __ldcg(reinterpret_cast<const float4*>(src + skip * stride));
#pragma unroll 4
      for (int b = 1; b <= hi - lo; ++b) {
        const float4 p = __ldcg(reinterpret_cast<const float4*>(src + b * 2 * stride));
        v.x += p.x;
        v.y += p.y;
        v.z += p.z;
        v.w += p.w;
      }
      const __nv_bfloat162 y0 = __floats2bfloat162_rn(v.x, v.y), y1 = __floats2bfloat162_rn(v.z, v.w);
      *reinterpret_cast<uint2*>(a.y + (int64_t)t * a.H + rp * 256 + c4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    }
  }
  if (Z == 0)                             // no expert at all: every slot was rejected
    for (int i = c * kThreads + tid; i < a.T * a.H / 4; i += G * kThreads)
      reinterpret_cast<uint2*>(a.y)[i] = make_uint2(0u, 0u);
}

}  // namespace few
}  // namespace moe

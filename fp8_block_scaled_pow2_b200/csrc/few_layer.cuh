// The whole MoE layer for a few tokens (T <= 16) with MXFP4 experts, in two
// kernels.
//
// A step for a few tokens is a stream of weights: one token of the 256-expert
// layer reads 7 experts (94 MB, 14.3 us at the copy rate) and multiplies each
// weight once.  The grouped path (quantise, route, group, two plans and GEMMs,
// combine) spends 53 us on it, most of it in launches and hand-overs.  Here
//   gate_up_kernel   every block routes all tokens and quantises x for itself
//                    (cheaper than waiting for another kernel to do it), then
//                    computes its share of all chosen experts' gate and up
//                    rows and writes h = SwiGLU in float32;
//   down_kernel      every block quantises h for itself and computes its own
//                    output rows over all experts, router weights applied to
//                    the sums, so y needs no second pass and no atomics.
// down_kernel repeats the routing and starts loading w2 before gate_up_kernel
// has ended (programmatic launch), which hides the hand-over.
//
// Shares are cut in subunits: rows {i, i + 32, i + 64, i + 96} of a 128-row
// weight block, whose scales are one 16-byte word of the prepared block.  With
// whole 128-row blocks, one token's 112 gate / up blocks would keep 112 of 148
// SMs busy; in subunits the largest share is within 3 % of the mean.  Inside
// a block the warps split K, so that a share of any size uses all of them.
#pragma once

#include "common.cuh"
#include "elementwise.cuh"
#include "mma_few.cuh"

namespace moe {
namespace few {

constexpr int kMaxTokens = 16;
constexpr int kMaxWidth = 8192;         // H and I: one row in a block's shared memory
constexpr int kWBlock = 8192 + 512;     // prepared weight block (moe_prepare_weights)
constexpr int kWarps = 8;
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

// Routing of all tokens and the list, by the whole block.  `emit`: this block
// also writes the routing outputs and records errors.
__device__ __forceinline__ void build_list(List& L, const Args& a, const Routing& r, bool emit) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, tid = threadIdx.x;
  if (tid < 32) L.chosen[tid] = 0u;
  __syncthreads();
  for (int t = wid; t < a.T; t += kWarps) {
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
  for (int p = tid; p < a.T * a.k; p += kThreads) {
    const int e = L.idx[p];
    if (e >= 0)
      atomicOr(&L.mask[L.word_at[e >> 5] + __popc(L.chosen[e >> 5] & ((1u << (e & 31)) - 1u))], 1u << (p / a.k));
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

// 128 columns by a half-warp, 8 per lane (the a1 rule): returns the exponent
// k, writes the lane's 8 E4M3 bytes in the token operand's order.
__device__ __forceinline__ int quant8(const float (&f)[8], uint8_t* dst) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(f[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const int k = pow2_scale_exponent(m);
  const float sc = exp2_int(-k);
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(f[i], sc);
  if (dst) *reinterpret_cast<uint2*>(dst) = fewmma::pack_evens_odds(v);
  return k;
}

// --------------------------- gate / up kernel -------------------------------
// Work of a warp: steps of one K step (128 columns) times an item of up to 8
// subunits (8 x 4 gate rows and as many up rows: 4 tiles of 8 gate + 8 up
// rows).  Each warp has a ring of its own, filled by its own lanes
// (cp.async): no block-wide hand-over between copies and products.
constexpr int kUpTiles = 4;
constexpr int kUpSub = 2 * kUpTiles;
constexpr int kUpStage = kUpTiles * 1024 + 2 * kUpSub * 16;
constexpr int kUpRed = kWarps * 2 * kUpTiles * 16;      // floats of one reduction buffer

struct UpSmem {
  static constexpr int kRed = 2 * kUpRed * 4;
  __host__ __device__ static constexpr int ring(int stages) { return kWarps * stages * kUpStage; }
  __host__ __device__ static int x_stride(int H) { return H + 16; }     // 16 bytes apart: token rows on other banks
  __host__ __device__ static size_t total(int stages, int T, int H) {
    return (size_t)ring(stages) + kRed + (sizeof(List) + 15) / 16 * 16 + (size_t)T * x_stride(H) + (size_t)T * (H / 128) * 4;
  }
};

// The block's subunits: [pos, end) of the shared expert, then [b, b_end) of
// the routed entries (a.I / 4 subunits each).
struct Cursor {
  int pos, end, b, b_end, shared;
};
struct Item {
  int d, su, n;                           // list entry, first subunit within the expert, subunits
};
__device__ __forceinline__ bool next_item(Cursor& c, Item& it, int per_expert, int sh) {
  if (c.pos >= c.end) {
    if (!c.shared) return false;
    c.shared = 0;
    c.pos = c.b;
    c.end = c.b_end;
    if (c.pos >= c.end) return false;
  }
  const int d = c.shared ? 0 : c.pos / per_expert;
  it.su = c.pos - d * per_expert;
  it.d = c.shared ? 0 : sh + d;
  it.n = min(min(kUpSub, c.end - c.pos), per_expert - it.su);
  c.pos += it.n;
  return true;
}

template <int NTP, int STAGES>
__global__ void __launch_bounds__(kThreads, NTP <= 2 ? 2 : 1) gate_up_kernel(const Args a, const Routing r) {
  using namespace fewmma;
  pdl_wait();
  pdl_trigger();                          // only now: down_kernel reads the inputs before its own wait
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* ring_all = smem;
  float* red = reinterpret_cast<float*>(smem + UpSmem::ring(STAGES));
  List& L = *reinterpret_cast<List*>(smem + UpSmem::ring(STAGES) + UpSmem::kRed);
  uint8_t* xs = smem + UpSmem::ring(STAGES) + UpSmem::kRed + (sizeof(List) + 15) / 16 * 16;
  const int xstride = UpSmem::x_stride(a.H);
  float* sxf = reinterpret_cast<float*>(xs + (size_t)a.T * xstride);      // [kt][T]
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, tid = threadIdx.x;
  const int g = lane >> 2, q = lane & 3;
  const int KT = a.H / 128, per = a.I / 4, FB = a.I / 128, sh = a.has_shared;
  const int G = gridDim.x, c = blockIdx.x;

  // ---- copies ----
  Cursor fc;
  fc.shared = 1;
  fc.pos = sh ? (int)((int64_t)c * per / G) : 0;
  fc.end = sh ? (int)((int64_t)(c + 1) * per / G) : 0;
  fc.b = fc.b_end = 0;
  const uint32_t ring = sm100::smem_u32(ring_all + wid * STAGES * kUpStage);
  const int sub = lane >> 2, chunk = lane & 3;                 // weights: subunit and 16 bytes of a lane
  const int shalf = lane >> 3, ssub = lane & 7;                // scales: half and subunit of lanes 0..15
  const uint8_t *src = nullptr, *ssrc = nullptr;
  Item fi;
  const int own_steps = wid < KT ? (KT - wid + kWarps - 1) / kWarps : 0;     // this warp's steps of an item
  int fkt = KT, fslot = 0;                                     // no item yet: the first fetch takes one
  bool fmore = own_steps > 0, fw = false, fs = false;
  auto fetch = [&]() {
    if (fmore && fkt >= KT) {
      fkt = wid;
      fmore = next_item(fc, fi, per, sh);
      if (fmore) {
        const uint8_t* base = a.w13 + (int64_t)(fi.d < sh ? a.E : L.expert[fi.d]) * FB * KT * 2 * kWBlock;
        int su = fi.su + sub;
        fw = sub < fi.n;
        src = base + (int64_t)(su >> 5) * KT * 2 * kWBlock + (su & 31) * 64 + chunk * 16;
        su = fi.su + ssub;
        fs = lane < 16 && ssub < fi.n;
        ssrc = base + (int64_t)(su >> 5) * KT * 2 * kWBlock + shalf * kWBlock + 8192 + (su & 31) * 16;
      }
    }
    if (fmore) {
      const uint32_t st = ring + fslot * kUpStage;
      const int64_t o = (int64_t)fkt * 2 * kWBlock;
      if (fw) {
        const uint32_t dst = st + (sub >> 1) * 1024 + (sub & 1) * 64 + chunk * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int qr = 0; qr < 4; ++qr)
            cp_async16(dst + (h * 8 + qr * 2) * 64, src + o + h * kWBlock + qr * 2048);
      }
      if (fs) cp_async16(st + kUpTiles * 1024 + shalf * kUpSub * 16 + ssub * 16, ssrc + o);
      fkt += kWarps;
    }
    cp_async_commit();
    fslot = fslot + 1 == STAGES ? 0 : fslot + 1;
  };
  // the shared expert's steps need no routing: start their copies now
  const int pre = min(STAGES, (fc.end - fc.pos + kUpSub - 1) / kUpSub * own_steps);
  Cursor cc = fc;                          // the products' cursor
  for (int s = 0; s < pre; ++s) fetch();

  // ---- routing, x ----
  {
    // half-warps: 128-column groups of all tokens
    const int groups = a.T * KT, hl = lane & 15;
    for (int p0 = wid * 2; p0 < groups; p0 += 2 * kWarps) {
      const int p = p0 + (lane >> 4);
      const bool in = p < groups;
      const int t = in ? p / KT : 0, kt = in ? p % KT : 0;
      const uint4 u = in ? __ldg(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H + kt * 128) + hl)
                         : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      float f[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
      }
      const int k = quant8(f, in ? xs + t * xstride + kt * 128 + hl * 8 : nullptr);
      if (in && hl == 0) sxf[kt * a.T + t] = exp2_int(k) * kE2m1Unit;
    }
  }
  build_list(L, a, r, c == 0);            // ends with a barrier: xs and sxf are complete too
  {
    const int64_t S = (int64_t)(L.n - sh) * per;
    fc.b = cc.b = (int)(c * S / G);
    fc.b_end = cc.b_end = (int)((c + 1) * S / G);
  }
  for (int s = pre; s < STAGES; ++s) fetch();

  // ---- products ----
  Item it;
  int slot = 0, buf = 0;
  const uint8_t* ring_p = ring_all + wid * STAGES * kUpStage;
  while (next_item(cc, it, per, sh)) {
    const uint32_t mask = L.mask[it.d];
    const int cnt = __popc(mask), tiles = (it.n + 1) >> 1;
    float acc[kUpTiles][NTP][2];
#pragma unroll
    for (int i = 0; i < kUpTiles; ++i)
#pragma unroll
      for (int n = 0; n < NTP; ++n) acc[i][n][0] = acc[i][n][1] = 0.f;
    for (int kt = wid; kt < KT; kt += kWarps) {
      cp_async_wait<STAGES - 1>();
      __syncwarp();
      const uint8_t* st = ring_p + slot * kUpStage;
      const uint8_t* sc = st + kUpTiles * 1024 + (g & 1) * 16 + (g >> 1) * 4 + (q & 1) * 2;
      const uint8_t* xk = xs + kt * 128 + q * 32;
      const float* sk = sxf + kt * a.T;
      // column sets: the expert's tokens two by two
      auto toks = [&](uint32_t& m, int& t0, int& t1) {
        t0 = __ffs(m) - 1;
        m &= m - 1u;
        t1 = __ffs(m) - 1;
        m = m ? m & (m - 1u) : 0u;
      };
      TokB b0;
      float f0;
      {
        uint32_t m = mask;
        int t0, t1;
        toks(m, t0, t1);
        const int tb = g < 4 ? t0 : t1, tc = q < 2 ? t0 : t1;
        load_tok(b0, q == (g & 3) && tb >= 0 ? xk + tb * xstride : nullptr);
        f0 = tc >= 0 ? sk[tc] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kUpTiles; ++i) {
        if (i < tiles) {
          TileA ta;
          load_tile(ta, st + i * 1024 + g * 64 + q * 16, st + i * 1024 + 512 + g * 64 + q * 16);
          const float2 sg = e8m0x2(*reinterpret_cast<const uint16_t*>(sc + i * 32));
          const float2 su = e8m0x2(*reinterpret_cast<const uint16_t*>(sc + kUpSub * 16 + i * 32));
          float cf[4];
          tile_mma(cf, ta, b0);
          acc[i][0][0] = fmaf(cf[0], sg.x * f0, fmaf(cf[1], sg.y * f0, acc[i][0][0]));
          acc[i][0][1] = fmaf(cf[2], su.x * f0, fmaf(cf[3], su.y * f0, acc[i][0][1]));
          if constexpr (NTP > 1) {
            uint32_t m = mask & (mask - 1u);
            m = m ? m & (m - 1u) : 0u;
#pragma unroll
            for (int n = 1; n < NTP; ++n) {
              if (2 * n < cnt) {
                int t0, t1;
                toks(m, t0, t1);
                const int tb = g < 4 ? t0 : t1, tc = q < 2 ? t0 : t1;
                TokB b;
                load_tok(b, q == (g & 3) && tb >= 0 ? xk + tb * xstride : nullptr);
                const float f = tc >= 0 ? sk[tc] : 0.f;
                tile_mma(cf, ta, b);
                acc[i][n][0] = fmaf(cf[0], sg.x * f, fmaf(cf[1], sg.y * f, acc[i][n][0]));
                acc[i][n][1] = fmaf(cf[2], su.x * f, fmaf(cf[3], su.y * f, acc[i][n][1]));
              }
            }
          }
        }
      }
      __syncwarp();
      fetch();
      slot = slot + 1 == STAGES ? 0 : slot + 1;
    }
    // ---- sum over the warps (K), two column sets a round; SwiGLU ----
    uint32_t m = mask;
    int hrow = L.base[it.d];
#pragma unroll
    for (int n = 0; n < NTP; ++n) {
      if (2 * n < cnt) {
        float* rb = red + buf * kUpRed;
        buf ^= 1;
#pragma unroll
        for (int i = 0; i < kUpTiles; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v = acc[i][n][h];
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
            if ((q & 1) == 0) rb[((wid * 2 + (q >> 1)) * kUpTiles + i) * 16 + h * 8 + g] = v;
          }
        }
        __syncthreads();                  // the other buffer's readers are past it, too
        if (tid < 2 * kUpTiles * 8) {
          const int set = tid / (kUpTiles * 8), i = (tid / 8) % kUpTiles, gg = tid % 8;
          const int s = 2 * i + (gg & 1), su = it.su + s;
          if (2 * n + set < cnt && s < it.n) {
            float gate = 0.f, up = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float* p = rb + ((w * 2 + set) * kUpTiles + i) * 16 + gg;
              gate += p[0];
              up += p[8];
            }
            a.h[(int64_t)(hrow + set) * a.I + (su >> 5) * 128 + 32 * (gg >> 1) + (su & 31)] =
                swiglu_clamped(gate, up, a.limit);
          }
        }
        hrow += 2;
      }
    }
  }
  cp_async_wait<0>();
}

// ------------------------------ down kernel ---------------------------------
// A block owns up to 8 subunits of output rows at a time (28 rows at hidden
// 4096) and runs over all (entry, K step) pairs, the pairs dealt to its warps
// in turn.  Columns are the tokens themselves, so the accumulators stay in
// registers over all experts: the factor of a token that did not choose the
// expert is 0.  Rows of h are quantised into shared memory in chunks of
// consecutive rows (whole entries), the next chunk between the products of
// the present one.
constexpr int kDnTiles = 2;
constexpr int kDnSub = 4 * kDnTiles;
constexpr int kDnStage = kDnTiles * 1024 + kDnSub * 16;
constexpr int kDnStages = 4;

struct DownSmem {
  static constexpr int kRing = kWarps * kDnStages * kDnStage;
  static constexpr int kRed = kWarps * 2 * kDnTiles * 16 * 4;
  __host__ __device__ static int h_stride(int I) { return I + 16; }
  __host__ __device__ static size_t chunk(int rows, int I) {             // rows, then their factors [row][K step]
    return ((size_t)rows * (h_stride(I) + (I / 128) * 4) + 15) / 16 * 16;
  }
  __host__ __device__ static size_t total(int rows, int bufs, int I) {
    return (size_t)kRing + kRed + (sizeof(List) + 15) / 16 * 16 + bufs * chunk(rows, I);
  }
};

template <int NTP>
__global__ void __launch_bounds__(kThreads, NTP <= 2 ? 2 : 1) down_kernel(const Args a, const Routing r, int chunk_rows,
                                                                         int bufs) {
  using namespace fewmma;
  pdl_trigger();
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t* ring_all = smem;
  float* red = reinterpret_cast<float*>(smem + DownSmem::kRing);
  List& L = *reinterpret_cast<List*>(smem + DownSmem::kRing + DownSmem::kRed);
  uint8_t* hs_all = smem + DownSmem::kRing + DownSmem::kRed + (sizeof(List) + 15) / 16 * 16;
  const int hstride = DownSmem::h_stride(a.I);
  const size_t chunk_bytes = DownSmem::chunk(chunk_rows, a.I);
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, tid = threadIdx.x;
  const int g = lane >> 2, q = lane & 3;
  const int KT = a.I / 128, RB = a.H / 128;
  const int G = gridDim.x, S = a.H / 4;
  // Routing and weights are inputs of the call, complete before gate_up_kernel
  // let this kernel start (it does so after its own wait): read before the wait.
  build_list(L, a, r, false);
  const int steps = L.n * KT;

  bool waited = false;
  for (int u0 = (int)((int64_t)blockIdx.x * S / G); u0 < (int)((int64_t)(blockIdx.x + 1) * S / G); u0 += kDnSub) {
    const int nsub = min(kDnSub, (int)((int64_t)(blockIdx.x + 1) * S / G) - u0);
    const int tiles = (nsub + 3) >> 2;
    // ---- copies ----
    const uint32_t ring = sm100::smem_u32(ring_all + wid * kDnStages * kDnStage);
    const int sub = lane >> 2, chunk = lane & 3;
    const uint8_t *src, *ssrc;
    {
      int su = u0 + sub;
      src = a.w2 + (int64_t)(su >> 5) * KT * kWBlock + (su & 31) * 64 + chunk * 16;
      su = u0 + (lane & 7);
      ssrc = a.w2 + (int64_t)(su >> 5) * KT * kWBlock + 8192 + (su & 31) * 16;
    }
    const bool fw = sub < nsub, fs = lane < 8 && lane < nsub;
    const uint32_t dst = (sub >> 2) * 1024 + ((sub >> 1) & 1) * 512 + (sub & 1) * 64 + chunk * 16;
    int fstep = wid, fslot = 0, fd = wid / KT, fkt = wid % KT;
    auto fetch = [&]() {
      if (fstep < steps) {
        const uint32_t st = ring + fslot * kDnStage;
        const int64_t o = ((int64_t)L.expert[fd] * RB * KT + fkt) * kWBlock;
        if (fw) {
#pragma unroll
          for (int qr = 0; qr < 4; ++qr) cp_async16(st + dst + qr * 128, src + o + qr * 2048);
        }
        if (fs) cp_async16(st + kDnTiles * 1024 + lane * 16, ssrc + o);
        fstep += kWarps;
        fkt += kWarps;
        while (fkt >= KT) {
          fkt -= KT;
          ++fd;
        }
      }
      cp_async_commit();
      fslot = fslot + 1 == kDnStages ? 0 : fslot + 1;
    };
    for (int s = 0; s < kDnStages; ++s) fetch();
    if (!waited) {
      pdl_wait();                         // h is complete
      waited = true;
    }

    // ---- quantisation of h: task (row, K step) of a chunk by a half-warp ----
    auto chunk_end = [&](int d0) {        // entries [d0, d1) of the chunk that starts at d0
      int d1 = d0 + 1;
      while (d1 < L.n && L.base[d1 + 1] - L.base[d0] <= chunk_rows) ++d1;
      return d1;
    };
    auto row_weight = [&](int d, int row) {   // router weight of row `row` (of all) in entry d
      const int e = L.expert[d];
      if (e == a.E) return 1.0f;
      uint32_t m = L.mask[d];
      for (int i = L.base[d]; i < row; ++i) m &= m - 1u;
      const int t = __ffs(m) - 1;
      float w = 0.f;
      for (int j = 0; j < a.k; ++j)
        if (L.idx[t * a.k + j] == e) w += L.w[t * a.k + j];
      return w;
    };
    auto load8 = [&](int row, int kt, float (&f)[8]) {
      const float4* p = reinterpret_cast<const float4*>(a.h + (int64_t)row * a.I + kt * 128) + 2 * (lane & 15);
      const float4 u = __ldcg(p), v = __ldcg(p + 1);
      f[0] = u.x; f[1] = u.y; f[2] = u.z; f[3] = u.w;
      f[4] = v.x; f[5] = v.y; f[6] = v.z; f[7] = v.w;
    };
    auto quant_task = [&](int task, int n_tasks, int d0, int d1, uint8_t* hs) {
      float f[8];
      const bool in = task < n_tasks;
      const int lr = in ? task / KT : 0, kt = in ? task % KT : 0;
      const int row = L.base[d0] + lr;
      load8(row, kt, f);
      const int k = quant8(f, in ? hs + lr * hstride + kt * 128 + (lane & 15) * 8 : nullptr);
      if (in && (lane & 15) == 0) {
        int d = d0;
        while (L.base[d + 1] <= row) ++d;
        reinterpret_cast<float*>(hs + (size_t)chunk_rows * hstride)[lr * KT + kt] =
            row_weight(d, row) * (exp2_int(k) * kE2m1Unit);
      }
    };

    float acc[kDnTiles][NTP][2];
#pragma unroll
    for (int i = 0; i < kDnTiles; ++i)
#pragma unroll
      for (int n = 0; n < NTP; ++n) acc[i][n][0] = acc[i][n][1] = 0.f;
    int step = wid, slot = 0, buf = 0;
    const uint8_t* ring_p = ring_all + wid * kDnStages * kDnStage;
    int d0 = 0, d1 = L.n > 0 ? chunk_end(0) : 0;
    if (L.n > 0) {
      const int n_tasks = (L.base[d1] - L.base[d0]) * KT;
      for (int task = 2 * wid; task < n_tasks; task += 2 * kWarps)
        quant_task(task + (lane >> 4), n_tasks, d0, d1, hs_all);
    }
    __syncthreads();
    while (d0 < L.n) {
      const int e0 = d1, e1 = d1 < L.n ? chunk_end(d1) : d1;      // the next chunk
      const int n_tasks = e1 > e0 ? (L.base[e1] - L.base[e0]) * KT : 0;
      uint8_t* next_hs = hs_all + (bufs > 1 ? (buf ^ 1) : 0) * chunk_bytes;
      const uint8_t* hs = hs_all + buf * chunk_bytes;
      const float* fac = reinterpret_cast<const float*>(hs + (size_t)chunk_rows * hstride);
      int task = 2 * wid;
      for (; step < d1 * KT; step += kWarps) {
        const int d = step / KT, kt = step - d * KT;
        cp_async_wait<kDnStages - 1>();
        __syncwarp();
        const uint8_t* st = ring_p + slot * kDnStage;
        const uint8_t* sc = st + kDnTiles * 1024 + (g & 1) * 16 + (g >> 1) * 4 + (q & 1) * 2;
        const uint32_t mask = L.mask[d];
        const int r0 = L.base[d] - L.base[d0];
        TileA ta[kDnTiles];
        float2 s0[kDnTiles], s8[kDnTiles];
#pragma unroll
        for (int i = 0; i < kDnTiles; ++i) {
          if (i < tiles) {
            load_tile(ta[i], st + i * 1024 + g * 64 + q * 16, st + i * 1024 + 512 + g * 64 + q * 16);
            s0[i] = e8m0x2(*reinterpret_cast<const uint16_t*>(sc + i * 64));
            s8[i] = e8m0x2(*reinterpret_cast<const uint16_t*>(sc + i * 64 + 32));
          }
        }
#pragma unroll
        for (int n = 0; n < NTP; ++n) {
          if ((mask >> (2 * n)) & 3u) {
            const int tb = 2 * n + (g >> 2), tc = 2 * n + (q >> 1);
            TokB b;
            load_tok(b, q == (g & 3) && ((mask >> tb) & 1u)
                            ? hs + (r0 + __popc(mask & ((1u << tb) - 1u))) * hstride + kt * 128 + q * 32
                            : nullptr);
            const float f = ((mask >> tc) & 1u) ? fac[(r0 + __popc(mask & ((1u << tc) - 1u))) * KT + kt] : 0.f;
#pragma unroll
            for (int i = 0; i < kDnTiles; ++i) {
              if (i < tiles) {
                float cf[4];
                tile_mma(cf, ta[i], b);
                acc[i][n][0] = fmaf(cf[0], s0[i].x * f, fmaf(cf[1], s0[i].y * f, acc[i][n][0]));
                acc[i][n][1] = fmaf(cf[2], s8[i].x * f, fmaf(cf[3], s8[i].y * f, acc[i][n][1]));
              }
            }
          }
        }
        __syncwarp();
        fetch();
        slot = slot + 1 == kDnStages ? 0 : slot + 1;
        if (bufs > 1 && task < n_tasks) {
          quant_task(task + (lane >> 4), n_tasks, e0, e1, next_hs);
          task += 2 * kWarps;
        }
      }
      if (bufs == 1) __syncthreads();     // the chunk's readers are done
      for (; task < n_tasks; task += 2 * kWarps) quant_task(task + (lane >> 4), n_tasks, e0, e1, next_hs);
      __syncthreads();
      d0 = e0;
      d1 = e1;
      if (bufs > 1) buf ^= 1;
    }
    // ---- sum over the warps, two tokens a round ----
#pragma unroll
    for (int n = 0; n < NTP; ++n) {
      if (2 * n < a.T) {
#pragma unroll
        for (int i = 0; i < kDnTiles; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float v = acc[i][n][h];
            v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
            if ((q & 1) == 0) red[((wid * 2 + (q >> 1)) * kDnTiles + i) * 16 + h * 8 + g] = v;
          }
        }
        __syncthreads();
        if (tid < 2 * kDnTiles * 16) {
          const int set = tid / (kDnTiles * 16), i = (tid / 16) % kDnTiles, rr = tid % 16;
          const int s = 4 * i + 2 * (rr >> 3) + (rr & 1), su = u0 + s, t = 2 * n + set;
          if (t < a.T && s < nsub) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[((w * 2 + set) * kDnTiles + i) * 16 + rr];
            reinterpret_cast<__nv_bfloat16*>(a.y)[(int64_t)t * a.H + (su >> 5) * 128 + 32 * ((rr & 7) >> 1) + (su & 31)] =
                __float2bfloat16_rn(v);
          }
        }
        __syncthreads();
      }
    }
  }
  if (!waited) pdl_wait();
  cp_async_wait<0>();
}

}  // namespace few
}  // namespace moe

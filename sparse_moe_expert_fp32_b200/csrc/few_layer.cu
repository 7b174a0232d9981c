// few_layer.cu -- the whole MoE layer for 1 to 8 tokens in one kernel (Qwen3.8-Flash-Next
// architecture study, MoE section: "Router [T, 512] -> Top 10 + normalize -> Dispatch R tokens
// -> Grouped expert GEMMs -> Weighted combine + gated shared expert").
//
// With a few tokens the layer is the reading of the activated experts' weights; launches, and
// the waits between them, are the rest. So one cooperative kernel, one CTA per SM, runs the
// stages with two grid-wide barriers between them:
//   1. logits. A CTA takes E / grid rows of the router matrix; sums in 64 bits, so that the
//      choice of experts is the exact one (a near-tie decided by rounding would change the
//      output by whole experts).
//   2. shared expert's gate|up tiles, which need no routing, while the barrier fills.
//   -- barrier: all logits are there. Every CTA selects the top-k of all tokens for itself.
//   3. gate|up tiles of the chosen experts: 8 channels (8 gate rows and the 8 up rows: one m16
//      tile, so a thread holds the gate and the up sum of the same channel) by the full hidden
//      size, split over the CTA's 16 warps. The epilogue multiplies h = SiLU(gate) up by the
//      routing weight and stores it as three bf16 pieces (truncations; exactly fp32's 24 bits).
//   -- barrier: all of h is there.
//   4. down. A CTA owns H / grid output rows and runs through all chosen experts, accumulating
//      in registers: the routing weights are in h, so the weighted combine is the sum over the
//      experts and nothing is added atomically. The result does not depend on timing.
// The MMA columns are the tokens themselves: a tile multiplies all tokens, and the columns of
// tokens not routed to its expert are dropped (not multiplied by zero, so that an infinite or
// NaN weight stays within the tokens that chose its expert).
#include <float.h>

#include <mutex>

#include "moe_internal.h"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kFewWarps = 16;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewPairs = kFewMaxT * (kMaxK + 1);  // (token, expert) pairs, shared expert included
constexpr int kFewRows = 32;                       // output rows of one pass of the down stage
static_assert(2 * 16 * kFewMaxT == kFewRows * kFewMaxT, "the two users of FewShared::red");
constexpr uint64_t kFewWaitNs = 2000000000ull;

struct FewArgs {
  const uint16_t* x;
  const float* w_router;
  const float* bias;
  const uint16_t* wsg;
  const uint8_t* gate_up;  // routed banks: bf16, or codes
  const uint8_t* down;
  const uint16_t* s_gate_up;  // scales of the codes
  const uint16_t* s_down;
  const uint16_t* ws_gate_up;
  const uint16_t* ws_down;
  float* out;
  int32_t* ids;
  float* w;
  float* gap;
  double* logits;   // [T][E]
  uint16_t* h;      // [3][pairs][ldh]
  size_t h_plane;
  uint32_t* sync;   // barrier counters: zero between calls
  uint32_t* status;
  int T, H, E, k, I, Is, ldh, shift;
};

struct FewShared {
  double part[kFewWarps][32];               // router partial sums
  float red[2][kFewWarps][16 * kFewMaxT];   // cross-warp sums; the down stage uses both halves
  uint32_t mask[kMaxE];                     // tokens that chose an expert
  uint16_t index[kMaxE];                    // its place among the active ones
  int scan[2 * kFewWarps + 2];
  float sel_w[kFewMaxT][kMaxK];
  int16_t sel_e[kFewMaxT][kMaxK];
  float sgate[kFewMaxT];
  float pair_w[kFewPairs];
  int16_t act_e[kFewMaxT * kMaxK + 1];      // entry 0: the shared expert
  int16_t act_pair[kFewMaxT * kMaxK + 1];   // first pair of the expert
  uint8_t act_mask[kFewMaxT * kMaxK + 1];
  int n_act;
};

__device__ __forceinline__ uint4 ld_cg_v4(const void* p) {
  return __ldcg(reinterpret_cast<const uint4*>(p));
}

__device__ __forceinline__ void grid_arrive(uint32_t* c) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(c, 1u);
  }
}

// Bounded: on expiry the flag is set and the kernel runs on with what it has.
__device__ __forceinline__ void grid_wait(uint32_t* c, uint32_t* status) {
  if (threadIdx.x == 0) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t spin = 1;; ++spin) {
      uint32_t v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(c) : "memory");
      if (v >= gridDim.x) break;
      if ((spin & 63u) == 0 && globaltimer_ns() - t0 > kFewWaitNs) {
        set_flag(status, kFlagTimeout);
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();
}

// Order-preserving key of a logit: larger key = larger value, NaN below everything, 0 = none.
__device__ __forceinline__ uint64_t logit_key(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);  // -0 and +0 are equal
  const uint64_t k = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return v == v ? k : 1ull;
}
__device__ __forceinline__ double key_logit(uint64_t k) {
  if (k == 1ull) return __longlong_as_double(0x7ff8000000000000ll);
  return __longlong_as_double((long long)((k >> 63) ? (k & 0x7fffffffffffffffull) : ~k));
}

// One warp: top-k of token t (largest first, ties to the lowest index), softmax over the chosen.
__device__ void select_token(const FewArgs& a, FewShared& S, int t, int lane) {
  constexpr int VPL = kMaxE / 32;
  uint64_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = lane + 32 * i;
    key[i] = 0;
    if (e < a.E) {
      double v = __ldcg(a.logits + (size_t)t * a.E + e);
      if (a.bias) v += (double)__ldg(a.bias + e);
      key[i] = logit_key(v);
    }
  }
  int my_e = 0;
  double my_v = 0.0, next = 0.0;
  const int rounds = a.k < a.E ? a.k + 1 : a.k;
  for (int r = 0; r < rounds; ++r) {
    uint64_t best = 0;
    int be = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) {
        best = key[i];
        be = lane + 32 * i;
      }
    const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(best >> 32));
    bool c = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, c ? (uint32_t)best : 0u);
    c = c && (uint32_t)best == lo;
    const int e = __reduce_min_sync(0xffffffffu, c ? be : 0x7fffffff);
    const double v = key_logit(((uint64_t)hi << 32) | lo);
    if (r < a.k) {
      if (lane == r) {
        my_e = e;
        my_v = v;
      }
    } else {
      next = v;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (e == lane + 32 * i) key[i] = 0;
  }
  const double vmax = __shfl_sync(0xffffffffu, my_v, 0);
  const float ex = lane < a.k ? expf((float)(my_v - vmax)) : 0.f;
  const float p = ex / warp_sum(ex);
  if (lane < a.k) {
    S.sel_e[t][lane] = (int16_t)my_e;
    S.sel_w[t][lane] = p;
    atomicOr(&S.mask[my_e], 1u << t);
    if (blockIdx.x == 0) {
      if (a.ids) a.ids[(size_t)t * a.k + lane] = my_e;
      if (a.w) a.w[(size_t)t * a.k + lane] = p;
    }
  }
  const double kth = __shfl_sync(0xffffffffu, my_v, a.k - 1);
  if (blockIdx.x == 0 && a.gap && lane == 0)
    a.gap[t] = a.k < a.E ? (float)(kth - next) : __int_as_float(0x7f800000);
}

// The active experts in ascending order, and the pairs (expert, token) in that order.
__device__ void build_active(const FewArgs& a, FewShared& S) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int e0 = 2 * tid;  // two experts a thread
  const uint32_t m0 = e0 < a.E ? S.mask[e0] : 0u, m1 = e0 + 1 < a.E ? S.mask[e0 + 1] : 0u;
  const int n = (((m0 != 0) + (m1 != 0)) << 16) | (__popc(m0) + __popc(m1));
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) S.scan[warp] = incl;
  __syncthreads();
  int before = (1 << 16) | a.T, total = 0;  // entry 0 and the pairs 0 .. T-1: the shared expert
  for (int i = 0; i < kFewWarps; ++i) {
    if (i < warp) before += S.scan[i];
    total += S.scan[i];
  }
  before += incl - n;
  int at = before >> 16, pair = before & 0xffff;
  const uint32_t m[2] = {m0, m1};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!m[i]) continue;
    S.act_e[at] = (int16_t)(e0 + i);
    S.act_pair[at] = (int16_t)pair;
    S.act_mask[at] = (uint8_t)m[i];
    S.index[e0 + i] = (uint16_t)at;
    ++at;
    pair += __popc(m[i]);
  }
  if (tid == 0) S.n_act = 1 + (total >> 16);
  __syncthreads();
  if (tid < a.T * a.k) {
    const int t = tid / a.k, j = tid - t * a.k;
    const int s = S.index[S.sel_e[t][j]];
    S.pair_w[S.act_pair[s] + __popc(S.act_mask[s] & ((1u << t) - 1u))] = S.sel_w[t][j];
  }
  __syncthreads();
}

// Row sums of one 8-channel gate|up tile over this warp's share of the hidden size.
__device__ __forceinline__ void tile_bf16(const uint8_t* gate, const uint8_t* up, int nk, const uint8_t* xs,
                                          bool tok, int warp, int t4, float (&acc)[4]) {
  for (int kb = warp; kb < nk; kb += 4 * kFewWarps) {
    uint4 wa[4], wb[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (kb + u * kFewWarps < nk) {
        const size_t at = (size_t)(kb + u * kFewWarps) * 64 + 16 * t4;
        wa[u] = ld_stream_v4(gate + at);
        wb[u] = ld_stream_v4(up + at);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (kb + u * kFewWarps < nk) {
        uint4 xb = make_uint4(0u, 0u, 0u, 0u);
        if (tok) xb = *reinterpret_cast<const uint4*>(xs + (size_t)(kb + u * kFewWarps) * 64 + 16 * t4);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma_k32<false>(d, wa[u], wb[u], xb);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += d[i];
      }
  }
}

__device__ __forceinline__ void tile_w4(const uint8_t* gate, const uint8_t* up, const uint16_t* sgp,
                                        const uint16_t* sup, int nk, int shift, const uint8_t* xs,
                                        bool tok, int warp, int t4, float (&acc)[4]) {
  const int nb = (nk + 3) / 4;
  for (int b = warp; b < nb; b += kFewWarps) {
    const uint4 wa = ld_stream_v4(gate + (size_t)b * 64 + 16 * t4);
    const uint4 wb = ld_stream_v4(up + (size_t)b * 64 + 16 * t4);
    float sa[4], sb[4];
    w4_block_scales(sgp, b, shift, sa);
    w4_block_scales(sup, b, shift, sb);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (4 * b + j >= nk) break;
      uint4 xb = make_uint4(0u, 0u, 0u, 0u);
      if (tok) xb = *reinterpret_cast<const uint4*>(xs + (size_t)(4 * b + j) * 64 + 16 * t4);
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_k32<false>(d, w4_pairs<false>((&wa.x)[j]), w4_pairs<false>((&wb.x)[j]), xb);
      acc[0] = fmaf(d[0], sa[j], acc[0]);
      acc[1] = fmaf(d[1], sa[j], acc[1]);
      acc[2] = fmaf(d[2], sb[j], acc[2]);
      acc[3] = fmaf(d[3], sb[j], acc[3]);
    }
  }
}

// Gate|up tiles [u0, u1) of this CTA's stride: tiles of the shared expert first.
template <bool W4>
__device__ void gate_up_tiles(const FewArgs& a, FewShared& S, const uint8_t* xs, int xpitch, int u0,
                              int u1) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int ns = a.Is / 8, nr = a.I / 8;
  const bool tok = g < a.T;
  const uint8_t* xg = xs + (size_t)g * xpitch;
  int buf = 0;
  for (int u = u0 + (int)((blockIdx.x + gridDim.x - u0 % gridDim.x) % gridDim.x); u < u1; u += gridDim.x) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    int s = 0, c0 = 8 * u;
    if (u < ns) {
      const uint8_t* base = reinterpret_cast<const uint8_t*>(a.ws_gate_up);
      const size_t rb = 2 * (size_t)a.H;
      tile_bf16(base + (size_t)(c0 + g) * rb, base + (size_t)(a.Is + c0 + g) * rb, a.H / 32, xg, tok,
                warp, t4, acc);
    } else {
      s = 1 + (u - ns) / nr;
      c0 = 8 * ((u - ns) % nr);
      const size_t row = (size_t)S.act_e[s] * 2 * a.I + c0 + g;
      if constexpr (W4) {
        const size_t rb = w4_row_bytes(a.H), rs = w4_row_scales(a.H, 32 << a.shift);
        tile_w4(a.gate_up + row * rb, a.gate_up + (row + a.I) * rb, a.s_gate_up + row * rs,
                a.s_gate_up + (row + a.I) * rs, a.H / 32, a.shift, xg, tok, warp, t4, acc);
      } else {
        const size_t rb = 2 * (size_t)a.H;
        tile_bf16(a.gate_up + row * rb, a.gate_up + (row + a.I) * rb, a.H / 32, xg, tok, warp, t4, acc);
      }
    }
    float* red = S.red[buf][warp];
    *reinterpret_cast<float2*>(red + 8 * g + 2 * t4) = make_float2(acc[0], acc[1]);
    *reinterpret_cast<float2*>(red + 8 * (g + 8) + 2 * t4) = make_float2(acc[2], acc[3]);
    __syncthreads();
    if (tid < 64) {
      const int t = tid >> 3, c = tid & 7;
      const uint32_t m = s ? S.act_mask[s] : (1u << a.T) - 1u;
      if ((m >> t) & 1u) {
        float gate = 0.f, up = 0.f;
        for (int w = 0; w < kFewWarps; ++w) {
          gate += S.red[buf][w][8 * c + t];
          up += S.red[buf][w][8 * (c + 8) + t];
        }
        const int pair = s ? S.act_pair[s] + __popc(m & ((1u << t) - 1u)) : t;
        const float h = gate / (1.f + expf(-gate)) * up * (s ? S.pair_w[pair] : S.sgate[t]);
        // three truncated pieces: 8 + 8 + 8 significant bits, h exactly (an infinity or NaN in
        // the first alone)
        const uint32_t hb = __float_as_uint(h);
        const bool fin = fabsf(h) <= FLT_MAX;
        const float r1 = fin ? h - __uint_as_float(hb & 0xffff0000u) : 0.f;
        const uint32_t mb = __float_as_uint(r1);
        const float r2 = r1 - __uint_as_float(mb & 0xffff0000u);
        uint16_t* o = a.h + (size_t)pair * a.ldh + c0 + c;
        o[0] = (h == h) ? (uint16_t)(hb >> 16) : (uint16_t)0x7fc0u;
        o[a.h_plane] = (uint16_t)(mb >> 16);
        o[2 * a.h_plane] = (uint16_t)(__float_as_uint(r2) >> 16);
      }
    }
    buf ^= 1;  // the next tile's sums go to the other half: one barrier a tile is enough
  }
}

template <bool W4>
__device__ void down_rows(const FewArgs& a, FewShared& S) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int n0 = (int)((int64_t)blockIdx.x * a.H / gridDim.x);
  const int n1 = (int)((int64_t)(blockIdx.x + 1) * a.H / gridDim.x);
  float* red = &S.red[0][0][0];  // [warp][row][token]
  for (int r0 = n0; r0 < n1; r0 += kFewRows) {
    const int nr = min(kFewRows, n1 - r0);
    float acc[2][4] = {};
    int turn = 0;  // the blocks of all experts go to the warps in turn
    for (int s = 0; s < S.n_act; ++s) {
      const bool w4 = W4 && s > 0;
      const int K = s ? a.I : a.Is;
      const int nk = K / 32, n = w4 ? (nk + 3) / 4 : nk;
      const uint32_t m = s ? S.act_mask[s] : (1u << a.T) - 1u;
      const bool tok = (m >> g) & 1u;
      const bool c0 = (m >> (2 * t4)) & 1u, c1 = (m >> (2 * t4 + 1)) & 1u;
      const int pair = (s ? S.act_pair[s] : 0) + __popc(m & ((1u << g) - 1u));
      const uint8_t* h = reinterpret_cast<const uint8_t*>(a.h + (size_t)pair * a.ldh) + 16 * t4;
      const size_t row = s ? (size_t)S.act_e[s] * a.H + r0 + g : (size_t)(r0 + g);
      const size_t rb = w4 ? (size_t)w4_row_bytes(K) : 2 * (size_t)K;
      const uint8_t* base = (s ? a.down : reinterpret_cast<const uint8_t*>(a.ws_down)) + row * rb + 16 * t4;
      for (int b = (warp + kFewWarps - turn) % kFewWarps; b < n; b += kFewWarps) {
        uint4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t zero = w4 ? 0x88888888u : 0u;
          w[i] = make_uint4(zero, zero, zero, zero);
          if (g + 8 * i < nr) w[i] = ld_stream_v4(base + 8 * i * rb + (size_t)b * 64);
        }
        auto part = [&](int kb, const uint4& xa, const uint4& xb, int i, float s0, float s1) {
          uint4 hp[3] = {};
          if (tok)
#pragma unroll
            for (int p = 0; p < 3; ++p) hp[p] = ld_cg_v4(h + 2 * p * a.h_plane + (size_t)kb * 64);
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int p = 2; p >= 0; --p) mma_k32<false>(d, xa, xb, hp[p]);  // small pieces first
          if (c0) {
            acc[i][0] = fmaf(d[0], s0, acc[i][0]);
            acc[i][2] = fmaf(d[2], s1, acc[i][2]);
          }
          if (c1) {
            acc[i][1] = fmaf(d[1], s0, acc[i][1]);
            acc[i][3] = fmaf(d[3], s1, acc[i][3]);
          }
        };
        if (W4 && w4) {
          float sc[4][4] = {};
          const size_t rs = w4_row_scales(K, 32 << a.shift);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (g + 8 * i < nr) w4_block_scales(a.s_down + (row + 8 * i) * rs, b, a.shift, sc[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (4 * b + j >= nk) break;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              part(4 * b + j, w4_pairs<false>((&w[2 * i].x)[j]), w4_pairs<false>((&w[2 * i + 1].x)[j]), i,
                   sc[2 * i][j], sc[2 * i + 1][j]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) part(b, w[2 * i], w[2 * i + 1], i, 1.f, 1.f);
        }
      }
      turn = (turn + n) % kFewWarps;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
        *reinterpret_cast<float2*>(red + (warp * kFewRows + 16 * i + 8 * p + g) * kFewMaxT + 2 * t4) =
            make_float2(acc[i][2 * p], acc[i][2 * p + 1]);
    __syncthreads();
    const int r = tid % kFewRows, t = tid / kFewRows;
    float sum = 0.f;
    if (t < kFewMaxT)
      for (int w = 0; w < kFewWarps; ++w) sum += red[(w * kFewRows + r) * kFewMaxT + t];
    if (t < a.T && r < nr) a.out[(size_t)t * a.H + r0 + r] = sum;
  }
}

template <bool W4>
__global__ void __launch_bounds__(kFewThreads, 1) few_layer_kernel(const FewArgs a) {
  extern __shared__ uint4 smem[];
  FewShared& S = *reinterpret_cast<FewShared*>(smem);
  uint8_t* xs = reinterpret_cast<uint8_t*>(smem) + (sizeof(FewShared) + 127) / 128 * 128;
  const int xpitch = 2 * a.H + 64;  // 64 mod 128: two tokens' 64-byte reads share no bank
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  for (int i = tid; i < a.T * (a.H / 8); i += kFewThreads) {
    const int t = i / (a.H / 8), c = i - t * (a.H / 8);
    *reinterpret_cast<uint4*>(xs + (size_t)t * xpitch + 16 * c) = ld_v4(a.x + (size_t)t * a.H + 8 * c);
  }
  for (int e = tid; e < a.E; e += kFewThreads) S.mask[e] = 0;
  __syncthreads();

  // logits of this CTA's router rows, four at a time; a warp takes a slice of the hidden size
  const int e0 = (int)((int64_t)blockIdx.x * a.E / gridDim.x);
  const int e1 = (int)((int64_t)(blockIdx.x + 1) * a.E / gridDim.x);
  for (int e = e0; e < e1; e += 4) {
    double acc[4][kFewMaxT] = {};
    for (int c = warp * 32 + lane; c < a.H; c += kFewThreads) {
      float w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = e + i < e1 ? __ldg(a.w_router + (size_t)(e + i) * a.H + c) : 0.f;
#pragma unroll
      for (int t = 0; t < kFewMaxT; ++t)
        if (t < a.T) {
          const uint32_t b = *reinterpret_cast<const uint16_t*>(xs + (size_t)t * xpitch + 2 * c);
          const double xv = (double)__uint_as_float(b << 16);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i][t] = fma((double)w[i], xv, acc[i][t]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < kFewMaxT; ++t)
        if (t < a.T) {
          double v = acc[i][t];
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          if (lane == 0) S.part[warp][i * kFewMaxT + t] = v;
        }
    __syncthreads();
    if (tid < 32) {
      const int i = tid / kFewMaxT, t = tid % kFewMaxT;
      if (t < a.T && e + i < e1) {
        double v = 0.0;
        for (int w = 0; w < kFewWarps; ++w) v += S.part[w][tid];
        a.logits[(size_t)t * a.E + e + i] = v;
      }
    }
    __syncthreads();
  }
  grid_arrive(a.sync);

  // the shared expert: its output gate, then its gate|up tiles
  if (warp < a.T) {
    float v = 0.f;
    const uint8_t* xr = xs + (size_t)warp * xpitch;
    for (int c = lane; c < a.H / 8; c += 32) {
      float xf[8];
      unpack8(*reinterpret_cast<const uint4*>(xr + 16 * c), xf);
      v = dot8_acc(ld_v4(a.wsg + 8 * c), xf, v);
    }
    v = warp_sum(v);
    if (lane == 0) S.sgate[warp] = 1.f / (1.f + expf(-v));
  }
  __syncthreads();
  const int ns = a.Is / 8;
  gate_up_tiles<W4>(a, S, xs, xpitch, 0, ns);

  grid_wait(a.sync, a.status);
  if (warp < a.T) select_token(a, S, warp, lane);
  __syncthreads();
  build_active(a, S);
  gate_up_tiles<W4>(a, S, xs, xpitch, ns, ns + (S.n_act - 1) * (a.I / 8));

  grid_arrive(a.sync + 1);
  grid_wait(a.sync + 1, a.status);
  down_rows<W4>(a, S);

  // the last CTA to leave makes the counters ready for the next call
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(a.sync + 2, 1u) + 1 == gridDim.x) {
      a.sync[0] = 0;
      a.sync[1] = 0;
      a.sync[2] = 0;
    }
  }
}

}  // namespace

bool few_supported(const moe_shape& s) {
  return s.T <= kFewMaxT && (int64_t)s.T * s.H <= kFewMaxTH;
}

cudaError_t launch_few_layer(const moe_shape& s, const Layout& L, char* ws, const uint16_t* x,
                             const moe_weights& w, const moe_w4_experts* q, float* out,
                             int32_t* ids, float* topk_w, float* gap, int sms, cudaStream_t st) {
  FewArgs a{};
  a.x = x;
  a.w_router = w.w_router;
  a.bias = w.router_bias;
  a.wsg = static_cast<const uint16_t*>(w.w_shared_gate);
  a.gate_up = static_cast<const uint8_t*>(q ? q->q_gate_up : w.w_gate_up);
  a.down = static_cast<const uint8_t*>(q ? q->q_down : w.w_down);
  a.s_gate_up = q ? static_cast<const uint16_t*>(q->s_gate_up) : nullptr;
  a.s_down = q ? static_cast<const uint16_t*>(q->s_down) : nullptr;
  a.shift = q ? (q->group == 32 ? 0 : q->group == 64 ? 1 : 2) : 0;
  a.ws_gate_up = static_cast<const uint16_t*>(w.ws_gate_up);
  a.ws_down = static_cast<const uint16_t*>(w.ws_down);
  a.out = out;
  a.ids = ids;
  a.w = topk_w;
  a.gap = gap;
  a.logits = reinterpret_cast<double*>(ws + L.logits);
  a.h = reinterpret_cast<uint16_t*>(ws + L.few_h);
  a.h_plane = (size_t)s.T * (s.k + 1) * L.ldh;
  a.ldh = L.ldh;
  a.sync = reinterpret_cast<uint32_t*>(ws + L.status) + kFewSyncWord;
  a.status = reinterpret_cast<uint32_t*>(ws + L.status);
  a.T = s.T; a.H = s.H; a.E = s.E; a.k = s.k; a.I = s.I; a.Is = s.Is;
  const size_t smem = (sizeof(FewShared) + 127) / 128 * 128 + (size_t)s.T * (2 * s.H + 64);
  const void* fn = q ? (const void*)few_layer_kernel<true> : (const void*)few_layer_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  LaunchScope scope(MOE_K_OTHER, st);
  void* params[] = {&a};
  // cooperative: the CTAs wait for one another, so all of them have to be resident at once
  e = cudaLaunchCooperativeKernel(fn, dim3(sms), dim3(kFewThreads), params, smem, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

// few_layer.cu -- the whole MoE layer for 1 to 8 tokens in one kernel (Qwen3.8-Flash-Next
// architecture study, MoE section: "Router [T, 512] -> Top 10 + normalize -> Dispatch R tokens
// -> Grouped expert GEMMs -> Weighted combine + gated shared expert").
//
// With a few tokens the layer is the reading of the activated experts' weights; launches, and
// the waits between them, are the rest. So one cooperative kernel, one CTA per SM, runs the
// stages with two grid-wide barriers between them:
//   1. logits. A CTA takes E / grid rows of the router matrix; sums and comparisons in 64 bits
//      (a near-tie decided by fp32 rounding would change the output by whole experts). The calls
//      for whole batches compare logits rounded to fp32: what is a tie there is none here.
//   2. shared expert's gate|up tiles, which need no routing, while the barrier fills.
//   -- barrier: all logits are there. Every CTA selects the top-k of all tokens for itself.
//   3. gate|up tiles of the chosen experts: 8 channels (8 gate rows and the 8 up rows) by the full
//      hidden size, by a team of four of the twelve consumer warps, which split K. The epilogue
//      multiplies h = SiLU(gate) up by the routing weight and stores it as three bf16 pieces
//      (truncations; exactly fp32's 24 bits).
//   -- barrier: all of h is there.
//   4. down. A CTA owns H / grid output rows and runs through all chosen experts, a stage's blocks
//      of K split over a team; every warp keeps sums of its own, added up at the end: the routing
//      weights are in h, so the weighted combine is the sum over the experts and nothing is added
//      atomically. The result does not depend on timing.
// A tile multiplies all tokens (they are the MMA's columns), and the columns of tokens not routed to
// its expert are dropped, not multiplied by zero, so that an infinite or NaN weight stays within the
// tokens that chose its expert.
//
// mma.sync rather than tcgen05: a weight is used 1 to 8 times, so its bytes are the bound, and what
// counts is how few instructions make operands of them. bf16 weights are the A of m16n8k16 just as a
// 16-byte load leaves them (mma_rows); a tcgen05 tile would have 128 rows of one expert and leave
// 7/8 of its columns empty, and 4-bit weights would go back to shared memory as bf16 first.
//
// Measured on one B200, weights not in L2, H = 2560, E = 512, k = 10, I = Is = 640 unless said; the
// floor is the weights' bytes at the measured copy rate of 6.56 TB/s:
//   bf16   1 token 35.3 us (floor 17), 8 tokens 146 us (115: 5.1 TB/s)
//          4 tokens, H = 8192, E = 64, I = Is = 2048, some 26 experts chosen: 446 us (415: 6.1 TB/s)
//   4-bit  1 token 29 us (6.5), 5 tokens 66 us (21); 8 tokens, H = 8192, I = 2048: 439 us (204)
// bf16 with several tokens is bound by HBM. One token: a layer with 1 MB of weights takes 16.4 us, which is
// launch, router, two grid barriers and the choice, none of them hidden. 4-bit weights are at no limit
// of the hardware: a clock and SM executes 1.55 of 4 instructions, 26 for each MMA, at 21 % of the DRAM rate.
// 9 of the 26 unpack codes; the rest of a block's work, and what surrounds the 5 blocks that a warp has
// of a tile (wait, fold, barrier, epilogue), are dependent chains, and three warps a scheduler cover little.
#include <float.h>

#include <algorithm>
#include <type_traits>

#include "moe_internal.h"
#include "sm100_ptx.cuh"
#include "tc_common.cuh"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kFewWarps = 12;    // consumers
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewTeam = 4;      // warps that share a stage; the stages go to the teams in turn
constexpr int kFewTeams = kFewWarps / kFewTeam;
constexpr int kFewBlock = kFewThreads + 2 * 32;  // and one warp that feeds them weights, one h
constexpr int kFewPairs = kFewMaxT * (kMaxK + 1);  // (token, expert) pairs, shared expert included
constexpr int kFewRows = 32;                       // output rows of one pass of the down stage
constexpr int kFewMaxStages = 16;
constexpr int kFewParts = kFewWarps * kFewRows * kFewMaxT / 2;  // router partial sums; shares a place with sums of the tiles
constexpr uint64_t kFewWaitNs = 2000000000ull;
constexpr uint64_t kFewDrainNs = 200000000ull;
constexpr int kBarConsumers = 1, kBarRouted = 2, kBarTeam = 3;  // named barriers

// How a weight matrix comes through the ring: `n` chunks of a row, `cb` 64-byte blocks each (a block
// is 32 bf16 or 128 4-bit weights); scales `sc` bytes of a row and chunk.
struct FewChunks {
  int n, cb, sc, blocks;
  __device__ int scale_at(int c, int shift) const { return c * cb * 8 >> shift; }  // bytes, of chunk c
};

struct FewArgs {
  const uint16_t* x;
  const float* w_router;
  const float* bias;
  const uint16_t* wsg;
  float* out;
  int32_t* ids;
  float* w;
  float* gap;
  double* logits;   // [T][ldl]: router logits, then the shared expert's gate; rows of 16-byte units
  uint16_t* h;      // [pairs][ldh / 32][3][32]: three pieces of 32 channels side by side
  uint32_t* sync;   // barrier counters: zero between calls
  uint32_t* status;
  int T, H, E, k, I, Is, ldh, ldl, shift;
  uint32_t per_tile;  // 2^32 over the tiles of an expert, rounded up
  FewChunks gu, gu_s, dn, dn_s;  // gate|up and down matrices, routed and shared
  int rows;                      // output rows of a pass
  int stages, stage_bytes;
  int group, slot;               // experts of a down stage at most, bytes of one of them in it
  int unit, units, h_bytes;      // ring of h: bytes of a token's chunk, number of them, region
};

// Tensor maps of the weights (bytes; innermost first), each stage one box of each:
//   gate|up  [64][channel][block][gate, up][expert], box 64 x 8 x cb x 2 x 1
//   down     [64][output row][block][expert], box 64 x rows x cb x 1
//   scales   [bytes of a row][channel][gate, up][expert] and [bytes of a row][output row][expert]
struct FewMaps {
  CUtensorMap gu, gu_s, dn, dn_s, gu_sc, dn_sc;
};

struct FewShared {
  uint64_t full[kFewMaxStages], empty[kFewMaxStages], x_full, logits_full;
  int tag[kFewMaxStages];                   // number of the stage that a slot is filled with
  uint8_t stage_units[kFewMaxStages];       // units of h that a stage in flight uses
  union {
    double part[kFewParts];  // router partial sums: [stage][warp of the team][token]
    struct {
      uint64_t key[kFewMaxT][64];            // selection: candidates of a token
      uint16_t e[kFewMaxT][64];
    } cand;
    float red[2][kFewTeams][kFewTeam][16 * kFewMaxT];  // cross-warp sums of the teams' tiles
    float out[kFewWarps][kFewRows][kFewMaxT];          // and of the down stage
  };
  uint32_t mask[kMaxE];                     // tokens that chose an expert
  uint16_t index[kMaxE];                    // its place among the active ones
  int scan[kFewWarps];
  double sel_v[kFewMaxT][kMaxK + 1];
  float sel_w[kFewMaxT][kMaxK];
  int16_t sel_e[kFewMaxT][kMaxK + 1];
  float sgate[kFewMaxT];                    // zero behind the last token
  float pair_w[kFewPairs];
  int16_t act_e[kFewMaxT * kMaxK + 1];      // entry 0: the shared expert
  int16_t act_pair[kFewMaxT * kMaxK + 2];   // first pair of the expert; behind the last one: pairs
  uint8_t act_mask[kFewMaxT * kMaxK + 1];
  int n_act;
  int aborted;
  int parked;  // feeders that arrive on no barrier: not before the experts are known, or never again
};


constexpr size_t kFewSharedBytes = (sizeof(FewShared) + 127) / 128 * 128;
constexpr size_t kFewSmem = 227 * 1024;

__device__ __forceinline__ void sync_consumers() { ptx::bar_sync(kBarConsumers, kFewThreads); }

__device__ __forceinline__ void give_up(FewShared& S, uint32_t* status) {
  *reinterpret_cast<volatile int*>(&S.aborted) = 1;
  set_flag(status, kFlagTimeout);
}

// What a thread does whose wait has run out, or that of another thread of the block. A consumer goes on
// without its stage and gives back a slot whose copies may still be in flight. Nobody may arrive on the
// slot's barrier until they have landed, so it waits (with a limit) until the feeders have stopped: they do
// at their next wait, at the end of the grid's barrier, or where they wait for the experts. x and the logits
// have no feeder that waits for them to land. (Kept out of the loops: a test of each wait's result there
// cost 1 token 0.5 to 0.8 us, this 0.3 to 0.5.)
__device__ __noinline__ bool run_out(uint64_t* bar, uint32_t parity, FewShared& S) {
  if (threadIdx.x >= kFewThreads) return false;
  __threadfence_block();
  const uint64_t t0 = globaltimer_ns();
  while (*reinterpret_cast<volatile int*>(&S.parked) != 2 && globaltimer_ns() - t0 < 2 * kFewWaitNs) {
  }
  if (bar == &S.x_full || bar == &S.logits_full) drain_phase(bar, parity);
  return false;
}

// Bounded wait on an mbarrier phase; false once any wait of the block has run out.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, FewShared& S, uint32_t* status) {
  uint64_t t0 = 0;
  for (uint32_t spin = 1;; ++spin) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if ((spin & 31u) == 0) {  // reading the clock is slow: only in long waits
      if (*reinterpret_cast<volatile int*>(&S.aborted)) return run_out(bar, parity, S);
      const uint64_t t = globaltimer_ns();
      if (!t0) t0 = t;
      if (t - t0 > kFewWaitNs) give_up(S, status);
    }
  }
}
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, FewShared& S, uint32_t* status) {
  if (ptx::mbar_test_wait(bar, parity)) return true;
  return wait_slow(bar, parity, S, status);
}

// Grid barriers. Bounded: on expiry the flag is set and the kernel runs on with what it has
// (nothing it reads then is used as an address).
__device__ __forceinline__ void grid_arrive(uint32_t* c) {
  sync_consumers();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(c, 1u);
  }
}
__device__ __forceinline__ void grid_wait(uint32_t* c, FewShared& S, uint32_t* status) {
  uint64_t t0 = 0;
  for (uint32_t spin = 1;; ++spin) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(c) : "memory");
    if (v >= gridDim.x) break;
    if ((spin & 63u) == 0) {
      const uint64_t t = globaltimer_ns();
      if (!t0) t0 = t;
      if (t - t0 > kFewWaitNs) {
        give_up(S, status);
        break;
      }
    }
  }
  __threadfence();
}

// ---------------------------------------------------------------- the ring
// Weights reach the consumers through a ring of stages in shared memory, filled by TMA: the copies
// in flight hold no registers, and the feeding thread runs ahead of the consumers across their
// barriers, so that HBM works on the down matrices while the last gate|up tiles are summed and the
// grid waits for h. A stage is a K chunk of some weight rows, [block][row][64 bytes]: one box, so
// one instruction (row by row copies of 1.3 KB are issue bound at 5.0 TB/s, boxes reach 6.9), and a
// warp reads 8 rows of a block as 512 bytes in a row. In the down stage h of the expert's tokens
// comes through a second ring, a unit a token and chunk, in the place where x was.
struct Cursor {
  int s;
  uint32_t parity;
  __device__ void next(int stages) {
    if (++s == stages) {
      s = 0;
      parity ^= 1u;
    }
  }
};

// A consumer's place: the number of a stage and the ring's slot for it.
struct Place {
  int i;
  Cursor cur;
  __device__ void skip(int n, int stages) {
    i += n;
    for (cur.s += n; cur.s >= stages; cur.s -= stages) cur.parity ^= 1u;
  }
  __device__ void back(int n, int stages) {
    i -= n;
    for (cur.s -= n; cur.s < 0; cur.s += stages) cur.parity ^= 1u;
  }
};

// Wait for the stage at `at`. A slot's stages go to different teams, and a team may come to it while
// the stage before is still on its way, one phase behind: that looks like the phase it waits for.
// So the slot also says which stage it is being filled with (it is not before the last one has been
// used up).
__device__ __noinline__ void tag_slow(volatile int* tag, int i, FewShared& S, uint32_t* status) {
  uint64_t t0 = 0;
  for (uint32_t spin = 1; *tag != i; ++spin)
    if ((spin & 255u) == 0) {
      if (*reinterpret_cast<volatile int*>(&S.aborted)) {
        run_out(nullptr, 0u, S);
        return;
      }
      const uint64_t t = globaltimer_ns();
      if (!t0) t0 = t;
      if (t - t0 > kFewWaitNs) give_up(S, status);
    }
}
__device__ __forceinline__ void wait_stage(const Place& at, FewShared& S, uint32_t* status) {
  volatile int* tag = &S.tag[at.cur.s];
  if (*tag != at.i) tag_slow(tag, at.i, S, status);
  wait_phase(&S.full[at.cur.s], at.cur.parity, S, status);
}

__device__ __forceinline__ int round128(int v) { return (v + 127) & ~127; }

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          ptx::smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(ptx::smem_u32(bar))
      : "memory");
}

#define MOE_TMA_LOAD(N) \
  "cp.async.bulk.tensor." N "d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
__device__ __forceinline__ void tma_3d(void* dst, const void* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(MOE_TMA_LOAD("3") "{%3, %4, %5}], [%2];" ::"r"(ptx::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
               : "memory");
}
__device__ __forceinline__ void tma_4d(void* dst, const void* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(MOE_TMA_LOAD("4") "{%3, %4, %5, %6}], [%2];" ::"r"(ptx::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
__device__ __forceinline__ void tma_5d(void* dst, const void* map, uint64_t* bar, int c0, int c1, int c2, int c3,
                                       int c4) {
  asm volatile(MOE_TMA_LOAD("5") "{%3, %4, %5, %6, %7}], [%2];" ::"r"(ptx::smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(map)), "r"(ptx::smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
               "r"(c4)
               : "memory");
}

// A thread that follows the stages in the consumers' order and does its part of each.
struct Feeder {
  const FewArgs& a;
  FewShared& S;
  uint8_t* ring;
  Cursor cur;
  int count;  // stages filled so far
  bool ok;

  __device__ uint8_t* begin() {
    ok = ok && wait_phase(&S.empty[cur.s], cur.parity ^ 1u, S, a.status);
    return ring + (size_t)cur.s * a.stage_bytes;
  }
  __device__ void tag() { *const_cast<volatile int*>(&S.tag[cur.s]) = count; }  // before the arrival
  __device__ void end() {
    cur.next(a.stages);
    ++count;
  }
  // leave no copy in flight: wait for the last phase of every stage that was filled
  __device__ void drain() {
    for (int i = 0; i < min(count, a.stages); ++i) {
      cur.s = cur.s ? cur.s - 1 : a.stages - 1;
      if (cur.s == a.stages - 1) cur.parity ^= 1u;
      uint64_t t0 = 0;
      while (!ptx::mbar_try_wait(&S.full[cur.s], cur.parity)) {
        const uint64_t t = globaltimer_ns();
        if (!t0) t0 = t;
        if (t - t0 > kFewDrainNs) break;
      }
    }
  }
};

// Order-preserving keys of a logit: larger key = larger value, NaN below everything but 0, which is
// none. (-0 does not occur: the sums start from +0.) high_key: from its upper half, with the lowest
// bit set, so that values with equal upper halves have equal keys.
__device__ __forceinline__ uint64_t logit_key(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return v == v ? b ^ (b >> 63 ? ~0ull : 1ull << 63) : 1ull;
}
__device__ __forceinline__ uint32_t high_key(int high) {
  if ((high & 0x7fffffff) > 0x7ff00000) return 1u;
  return ((uint32_t)(high ^ ((high >> 31) | (int)0x80000000)) | 1u);
}

// Top-k of token t by one warp (largest first, ties to the lowest index), softmax over the chosen;
// `row` holds its logits in shared memory, VPL a lane. The (k+1)-th largest of the lanes' maxima (of
// the keys' upper halves) bounds the (k+1)-th largest logit from below, so only those at or above it
// (about 1.5 k) are ranked, two a lane, each against all others. If more than 64 are left (k close to
// 32, many equal logits), k + 1 rounds of a warp maximum take their place. One warp, nothing to hide
// its latencies behind: the loops are unrolled for independent instructions.
template <int VPL>
__device__ __forceinline__ void select_token(const FewArgs& a, FewShared& S, const double* row, int t, int lane) {
  constexpr uint32_t all = 0xffffffffu;
  const int* half = reinterpret_cast<const int*>(row) + 1;
  const int rounds = a.k < a.E ? a.k + 1 : a.k;
  uint32_t high[VPL], best = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const uint32_t key = high_key(half[2 * min(lane + 32 * i, a.E - 1)]);
    high[i] = lane + 32 * i < a.E ? key : 0u;
    best = max(best, high[i]);
  }
  uint32_t bound = 1;  // every expert's key is at least 1
  if (VPL > 2 && rounds <= 32) {
    int rank = 0;
#pragma unroll
    for (int o = 0; o < 32; ++o) {
      const uint32_t other = __shfl_sync(all, best, o);
      rank += other > best || (other == best && o < lane);
    }
    bound = max(__shfl_sync(all, best, __ffs(__ballot_sync(all, rank == rounds - 1)) - 1), 1u);
  }
  int n = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const uint32_t m = __ballot_sync(all, high[i] >= bound);
    const int at = n + __popc(m & ((1u << lane) - 1u));
    if (high[i] >= bound && at < 64) S.cand.e[t][at] = (uint16_t)(lane + 32 * i);
    n += __popc(m);
  }
  __syncwarp();
  if (n <= 64) {
    // candidates are in ascending order of the expert: ties go to the lower place
    const int e0 = S.cand.e[t][min(lane, n - 1)], e1 = S.cand.e[t][min(lane + 32, n - 1)];
    const uint64_t k0 = lane < n ? logit_key(row[e0]) : 0ull, k1 = lane + 32 < n ? logit_key(row[e1]) : 0ull;
    S.cand.key[t][lane] = k0;
    S.cand.key[t][lane + 32] = k1;
    __syncwarp();
    int r0 = 0, r1 = 0;
    for (int i0 = 0; i0 < n; i0 += 8)
#pragma unroll
      for (int i = i0; i < i0 + 8; ++i) {
        const uint64_t other = S.cand.key[t][i];
        r0 += other > k0 || (other == k0 && i < lane);
        r1 += other > k1 || (other == k1 && i < lane + 32);
      }
    if (lane < n && r0 < rounds) {
      S.sel_v[t][r0] = row[e0];
      S.sel_e[t][r0] = (int16_t)e0;
    }
    if (lane + 32 < n && r1 < rounds) {
      S.sel_v[t][r1] = row[e1];
      S.sel_e[t][r1] = (int16_t)e1;
    }
  } else {
    uint32_t taken = 0;
    for (int r = 0; r < rounds; ++r) {
      uint64_t top = 0;
      int be = 0x7fffffff;
      for (int e = lane, i = 0; e < a.E; e += 32, ++i) {
        const uint64_t key = logit_key(row[e]);
        if (!((taken >> i) & 1u) && key > top) {
          top = key;
          be = e;
        }
      }
      const uint32_t hi = __reduce_max_sync(all, (uint32_t)(top >> 32));
      bool c = (uint32_t)(top >> 32) == hi;
      const uint32_t lo = __reduce_max_sync(all, c ? (uint32_t)top : 0u);
      c = c && (uint32_t)top == lo;
      const int e = __reduce_min_sync(all, c ? be : 0x7fffffff);
      if (lane == 0) {
        S.sel_v[t][r] = row[e];
        S.sel_e[t][r] = (int16_t)e;
      }
      if ((e & 31) == lane) taken |= 1u << (e >> 5);
    }
  }
  __syncwarp();
  const int e = S.sel_e[t][min(lane, a.k - 1)];
  const float ex = lane < a.k ? expf((float)(S.sel_v[t][min(lane, a.k - 1)] - S.sel_v[t][0])) : 0.f;
  const float p = ex / warp_sum(ex);
  if (lane < a.k) {
    S.sel_w[t][lane] = p;
    atomicOr(&S.mask[e], 1u << t);
    if (blockIdx.x == 0) {
      if (a.ids) a.ids[(size_t)t * a.k + lane] = e;
      if (a.w) a.w[(size_t)t * a.k + lane] = p;
    }
  }
  if (blockIdx.x == 0 && a.gap && lane == 0)
    a.gap[t] = a.k < a.E ? (float)(S.sel_v[t][a.k - 1] - S.sel_v[t][a.k]) : __int_as_float(0x7f800000);
}

// The active experts in ascending order, and the pairs (expert, token) in that order. The feeders
// start as soon as they know the experts.
__device__ void build_active(const FewArgs& a, FewShared& S) {
  constexpr int N = (kMaxE + kFewThreads - 1) / kFewThreads;  // experts a thread
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t m[N];
  int n = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m[i] = N * tid + i < a.E ? S.mask[N * tid + i] : 0u;
    n += ((m[i] != 0) << 16) + __popc(m[i]);
  }
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) S.scan[warp] = incl;
  sync_consumers();
  int before = (1 << 16) | a.T, total = 0;  // entry 0 and the pairs 0 .. T-1: the shared expert
#pragma unroll
  for (int i = 0; i < kFewWarps; ++i) {
    const int v = S.scan[i];
    if (i < warp) before += v;
    total += v;
  }
  before += incl - n;
  int at = before >> 16, pair = before & 0xffff;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (!m[i]) continue;
    S.act_e[at] = (int16_t)(N * tid + i);
    S.act_pair[at] = (int16_t)pair;
    S.act_mask[at] = (uint8_t)m[i];
    S.index[N * tid + i] = (uint16_t)at;
    ++at;
    pair += __popc(m[i]);
  }
  if (tid == 0) {
    S.n_act = 1 + (total >> 16);
    S.act_pair[1 + (total >> 16)] = (int16_t)(a.T + (total & 0xffff));
  }
  asm volatile("fence.proxy.async;" ::: "memory");  // the logits' place becomes the ring again
  ptx::bar_arrive(kBarRouted, kFewBlock);
  sync_consumers();
  if (tid < a.T * a.k) {
    const int t = tid / a.k, j = tid - t * a.k;
    const int s = S.index[S.sel_e[t][j]];
    S.pair_w[S.act_pair[s] + __popc(S.act_mask[s] & ((1u << t) - 1u))] = S.sel_w[t][j];
  }
  sync_consumers();
}

// ---------------------------------------------------------------- gate|up
// Tiles of 8 channels, the shared expert's (s = 0) first, then expert by expert; CTA b takes the
// tiles b, b + grid, ... in order.
struct Tiles {
  int u, s, c;  // tile, its expert's place among the active ones, its place in the expert
  __device__ void begin() {
    u = c = blockIdx.x;
    s = 0;
  }
  __device__ void settle(int ns, int nr) {
    while (c >= (s ? nr : ns)) {
      c -= s ? nr : ns;
      ++s;
    }
  }
  __device__ void next() {
    u += gridDim.x;
    c += gridDim.x;
  }
};

// The weights' feeder; `h`: the feeder of h, which has nothing to add to these stages. Tiles up to
// tile `end`.
template <int FMT>
__device__ void feed_gate_up(Feeder& f, const FewMaps& m, bool h, Tiles& tile, int end) {
  const FewArgs& a = f.a;
  for (; tile.u < end; tile.next()) {
    tile.settle(a.Is / 8, a.I / 8);
    const bool shared = tile.s == 0, w4 = FMT >= 0 && !shared;
    const FewChunks& ch = shared ? a.gu_s : a.gu;
    const int e = shared ? 0 : f.S.act_e[tile.s], c0 = 8 * tile.c;
    for (int c = 0; c < ch.n; ++c) {
      uint8_t* dst = f.begin();
      if (!f.ok) return;
      uint64_t* bar = &f.S.full[f.cur.s];
      if (h) {
        ptx::mbar_arrive(bar);
      } else {
        f.tag();
        ptx::mbar_arrive_expect_tx(bar, 1024 * ch.cb + (w4 ? 16 * ch.sc : 0));
        tma_5d(dst, shared ? &m.gu_s : &m.gu, bar, 0, c0, c * ch.cb, 0, e);
        if (w4) tma_4d(dst + 1024 * ch.cb, &m.gu_sc, bar, ch.scale_at(c, a.shift) & ~15, c0, 0, e);
      }
      f.end();
    }
  }
}

// The chunks of one tile, by one team: this warp's blocks of the gate and the up rows. bf16 weights
// are the MMA's A by mma_rows, 8 rows at a time, for 4 NQ tokens: `low` says which half of a
// column's registers the lane gives. An MMA chain is a stage's blocks at most; stages add up in fp32.
template <int NQ>
__device__ __forceinline__ void tile_bf16(const FewArgs& a, FewShared& S, const FewChunks& ch, uint32_t ring,
                                          Place at, uint32_t xs, int xpitch, int warp, int lane,
                                          float (&gate)[NQ][4], float (&up)[NQ][4]) {
  const int g = lane >> 2, t4 = lane & 3, wt = warp & (kFewTeam - 1);
  const bool low = g < 4;
  const uint32_t xg = xs + (g & 3) * xpitch + 16 * t4;
  int tok[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) tok[q] = 4 * q + (g & 3) < a.T;
  uint4 x[NQ];  // stays zero in the lanes of no token
#pragma unroll
  for (int q = 0; q < NQ; ++q) x[q] = make_uint4(0u, 0u, 0u, 0u);
  for (int c = 0; c < ch.n; ++c, at.skip(1, a.stages)) {
    const uint32_t st = ring + at.cur.s * a.stage_bytes;
    const int b0 = c * ch.cb, nb = min(ch.cb, ch.blocks - b0);
    wait_stage(at, S, a.status);
    uint32_t wp = st + 64 * g + 16 * t4 + 512 * wt, xp = xg + (b0 + wt) * 64;
    const uint32_t up_at = 512 * ch.cb;
    float dg[NQ][4] = {}, du[NQ][4] = {};
#pragma unroll 2
    for (int b = wt; b < nb; b += kFewTeam, wp += 512 * kFewTeam, xp += 64 * kFewTeam) {
      const uint4 wg = lds_v4(wp), wu = lds_v4(wp + up_at);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        lds_v4_if(x[q], xp + 4 * q * xpitch, tok[q]);
        const uint2 y = make_uint2(low ? x[q].x : x[q].y, low ? x[q].z : x[q].w);
        mma_rows(dg[q], wg, y);
        mma_rows(du[q], wu, y);
      }
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        gate[q][i] += dg[q][i];
        up[q][i] += du[q][i];
      }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.empty[at.cur.s]);
  }
}

// A half block, the last one of a row: parts 2 and 3 are multiplied by zero. The scale of a group
// that lies behind the row is not read either (a group of 128 has its first half in the row).
template <int FMT>
__device__ __forceinline__ void w4_half(uint4 (&x)[4], uint2& s0, uint2& s1) {
  x[2] = x[3] = make_uint4(0u, 0u, 0u, 0u);
  if (FMT < 2) s0.y = s1.y = 0u;
}

// The same for 4-bit weights. Their operands come out of arithmetic and can go to any register, so
// the MMA's A is the 8 gate rows and the 8 up rows, and its columns are the tokens. Chunks c, c + step, ...
// acc[0], [1]: gate row g, tokens 2 t and 2 t + 1; acc[2], [3]: the up row.
template <int FMT>
__device__ __forceinline__ void tile_w4(const FewArgs& a, FewShared& S, const FewChunks& ch, uint32_t ring,
                                        Place at, int c, int step, uint32_t xs, int xpitch, int warp, int lane,
                                        float (&acc)[4]) {
  const int g = lane >> 2, t4 = lane & 3, wt = warp & (kFewTeam - 1), tok = g < a.T;
  const uint32_t xg = xs + g * xpitch + 16 * t4;
  uint4 x[4] = {};  // stays zero in the lanes of no token
  for (at.skip(c, a.stages); c < ch.n; c += step, at.skip(step, a.stages)) {
    const uint32_t st = ring + at.cur.s * a.stage_bytes;
    const int b0 = c * ch.cb, nb = min(ch.cb, ch.blocks - b0);
    wait_stage(at, S, a.status);
    uint32_t wp = st + 64 * g + 16 * t4 + 512 * wt, xp = xg + (b0 + wt) * 256;
    const uint32_t up_at = 512 * ch.cb, sp = st + 1024 * ch.cb + g * ch.sc + (ch.scale_at(c, FMT) & 15);
    for (int b = wt; b < nb; b += kFewTeam, wp += 512 * kFewTeam, xp += 256 * kFewTeam) {
      const uint4 wg = lds_v4(wp), wu = lds_v4(wp + up_at);
      uint2 sg = w4_block_scales<FMT>(sp, b), su = w4_block_scales<FMT>(sp + 8 * ch.sc, b);
      const bool half = a.H / 32 - 4 * (b0 + b) == 2;  // H is a multiple of 64: four parts or two
#pragma unroll
      for (int j = 0; j < 4; ++j) lds_v4_if(x[j], xp + 64 * j, tok && (j < 2 || !half));
      if (half) w4_half<FMT>(x, sg, su);
      float d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 pg = w4_pairs<false>(word(wg, j)), pu = w4_pairs<false>(word(wu, j));
        // the parts of a group share a chain and a scale
        if (j % (1 << FMT) == 0) mma16816_first<false>(d, pg.x, pu.x, pg.y, pu.y, x[j].x, x[j].y);
        else mma16816<false>(d, pg.x, pu.x, pg.y, pu.y, x[j].x, x[j].y);
        mma16816<false>(d, pg.z, pu.z, pg.w, pu.w, x[j].z, x[j].w);
        if ((j + 1) % (1 << FMT) == 0) {
          const float fg = w4_scale(sg, j), fu = w4_scale(su, j);
          acc[0] = fmaf(d[0], fg, acc[0]);
          acc[1] = fmaf(d[1], fg, acc[1]);
          acc[2] = fmaf(d[2], fu, acc[2]);
          acc[3] = fmaf(d[3], fu, acc[3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.empty[at.cur.s]);
  }
}

// The two halves of mma_rows' sums: lane 4 g + t gets weight row g and columns 2 (t & 1) (v0) and
// 2 (t & 1) + 1 (v1).
__device__ __forceinline__ void fold(const float (&d)[4], bool low, float& v0, float& v1) {
  v0 = low ? d[0] : d[2];
  v1 = low ? d[1] : d[3];
  v0 += __shfl_xor_sync(0xffffffffu, v0, 2);
  v1 += __shfl_xor_sync(0xffffffffu, v1, 2);
}

// The tiles first, first + grid, ... of the shared expert or (`routed`) of the chosen ones, `count` of
// them; the teams take them in turn. `at`: the first tile's first stage, on
// return the one behind the last tile's.
template <int FMT, int NQ>
__device__ __forceinline__ void gate_up_tiles(const FewArgs& a, FewShared& S, uint32_t xs, int xpitch,
                                              uint32_t ring, Place& at, bool routed, int first, int count, int& turn) {
  constexpr bool W4 = FMT >= 0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int team = warp / kFewTeam, wt = warp & (kFewTeam - 1);
  const FewChunks& chunks = routed ? a.gu : a.gu_s;
  // a tile with so many chunks that two of them do not fit in the ring is taken by all teams (8 tokens
  // of H = 8192, four chunks in four stages: 433 us, by single teams 447 us; with the teams' turns
  // carried on from tile to tile and no barrier of all of them 446 us)
  const bool whole = W4 && 2 * chunks.n > a.stages;
  const int step = whole ? 1 : kFewTeams;
  int buf = 0, i = whole ? 0 : team >= turn ? team - turn : team - turn + kFewTeams;
  at.skip(i * chunks.n, a.stages);
  for (; i < count; i += step, at.skip(step * chunks.n, a.stages)) {
    const int u = first + i * gridDim.x;
    int s = 0, c0 = 8 * u;
    if (routed) {
      const int q = (int)__umulhi((uint32_t)u, a.per_tile);  // u / (I / 8), or one more
      s = 1 + q - (q * (a.I / 8) > u);
      c0 -= (s - 1) * a.I;
    }
    {
      float* red = S.red[buf][team][wt];  // [gate, up][token][channel]
      if constexpr (W4) {
        float acc[4] = {};
        tile_w4<FMT < 0 ? 0 : FMT>(a, S, chunks, ring, at, whole ? team : 0, whole ? kFewTeams : 1, xs, xpitch, warp,
                                   lane, acc);
        float* to = red + 16 * t4 + g;
        to[0] = kW4Unit<false> * acc[0];
        to[8] = kW4Unit<false> * acc[1];
        to[64] = kW4Unit<false> * acc[2];
        to[72] = kW4Unit<false> * acc[3];
      } else {
        float gate[NQ][4] = {}, up[NQ][4] = {};
        tile_bf16<NQ>(a, S, chunks, ring, at, xs, xpitch, warp, lane, gate, up);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          float g0, g1, v0, v1;
          fold(gate[q], t4 < 2, g0, g1);
          fold(up[q], t4 < 2, v0, v1);
          float* to = red + 8 * (4 * q + 2 * (t4 & 1)) + g + (t4 < 2 ? 0 : 64);
          to[0] = t4 < 2 ? g0 : v0;
          to[8] = t4 < 2 ? g1 : v1;
        }
      }
      if (whole) sync_consumers();
      else ptx::bar_sync(kBarTeam + team, 32 * kFewTeam);
      if (wt >> 1 == buf && (!whole || team == 0)) {  // a pair of the team's warps finishes the tile, the other pair its next one
        const int at64 = tid & 63, t = at64 >> 3, c = at64 & 7;
        const uint32_t m = routed ? S.act_mask[s] : (1u << a.T) - 1u;
        if ((m >> t) & 1u) {
          float gate = 0.f, up = 0.f;
          for (int q = whole ? 0 : team; q < (whole ? kFewTeams : team + 1); ++q)
#pragma unroll
            for (int w = 0; w < kFewTeam; ++w) {
              gate += S.red[buf][q][w][at64];
              up += S.red[buf][q][w][64 + at64];
            }
          const int pair = routed ? S.act_pair[s] + __popc(m & ((1u << t) - 1u)) : t;
          // SiLU first, and from exp(-|gate|) <= 1: a quotient of numbers that fp32 holds, whatever the
          // gate, and no product beyond what SiLU(gate) up itself reaches
          const float e = expf(-fabsf(gate)), silu = gate * __fdividef(gate < 0.f ? e : 1.f, 1.f + e);
          const float h = silu * up * (routed ? S.pair_w[pair] : 1.f);
          // three truncated pieces: 8 + 8 + 8 significant bits, h exactly (an infinity or NaN in
          // the first alone)
          const uint32_t hb = __float_as_uint(h);
          const bool fin = fabsf(h) <= FLT_MAX;
          const float r1 = fin ? h - __uint_as_float(hb & 0xffff0000u) : 0.f;
          const uint32_t mb = __float_as_uint(r1);
          const float r2 = r1 - __uint_as_float(mb & 0xffff0000u);
          const int ch = c0 + c;
          uint16_t* o = a.h + ((size_t)pair * (a.ldh / 32) + ch / 32) * 96 + ch % 32;
          o[0] = (h == h) ? (uint16_t)(hb >> 16) : (uint16_t)0x7fc0u;
          o[32] = (uint16_t)(mb >> 16);
          o[64] = (uint16_t)(__float_as_uint(r2) >> 16);
        }
      }
      buf ^= 1;  // the team's next tile uses the other half: one barrier a tile is enough
    }
  }
  at.back((i - count) * chunks.n, a.stages);
  if (!whole) turn = (turn + count) % kFewTeams;
}

// ---------------------------------------------------------------- down
// CTA b owns the output rows [b H / grid, (b + 1) H / grid), a.rows (at most 32) in a pass.
__device__ __forceinline__ int row_begin(const FewArgs& a, int b) { return (int)((int64_t)b * a.H / gridDim.x); }

// Small experts come a.group to a stage, in order; the last stage may hold fewer.
__device__ __forceinline__ int group_size(const FewArgs& a, const FewShared& S, int s) { return min(a.group, S.n_act - s); }

template <int FMT>
__device__ void feed_down(Feeder& f, const FewMaps& m) {
  const FewArgs& a = f.a;
  const int n1 = row_begin(a, blockIdx.x + 1);
  for (int r0 = row_begin(a, blockIdx.x); r0 < n1; r0 += a.rows) {
    const int shared = a.rows * 64 * a.dn_s.cb, routed = a.rows * 64 * a.dn.cb, scales = FMT >= 0 ? a.rows * a.dn.sc : 0;
    for (int c = 0; c < a.dn_s.n; ++c) {
      uint8_t* dst = f.begin();
      if (!f.ok) return;
      uint64_t* bar = &f.S.full[f.cur.s];
      f.tag();
      ptx::mbar_arrive_expect_tx(bar, shared);
      tma_4d(dst, &m.dn_s, bar, 0, r0, c * a.dn_s.cb, 0);
      f.end();
    }
    for (int s = 1; s < f.S.n_act; s += a.group) {
      const int n = group_size(a, f.S, s);
      for (int c = 0; c < a.dn.n; ++c) {
        uint8_t* dst = f.begin();
        if (!f.ok) return;
        uint64_t* bar = &f.S.full[f.cur.s];
        f.tag();
        ptx::mbar_arrive_expect_tx(bar, n * (routed + scales));
        for (int j = 0; j < n; ++j, dst += a.slot) {
          const int e = f.S.act_e[s + j];
          tma_4d(dst, &m.dn, bar, 0, r0, c * a.dn.cb, e);
          if (FMT >= 0) tma_3d(dst + round128(routed), &m.dn_sc, bar, a.dn.scale_at(c, a.shift) & ~15, r0, e);
        }
        f.end();
      }
    }
  }
}

// h for the same stages, once all of it is there.
template <int FMT>
__device__ void feed_h(Feeder& f, uint8_t* units) {
  const FewArgs& a = f.a;
  FewShared& S = f.S;
  const int n1 = row_begin(a, blockIdx.x + 1);
  // A CTA without output rows (H < grid) does not wait: its consumers leave without h, and the last one
  // to leave sets the counter back to zero, which this thread, still looking, would wait for in vain.
  // Where there are rows, the consumers leave after this thread has brought them h.
  if (row_begin(a, blockIdx.x) == n1 || !f.ok) return;
  grid_wait(a.sync + 1, S, a.status);
  asm volatile("fence.proxy.async;" ::: "memory");
  Cursor done = f.cur;  // the oldest stage whose units are not known to be free
  int flight = 0, in_use = 0, at = 0;
  auto pop = [&] {
    in_use -= S.stage_units[done.s];
    done.next(a.stages);
    --flight;
  };
  for (int r0 = row_begin(a, blockIdx.x); r0 < n1; r0 += a.rows)
    for (int s = 0, next; s < S.n_act; s = next) {
      const FewChunks& ch = s ? a.dn : a.dn_s;
      next = s ? s + group_size(a, S, s) : 1;
      const int first = s ? S.act_pair[s] : 0, tokens = s ? S.act_pair[next] - first : a.T;
      const int block = FMT >= 0 && s ? 768 : 192, total = 6 * (s ? a.I : a.Is);
      // the group's pairs follow one another
      const uint8_t* src = reinterpret_cast<const uint8_t*>(a.h) + (size_t)first * a.ldh * 6;
      for (int c = 0; c < ch.n; ++c) {
        f.begin();
        if (f.ok && flight == a.stages) pop();  // it was in this place
        while (f.ok && in_use + tokens > a.units) {
          f.ok = wait_phase(&S.empty[done.s], done.parity, S, a.status);
          pop();
        }
        if (!f.ok) return;
        const int from = c * ch.cb * block, n = min(ch.cb * block, total - from);
        uint64_t* bar = &f.S.full[f.cur.s];
        ptx::mbar_arrive_expect_tx(bar, tokens * n);
        for (int q = 0; q < tokens; ++q) {
          bulk_load(units + (size_t)at * a.unit, src + (size_t)q * a.ldh * 6 + from, n, bar);
          if (++at == a.units) at = 0;
        }
        S.stage_units[f.cur.s] = (uint8_t)tokens;
        in_use += tokens;
        ++flight;
        f.end();
      }
    }
}

// W_down times h of an expert's tokens, for the blocks wt, wt + step, ... of a stage. The three
// pieces of h of a token are three columns of the MMA. A warp adds its sums to its own
// S.out[warp][row][token]; `open` multiplies them (the shared expert's gate).
//
// bf16 weights: mma_rows, N tokens (the lowest of `mask`) at a time, their units from `unit` on.
template <int NI, int N>
__device__ __forceinline__ void down_bf16(const FewArgs& a, FewShared& S, uint32_t st, uint32_t units, int unit,
                                          uint32_t mask, int nb, int nr, int wt, int step, bool gated, int warp,
                                          int lane) {
  const int g = lane >> 2, t4 = lane & 3, piece = (g & 3) < 3;
  const bool low = g < 4;
  // rows behind the pass read its last one: only the last tile can have any
  const uint32_t row = 64 * g + 16 * t4, last = 64 * min(8 * (NI - 1) + g, nr - 1) + 16 * t4;
  uint32_t wp = st + 64 * wt * a.rows, hu[N];
  uint4 x[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    int u = unit + n;
    if (u >= a.units) u -= a.units;
    hu[n] = units + u * a.unit + 64 * (g & 3) + 16 * t4 + wt * 192;
    x[n] = make_uint4(0u, 0u, 0u, 0u);
  }
  float sum[N][NI][4] = {};
#pragma unroll 2
  for (int b = wt; b < nb; b += step, wp += 64 * step * a.rows) {
    uint2 y[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      lds_v4_if(x[n], hu[n], piece);
      y[n] = make_uint2(low ? x[n].x : x[n].y, low ? x[n].z : x[n].w);
      hu[n] += 192 * step;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const uint4 w = lds_v4(wp + (i < NI - 1 ? row + 512 * i : last));
#pragma unroll
      for (int n = 0; n < N; ++n) mma_rows(sum[n][i], w, y[n]);
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int token = __ffs(mask) - 1;
    mask &= mask - 1;
    const float open = gated ? S.sgate[token] : 1.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float v0, v1;
      fold(sum[n][i], t4 < 2, v0, v1);
      // lane 0 has the first two pieces' sums, lane 1 the third's. An infinite weight gives the first
      // its infinity or NaN, and the others NaN where h ends before them.
      const float third = __shfl_xor_sync(0xffffffffu, v0, 1), v = fabsf(v0) <= FLT_MAX ? v0 + v1 + third : v0;
      if (t4 == 0) S.out[warp][8 * i + g][token] += open * v;
    }
  }
}

// 4-bit weights: the MMA's A is 16 rows, its columns 0-2 and 4-6 are one or two tokens' pieces.
template <int FMT, int NI>
__device__ __forceinline__ void down_w4(const FewArgs& a, FewShared& S, const FewChunks& ch, uint32_t st,
                                        uint32_t units, int unit, uint32_t mask, int c, int nb, int nr, int wt,
                                        int step, int warp, int lane) {
  const int g = lane >> 2, t4 = lane & 3, K = a.I, b0 = c * ch.cb;
  const bool two = mask & (mask - 1);
  const int piece = (g & 3) < 3 && (g < 4 || two);
  int u = unit + (g >> 2);
  if (u >= a.units) u -= a.units;
  uint32_t hu = units + u * a.unit + 64 * (g & 3) + 16 * t4 + wt * 768;
  uint32_t wp = st + 64 * wt * a.rows + 16 * t4;
  const uint32_t sp = st + round128(a.rows * 64 * ch.cb) + (ch.scale_at(c, FMT) & 15);
  constexpr int NP = (NI + 1) / 2;  // an odd last tile is both halves of its MMA, the second for nothing
  uint32_t row[NI];                 // rows behind the pass read its last one
#pragma unroll
  for (int i = 0; i < NI; ++i) row[i] = min(8 * i + g, nr - 1);
  uint4 x[4] = {};
  float sum[NP][4] = {};
  for (int b = wt; b < nb; b += step, wp += 64 * step * a.rows, hu += 768 * step) {
    const bool half = K / 32 - 4 * (b0 + b) == 2;  // K is a multiple of 64: four parts or two
    uint4 w[NI];
    uint2 sc[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      w[i] = lds_v4(wp + 64 * row[i]);
      sc[i] = w4_block_scales<FMT>(sp + row[i] * ch.sc, b);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) lds_v4_if(x[j], hu + 192 * j, piece && (j < 2 || !half));
    if (half) {
#pragma unroll
      for (int i = 0; i < NI; ++i) w4_half<FMT>(x, sc[i], sc[i]);
    }
    float d[NP][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const bool both = 2 * p + 1 < NI;
        const int p8 = both ? 2 * p + 1 : 2 * p;
        const uint4 v = w4_pairs<false>(word(w[2 * p], j)), v8 = both ? w4_pairs<false>(word(w[p8], j)) : v;
        // the parts of a group share a chain and a scale
        if (j % (1 << FMT) == 0) mma16816_first<false>(d[p], v.x, v8.x, v.y, v8.y, x[j].x, x[j].y);
        else mma16816<false>(d[p], v.x, v8.x, v.y, v8.y, x[j].x, x[j].y);
        mma16816<false>(d[p], v.z, v8.z, v.w, v8.w, x[j].z, x[j].w);
        if ((j + 1) % (1 << FMT) == 0) {
          const float f = w4_scale(sc[2 * p], j);
          sum[p][0] = fmaf(d[p][0], f, sum[p][0]);
          sum[p][1] = fmaf(d[p][1], f, sum[p][1]);
          if (both) {
            const float f8 = w4_scale(sc[p8], j);
            sum[p][2] = fmaf(d[p][2], f8, sum[p][2]);
            sum[p][3] = fmaf(d[p][3], f8, sum[p][3]);
          }
        }
      }
    }
  }
  // lanes t = 0, 1: the first token's pieces 0 and 1, and 2; t = 2, 3: the second's
  const int token = t4 < 2 ? __ffs(mask) - 1 : __ffs(mask & (mask - 1)) - 1;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    float v = sum[i / 2][2 * (i % 2)] + (t4 & 1 ? 0.f : sum[i / 2][2 * (i % 2) + 1]);
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    if (t4 == 0 || (t4 == 2 && two)) S.out[warp][8 * i + g][token] += kW4Unit<false> * v;
  }
}

// One expert's share of a stage: warps wt, wt + 1, ... of `step` take its blocks in turn.
template <int FMT, int NI>
__device__ __forceinline__ void down_stage(const FewArgs& a, FewShared& S, const FewChunks& ch, uint32_t st,
                                           uint32_t units, int unit, uint32_t mask, int c, bool gated, int nr,
                                           int wt, int step, int warp, int lane) {
  const int nb = min(ch.cb, ch.blocks - c * ch.cb);
  for (uint32_t left = mask; left;) {  // two tokens at a time
    if constexpr (FMT >= 0)
      down_w4<FMT, NI>(a, S, ch, st, units, unit, left, c, nb, nr, wt, step, warp, lane);
    else if (left & (left - 1))
      down_bf16<NI, 2>(a, S, st, units, unit, left, nb, nr, wt, step, gated, warp, lane);
    else
      down_bf16<NI, 1>(a, S, st, units, unit, left, nb, nr, wt, step, gated, warp, lane);
    left &= left - 1;
    left &= left - 1;
    unit += 2;
    if (unit >= a.units) unit -= a.units;
  }
}

// One pass of NI row tiles. The teams take the stages in turn (`turn`: the team of the pass's first one,
// `unit`: its first unit of h), and the warps of a team share each of a stage's experts.
template <int FMT, int NI>
__device__ __forceinline__ void down_pass(const FewArgs& a, FewShared& S, uint32_t ring, Place& at, int& turn,
                                          uint32_t units, int& unit, int nr, int warp, int lane) {
  const int team = warp / kFewTeam, wt = warp & (kFewTeam - 1);
  for (int i = lane; i < kFewRows * kFewMaxT; i += 32) (&S.out[warp][0][0])[i] = 0.f;
  __syncwarp();
  const int share = kFewTeam / a.group, mine = wt / share;  // warps of an expert; this warp's expert of a group
  const int groups = (S.n_act - 1 + a.group - 1) / a.group, end = a.dn_s.n + groups * a.dn.n;
  const int first = team >= turn ? team - turn : team - turn + kFewTeams;
  const int routed = unit + a.dn_s.n * a.T, pairs = S.act_pair[S.n_act] - a.T;
  auto wrap = [&](int u) { return u < a.units ? u : u % a.units; };
  auto release = [&] {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.empty[at.cur.s]);
  };
  int j = first;
  at.skip(first, a.stages);
  for (; j < a.dn_s.n; j += kFewTeams, at.skip(kFewTeams, a.stages)) {
    wait_stage(at, S, a.status);
    down_stage<-1, NI>(a, S, a.dn_s, ring + at.cur.s * a.stage_bytes, units, wrap(unit + j * a.T), (1u << a.T) - 1u, j,
                       true, nr, wt, kFewTeam, warp, lane);
    release();
  }
  int s = 1, c = j - a.dn_s.n;  // the group's first expert, chunk
  for (; j < end; j += kFewTeams, c += kFewTeams, at.skip(kFewTeams, a.stages)) {
    for (; c >= a.dn.n; c -= a.dn.n) s += a.group;
    // chunk by chunk, a group's units follow one another as its pairs do
    const int e = s + mine, base = S.act_pair[s], n = S.act_pair[min(s + a.group, S.n_act)] - base;
    const int mask = e < S.n_act ? S.act_mask[e] : 0;
    const int u = wrap(routed + (base - a.T) * a.dn.n + c * n + (mask ? S.act_pair[e] - base : 0));
    wait_stage(at, S, a.status);
    down_stage<FMT, NI>(a, S, a.dn, ring + at.cur.s * a.stage_bytes + mine * a.slot, units, u, mask, c, false, nr,
                        wt & (share - 1), share, warp, lane);
    release();
  }
  at.back(j - end, a.stages);  // to the first stage of the next pass
  turn = (turn + end) % kFewTeams;
  unit = wrap(routed + pairs * a.dn.n);
}

template <int FMT>
__device__ void down_rows(const FewArgs& a, FewShared& S, uint32_t ring, Place& at, int& turn, uint32_t units) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n1 = row_begin(a, blockIdx.x + 1);
  int unit = 0;
  for (int r0 = row_begin(a, blockIdx.x); r0 < n1; r0 += a.rows) {
    const int nr = min(a.rows, n1 - r0);
    if (nr > 24) down_pass<FMT, 4>(a, S, ring, at, turn, units, unit, nr, warp, lane);
    else if (nr > 16) down_pass<FMT, 3>(a, S, ring, at, turn, units, unit, nr, warp, lane);
    else if (nr > 8) down_pass<FMT, 2>(a, S, ring, at, turn, units, unit, nr, warp, lane);
    else down_pass<FMT, 1>(a, S, ring, at, turn, units, unit, nr, warp, lane);
    sync_consumers();
    const int r = tid % kFewRows, t = tid / kFewRows;
    if (t < a.T && r < nr) {
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < kFewWarps; ++w) sum += S.out[w][r][t];
      a.out[(size_t)t * a.H + r0 + r] = sum;
    }
    if (r0 + a.rows < n1) sync_consumers();  // S.out is read
  }
}

// ---------------------------------------------------------------- router
// The CTA's rows [e0, e1) of the router matrix (row E: the shared expert's gate vector, bf16), the
// first stages of the ring: a stage is a row's next stage_bytes / 4 elements.
struct RouterRows {
  int e0, e1, chunk, n;
};
__device__ __forceinline__ RouterRows router_rows(const FewArgs& a) {
  RouterRows r;
  r.e0 = (int)((int64_t)blockIdx.x * (a.E + 1) / gridDim.x);
  r.e1 = (int)((int64_t)(blockIdx.x + 1) * (a.E + 1) / gridDim.x);
  r.chunk = a.stage_bytes / 4;
  r.n = (a.H + r.chunk - 1) / r.chunk;
  return r;
}

__device__ void feed_router(Feeder& f, uint8_t* xs, int xpitch, bool h) {
  const FewArgs& a = f.a;
  if (!h) {
    ptx::mbar_arrive_expect_tx(&f.S.x_full, 2 * a.T * a.H);
    for (int t = 0; t < a.T; ++t) bulk_load(xs + (size_t)t * xpitch, a.x + (size_t)t * a.H, 2 * a.H, &f.S.x_full);
  }
  const RouterRows r = router_rows(a);
  for (int e = r.e0; e < r.e1; ++e)
    for (int c = 0; c < r.n; ++c) {
      uint8_t* dst = f.begin();
      if (!f.ok) return;
      uint64_t* bar = &f.S.full[f.cur.s];
      if (h) {
        ptx::mbar_arrive(bar);
      } else {
        const int k = c * r.chunk, n = min(r.chunk, a.H - k);
        const bool gate = e == a.E;
        const void* src = gate ? static_cast<const void*>(a.wsg + k) : a.w_router + (size_t)e * a.H + k;
        f.tag();
        ptx::mbar_arrive_expect_tx(bar, n * (gate ? 2 : 4));
        bulk_load(dst, src, n * (gate ? 2 : 4), bar);
      }
      f.end();
    }
}

// Sums of N values a lane over the warp by recursive halving: lane l gets value l >> (5 - log2 N).
template <int N>
__device__ __forceinline__ double warp_sums(double (&v)[N], int lane) {
  int off = 16;
#pragma unroll
  for (int n = N / 2; n >= 1; n /= 2, off /= 2) {
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const double send = upper ? v[j] : v[j + n], keep = upper ? v[j + n] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, off);
    }
  }
  for (; off >= 1; off /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
  return v[0];
}

// Logits, in 64 bits: a team takes a stage, a thread four elements at a time. TT: tokens, rounded
// up to a power of two.
template <int TT>
__device__ __forceinline__ void router_logits(const FewArgs& a, FewShared& S, const uint8_t* xs, int xpitch,
                                              const uint8_t* ring, Place& at) {
  constexpr int log_t = TT == 1 ? 0 : TT == 2 ? 1 : TT == 4 ? 2 : 3;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, in_team = tid & (32 * kFewTeam - 1);
  const RouterRows r = router_rows(a);
  const int end = (r.e1 - r.e0) * r.n;
  const int my_e = r.e0 + tid / a.T, my_t = tid % a.T;  // the logit that this thread adds up
  const bool mine = my_e < r.e1;
  const float bias = mine && my_e < a.E && a.bias ? __ldg(a.bias + my_e) : 0.f;
  wait_phase(&S.x_full, 0u, S, a.status);
  Place mine_at = at;
  for (mine_at.skip(warp / kFewTeam, a.stages); mine_at.i < end; mine_at.skip(kFewTeams, a.stages)) {
    const uint8_t* st = ring + (size_t)mine_at.cur.s * a.stage_bytes;
    const int c = mine_at.i % r.n, k0 = c * r.chunk, n = min(r.chunk, a.H - k0);
    const bool gate = r.e0 + mine_at.i / r.n == a.E;
    double acc[TT] = {};
    wait_stage(mine_at, S, a.status);
    for (int k = 4 * in_team; k < n; k += 128 * kFewTeam) {
      float w[4];
      if (gate) {
        const uint2 v = *reinterpret_cast<const uint2*>(st + 2 * k);
        w[0] = bf16lo(v.x); w[1] = bf16hi(v.x); w[2] = bf16lo(v.y); w[3] = bf16hi(v.y);
      } else {
        const float4 v = *reinterpret_cast<const float4*>(st + 4 * k);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
      }
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < a.T) {
          const uint2 v = *reinterpret_cast<const uint2*>(xs + (size_t)t * xpitch + 2 * (k0 + k));
          acc[t] = fma((double)w[0], (double)bf16lo(v.x), acc[t]);
          acc[t] = fma((double)w[1], (double)bf16hi(v.x), acc[t]);
          acc[t] = fma((double)w[2], (double)bf16lo(v.y), acc[t]);
          acc[t] = fma((double)w[3], (double)bf16hi(v.y), acc[t]);
        }
    }
    const double v = warp_sums<TT>(acc, lane);
    const int t = lane >> (5 - log_t);
    if ((lane & ((32 >> log_t) - 1)) == 0 && t < a.T)
      S.part[(mine_at.i * kFewTeam + (warp & (kFewTeam - 1))) * a.T + t] = v;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&S.empty[mine_at.cur.s]);
  }
  at.skip(end, a.stages);
  sync_consumers();
  if (mine) {
    double l = 0.0;
    for (int c = 0; c < r.n; ++c)
#pragma unroll
      for (int w = 0; w < kFewTeam; ++w)
        l += S.part[(((my_e - r.e0) * r.n + c) * kFewTeam + w) * a.T + my_t];
    a.logits[(size_t)my_t * a.ldl + my_e] = l + (double)bias;
    asm volatile("fence.proxy.async.global;" ::: "memory");  // read by bulk copies
  }
}

// ---------------------------------------------------------------- the kernel
// All logits are there: every CTA chooses the experts of all tokens for itself. The ring holds
// nothing now (the feeders wait for the experts) and takes the logits.
__device__ void route(const FewArgs& a, FewShared& S, uint8_t* ring, int warp, int lane) {
  sync_consumers();  // the last tile's sums are read: S.cand shares their place
  if (threadIdx.x == 0) {
    grid_wait(a.sync, S, a.status);
    asm volatile("fence.proxy.async;" ::: "memory");
    ptx::mbar_arrive_expect_tx(&S.logits_full, 8 * a.T * a.ldl);
    bulk_load(ring, a.logits, 8 * a.T * a.ldl, &S.logits_full);
  }
  wait_phase(&S.logits_full, 0u, S, a.status);
  const double* row = reinterpret_cast<const double*>(ring);
  if (threadIdx.x >= kFewThreads - 32 && lane < a.T)
    S.sgate[lane] = 1.f / (1.f + expf(-(float)row[lane * a.ldl + a.E]));
  if (warp < a.T) {
    row += warp * a.ldl;
    if (a.E <= 64) select_token<2>(a, S, row, warp, lane);
    else if (a.E <= 512) select_token<16>(a, S, row, warp, lane);
    else select_token<32>(a, S, row, warp, lane);
  }
  sync_consumers();
  build_active(a, S);
}

template <int FMT>
__device__ void consume(const FewArgs& a, FewShared& S, uint8_t* xs, int xpitch, uint8_t* ring) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Place at{0, {0, 0u}};
  int turn = 0;  // the team that takes the next tile or stage
  for (int e = tid; e < a.E; e += kFewThreads) S.mask[e] = 0;
  if (tid < kFewMaxT) S.sgate[tid] = 0.f;
  if (a.T == 1) router_logits<1>(a, S, xs, xpitch, ring, at);
  else if (a.T <= 4) router_logits<4>(a, S, xs, xpitch, ring, at);
  else router_logits<8>(a, S, xs, xpitch, ring, at);
  grid_arrive(a.sync);

  const uint32_t xs_at = ptx::smem_u32(xs), ring_at = ptx::smem_u32(ring);
  // tiles b, b + grid, ...: of the shared expert (they need no routing), then of the chosen ones; bf16:
  // by the same code, which is warm by then
  const int grid = gridDim.x;
  int first = blockIdx.x, tiles = a.Is / 8;
  for (int pass = 0; pass < 2; ++pass) {
    if (pass) {
      route(a, S, ring, warp, lane);
      tiles = (S.n_act - 1) * (a.I / 8);
    }
    const int count = max((tiles - first + grid - 1) / grid, 0);
    auto run = [&](auto fmt) {
      constexpr int F = decltype(fmt)::value;
      if (a.T <= 4) gate_up_tiles<F, 1>(a, S, xs_at, xpitch, ring_at, at, pass, first, count, turn);
      else gate_up_tiles<F, 2>(a, S, xs_at, xpitch, ring_at, at, pass, first, count, turn);
    };
    if (FMT >= 0 && pass) run(std::integral_constant<int, FMT>{});
    else run(std::integral_constant<int, -1>{});
    first += count * grid - tiles;
  }

  // h of this CTA is written (for bulk copies to read); that of the others comes through the ring
  asm volatile("fence.proxy.async.global;" ::: "memory");
  grid_arrive(a.sync + 1);
  turn = 0;
  down_rows<FMT>(a, S, ring_at, at, turn, xs_at);

  // the last CTA to leave makes the counters ready for the next call
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(a.sync + 2, 1u) + 1 == gridDim.x) {
      a.sync[0] = 0;
      a.sync[1] = 0;
      a.sync[2] = 0;
    }
  }
}

// The warp behind the consumers feeds weights, the last one h; one thread of each.
template <int FMT>
__device__ void feed(const FewArgs& a, const FewMaps& m, FewShared& S, uint8_t* ring, uint8_t* xs, int xpitch) {
  const int lane = threadIdx.x & 31;
  const bool h = threadIdx.x >= kFewThreads + 32;
  Feeder f{a, S, ring, Cursor{0, 0u}, 0, true};
  Tiles tile;
  tile.begin();
  const int ns = a.Is / 8;
  if (lane == 0) {
    feed_router(f, xs, xpitch, h);
    feed_gate_up<FMT>(f, m, h, tile, ns);
    atomicAdd(&S.parked, 1);
  }
  __syncwarp();
  ptx::bar_sync(kBarRouted, kFewBlock);
  if (lane != 0) return;
  // a consumer that has run out and seen this feeder parked is seen here
  atomicSub(&S.parked, 1);
  __threadfence_block();
  if (*reinterpret_cast<volatile int*>(&S.aborted)) f.ok = false;
  feed_gate_up<FMT>(f, m, h, tile, ns + (S.n_act - 1) * (a.I / 8));
  if (h) feed_h<FMT>(f, xs);
  else feed_down<FMT>(f, m);
  atomicAdd(&S.parked, 1);
  f.drain();
}

template <int FMT>
__global__ void __launch_bounds__(kFewBlock, 1)
few_layer_kernel(const __grid_constant__ FewArgs a, const __grid_constant__ FewMaps m) {
  extern __shared__ __align__(128) uint8_t smem[];
  FewShared& S = *reinterpret_cast<FewShared*>(smem);
  uint8_t* xs = smem + kFewSharedBytes;  // x, then the units of h
  const int xpitch = 2 * a.H + 64;  // 64 mod 128: two tokens' 64-byte reads share no bank
  uint8_t* ring = xs + a.h_bytes;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      ptx::mbar_init(&S.full[i], 2);
      ptx::mbar_init(&S.empty[i], kFewTeam);
    }
    ptx::mbar_init(&S.x_full, 1);
    ptx::mbar_init(&S.logits_full, 1);
    for (int i = 0; i < a.stages; ++i) S.tag[i] = -1;
    S.aborted = S.parked = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x < kFewThreads) consume<FMT>(a, S, xs, xpitch, ring);
  else feed<FMT>(a, m, S, ring, xs, xpitch);
}

// Chunks of a row of K weights for stages of `stage` bytes with `rows` rows, at most `limit` blocks.
FewChunks few_chunks(int K, int rows, bool w4, int shift, int stage, int limit) {
  FewChunks c;
  c.blocks = w4 ? (int)w4_blocks(K) : K / 32;
  const int per = rows * (64 + (w4 ? 8 >> shift : 0));
  const int most = std::min((stage - 128 - (w4 ? 32 * rows : 0)) / per, limit);
  c.n = (c.blocks + most - 1) / most;
  c.cb = (c.blocks + c.n - 1) / c.n;
  c.n = (c.blocks + c.cb - 1) / c.cb;
  if (w4) {  // a box starts on 16 bytes of a row's scales: chunks that do not bring some more
    const int bytes = c.cb * 8 >> shift;
    c.sc = (bytes + 15) / 16 * 16 + (c.n > 1 && bytes % 16 ? 16 : 0);
  } else {
    c.sc = 0;
  }
  return c;
}

// The geometry of a call on `sms` SMs into `a` (shift: of the 4-bit experts, -1 for bf16); false if the kernel's
// fixed capacities do not hold it. 148 SMs hold every shape within the stated limits; a part of a device may not.
bool few_plan(const moe_shape& s, int shift, int sms, FewArgs& a) {
  const bool w4 = shift >= 0;
  a.shift = w4 ? shift : 0;
  a.ldl = (s.E + 2) / 2 * 2;
  a.T = s.T; a.H = s.H; a.E = s.E; a.k = s.k; a.I = s.I; a.Is = s.Is;
  const int cap = kFewRows;
  const int most_rows = (s.H + sms - 1) / sms, passes = (most_rows + cap - 1) / cap;
  a.rows = (most_rows + passes - 1) / passes;
  const int x_bytes = s.T * (2 * s.H + 64);
  // Six stages of 24 KB; where x leaves less room, smaller ones, below 15 KB fewer of them: a stage costs
  // its team some 700 clocks besides its weights. (8 tokens of H = 8192, I = 2048, 4-bit weights: six
  // stages of 12 KB 484 us, four of 18 KB 433 us, three of 24 KB 450 us.)
  const int most_bytes = 24576, least_bytes = 15360;
  for (a.stages = 6;; --a.stages) {
    for (a.stage_bytes = most_bytes;; a.stage_bytes -= 1024) {
      a.gu_s = few_chunks(s.H, 16, false, 0, a.stage_bytes, 32);
      a.gu = few_chunks(s.H, 16, w4, a.shift, a.stage_bytes, 32);
      // the limit keeps a unit of h near 6 KB
      a.dn_s = few_chunks(s.Is, a.rows, false, 0, a.stage_bytes, 32);
      a.dn = few_chunks(s.I, a.rows, w4, a.shift, a.stage_bytes, w4 ? 8 : 32);
      // 64 mod 128 bytes (banks), more of them than one stage can need
      a.unit = std::max(a.dn_s.cb * 192, a.dn.cb * (w4 ? 768 : 192)) | 64;
      a.h_bytes = (std::max(x_bytes, (s.T + 4) * a.unit) + 127) / 128 * 128;
      if (kFewSharedBytes + a.h_bytes + (size_t)a.stages * a.stage_bytes <= kFewSmem) break;
      if (a.stage_bytes <= least_bytes) break;
    }
    if (kFewSharedBytes + a.h_bytes + (size_t)a.stages * a.stage_bytes <= kFewSmem) break;
    if (a.stages <= 3) return false;
  }
  // what is left holds more units of h: several groups of experts in flight
  a.h_bytes = ((int)kFewSmem - (int)kFewSharedBytes - a.stages * a.stage_bytes) / 128 * 128;
  a.units = std::min(a.h_bytes / a.unit, 64);
  a.slot = (a.rows * 64 * a.dn.cb + 127) / 128 * 128 + (a.rows * a.dn.sc + 127) / 128 * 128;
  // experts of a stage: 1, 2 or 4, so that each has as many of the team's warps; bf16: and so few that a
  // warp's share of one is a chain of at most 8 instructions, as everywhere
  const int fit = std::min(a.stage_bytes / a.slot, a.units / s.T);
  a.group = a.dn.n > 1 || fit < 2 ? 1 : fit < kFewTeam ? 2 : kFewTeam;
  while (!w4 && a.group * a.dn.cb > 8 * kFewTeam) a.group /= 2;
  // the router's share of a CTA: a place for each partial sum, a thread for each logit
  const int64_t rows = (s.E + 1 + sms - 1) / sms, chunks = (s.H + a.stage_bytes / 4 - 1) / (a.stage_bytes / 4);
  return rows * chunks * kFewTeam * s.T <= kFewParts && rows * s.T <= kFewThreads &&
         8 * s.T * a.ldl <= a.stages * a.stage_bytes;
}

bool few_map(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
             const uint32_t* box) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, ones,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [64][n][blocks][halves][E] of E matrices of halves * n rows of `row` bytes
bool few_weight_map(CUtensorMap* m, const void* base, uint64_t n, const FewChunks& c, uint64_t row, uint64_t halves,
                    uint64_t E, uint32_t box_rows) {
  const uint64_t dims[5] = {64, n, (uint64_t)c.blocks, halves, E};
  const uint64_t strides[4] = {row, 64, n * row, halves * n * row};
  const uint32_t box[5] = {64, box_rows, (uint32_t)c.cb, (uint32_t)halves, 1};
  if (halves > 1) return few_map(m, base, 5, dims, strides, box);
  const uint64_t d4[4] = {64, n, (uint64_t)c.blocks, E}, s4[3] = {row, 64, n * row};
  const uint32_t b4[4] = {64, box_rows, (uint32_t)c.cb, 1};
  return few_map(m, base, 4, d4, s4, b4);
}

// the same for the scales, [row][n][halves][E]
bool few_scale_map(CUtensorMap* m, const void* base, uint64_t n, const FewChunks& c, uint64_t row, uint64_t halves,
                   uint64_t E, uint32_t box_rows) {
  const uint64_t d4[4] = {row, n, halves, E}, s4[3] = {row, n * row, halves * n * row};
  const uint32_t b4[4] = {(uint32_t)c.sc, box_rows, (uint32_t)halves, 1};
  if (halves > 1) return few_map(m, base, 4, d4, s4, b4);
  const uint64_t d3[3] = {row, n, E}, s3[2] = {row, n * row};
  const uint32_t b3[3] = {(uint32_t)c.sc, box_rows, 1};
  return few_map(m, base, 3, d3, s3, b3);
}

int few_shift(const moe_w4_experts* q) { return !q ? -1 : q->group == 32 ? 0 : q->group == 64 ? 1 : 2; }

}  // namespace

bool few_supported(const moe_shape& s, const moe_w4_experts* q, int sms) {
  if (s.T > kFewMaxT || (int64_t)s.T * s.H > kFewMaxTH) return false;
  FewArgs a{};
  return s.T == 0 || few_plan(s, few_shift(q), sms, a);
}

cudaError_t launch_few_layer(const moe_shape& s, const Layout& L, char* ws, const uint16_t* x,
                             const moe_weights& w, const moe_w4_experts* q, float* out,
                             int32_t* ids, float* topk_w, float* gap, int sms, cudaStream_t st) {
  FewArgs a{};
  a.x = x;
  a.w_router = w.w_router;
  a.bias = w.router_bias;
  a.wsg = static_cast<const uint16_t*>(w.w_shared_gate);
  a.out = out;
  a.ids = ids;
  a.w = topk_w;
  a.gap = gap;
  a.logits = reinterpret_cast<double*>(ws + L.logits);
  a.h = reinterpret_cast<uint16_t*>(ws + L.few_h);
  a.ldh = L.ldh;
  a.sync = reinterpret_cast<uint32_t*>(ws + L.status) + kFewSyncWord;
  a.status = reinterpret_cast<uint32_t*>(ws + L.status);
  a.per_tile = (uint32_t)(((1ull << 32) + s.I / 8 - 1) / (s.I / 8));
  if (!few_plan(s, few_shift(q), sms, a)) return cudaErrorInvalidValue;

  FewMaps m;
  bool ok = few_weight_map(&m.gu_s, w.ws_gate_up, s.Is, a.gu_s, 2 * (uint64_t)s.H, 2, 1, 8) &&
            few_weight_map(&m.dn_s, w.ws_down, s.H, a.dn_s, 2 * (uint64_t)s.Is, 1, 1, a.rows);
  if (q) {
    const uint64_t gr = w4_row_bytes(s.H), dr = w4_row_bytes(s.I);
    const uint64_t gs = 2 * w4_row_scales(s.H, q->group), ds = 2 * w4_row_scales(s.I, q->group);
    ok = ok && few_weight_map(&m.gu, q->q_gate_up, s.I, a.gu, gr, 2, s.E, 8) &&
         few_weight_map(&m.dn, q->q_down, s.H, a.dn, dr, 1, s.E, a.rows) &&
         few_scale_map(&m.gu_sc, q->s_gate_up, s.I, a.gu, gs, 2, s.E, 8) &&
         few_scale_map(&m.dn_sc, q->s_down, s.H, a.dn, ds, 1, s.E, a.rows);
  } else {
    ok = ok && few_weight_map(&m.gu, w.w_gate_up, s.I, a.gu, 2 * (uint64_t)s.H, 2, s.E, 8) &&
         few_weight_map(&m.dn, w.w_down, s.H, a.dn, 2 * (uint64_t)s.I, 1, s.E, a.rows);
  }
  if (!ok) return cudaErrorInvalidValue;

  const size_t smem = kFewSharedBytes + a.h_bytes + (size_t)a.stages * a.stage_bytes;
  const void* fn = !q ? (const void*)few_layer_kernel<-1>
                   : a.shift == 0 ? (const void*)few_layer_kernel<0>
                   : a.shift == 1 ? (const void*)few_layer_kernel<1>
                                  : (const void*)few_layer_kernel<2>;
  static std::atomic<uint64_t> done[4];
  cudaError_t e = allow_smem(fn, kFewSmem, done[q ? a.shift : 3]);
  if (e != cudaSuccess) return e;
  LaunchScope scope(MOE_K_OTHER, st);
  void* params[] = {&a, &m};
  // cooperative: the CTAs wait for one another, so all of them have to be resident at once
  e = cudaLaunchCooperativeKernel(fn, dim3(sms), dim3(kFewBlock), params, smem, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

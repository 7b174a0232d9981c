// w4_matvec.cu -- y = x W^T for 1 to 16 rows of x and a 4-bit matrix (format: w4.cuh).
//
//   y[t, n] = sum_k x[t, k] (c[n, k] - 8) s[n, k / group]
//
// A group of warps takes 32 matrix rows (16 if there are few) and splits
// their 128-element blocks; the fewer rows there are, the more warps a group has, without a second
// launch. 16 warps in whole groups make a CTA, so 75 to 148 of 148 SMs have one unless the matrix is
// large (5000 rows of 2560: 79; 65536 rows: 128). The codes come two blocks ahead; x is
// staged in shared memory. The MMA's A is 16
// matrix rows, made in registers, its columns are 8 rows of x. The codes enter as exact
// integers; the fp32 sum over a scale group is multiplied by the scale and added to the running
// fp32 sums, so no product or weight is rounded.
//
// Measured on one B200, weights not in L2 (floor: their bytes at 6.56 TB/s): 1 row by 65536 x 8192,
// groups of 128, 73 us (42); 16 rows 107 us; 5 rows by 4099 x 2501 7 us on the device. Neither HBM nor
// the instructions are at their limit: 1 row 48 % of the DRAM rate and 2.4 of 4 instructions a clock (on the
// SMs that have a CTA; 19 for each MMA), 16 rows 31 % and 2.0 (12); four warps a scheduler, each with 64
// bytes of a row to a request, wait for the copies, for the pipe that unpacks, and for one another. 16 rows
// in groups of 32 or 64 spill some 40 bytes. A ring of three blocks a warp took 1 row from 85
// to 73 us against one block ahead in registers; it leaves x 128 KB, since x in twice as many chunks
// costs 16 rows 8 us.
#include <cuda_fp16.h>

#include <algorithm>

#include "moe_internal.h"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kMvWarps = 16;
constexpr int kMvThreads = kMvWarps * 32;
constexpr int kMvXBytes = 131072;  // staged x; what is longer comes in K chunks

struct MvArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* q;
  const uint16_t* s;
  void* y;
  int64_t ldy;
  int64_t N, K, groups;
  int64_t row_bytes, row_scales;
  int T, kc, split, y_f32;  // split: warps of a row group
};

// The codes come through a ring of kMvDepth blocks in shared memory, a warp's own: a lane copies the 16
// bytes of its rows 8 i + g that it reads itself, so its own waits are all there is to wait for.
constexpr int kMvDepth = 3;
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <bool F16, int SHIFT, int NT, int NP>
__device__ __forceinline__ void mv_block(const uint4 (&w)[2 * NP], const uint2 (&s)[2 * NP], uint32_t xp, int pitch,
                                         const int (&tok)[NT], float (&acc)[NP][NT][4]) {
  float d[NP][NT][4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4 x[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      x[n] = make_uint4(0u, 0u, 0u, 0u);
      lds_v4_if(x[n], xp + 8 * n * pitch + 64 * j, tok[n]);
    }
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      const uint4 v = w4_pairs<F16>(word(w[2 * p], j)), v8 = w4_pairs<F16>(word(w[2 * p + 1], j));
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        // the parts of a group share a chain and a scale
        if (j % (1 << SHIFT) == 0) mma16816_first<F16>(d[p][n], v.x, v8.x, v.y, v8.y, x[n].x, x[n].y);
        else mma16816<F16>(d[p][n], v.x, v8.x, v.y, v8.y, x[n].x, x[n].y);
        mma16816<F16>(d[p][n], v.z, v8.z, v.w, v8.w, x[n].z, x[n].w);
        if ((j + 1) % (1 << SHIFT) == 0) {
          const float f = w4_scale(s[2 * p], j), f8 = w4_scale(s[2 * p + 1], j);
          acc[p][n][0] = fmaf(d[p][n][0], f, acc[p][n][0]);
          acc[p][n][1] = fmaf(d[p][n][1], f, acc[p][n][1]);
          acc[p][n][2] = fmaf(d[p][n][2], f8, acc[p][n][2]);
          acc[p][n][3] = fmaf(d[p][n][3], f8, acc[p][n][3]);
        }
      }
    }
  }
}

template <bool F16>
__device__ __forceinline__ void mv_store(const MvArgs& a, int t, int64_t n, float v) {
  const int64_t at = t * a.ldy + n;
  if (a.y_f32) static_cast<float*>(a.y)[at] = v;
  else if constexpr (F16) static_cast<__half*>(a.y)[at] = __float2half_rn(v);
  else static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_rn(v);
}

template <bool F16, int SHIFT, int NT, int NP>
__global__ void __launch_bounds__(kMvThreads)
matvec_w4_kernel(const MvArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int pitch = 2 * a.kc + 64;  // 64 mod 128: two tokens' 64-byte reads share no bank
  constexpr int ring = kMvDepth * 2 * NP * 512;  // bytes of a warp
  uint8_t* behind = smem + (size_t)a.T * pitch;
  const uint32_t mine = (uint32_t)__cvta_generic_to_shared(behind) + warp * ring + 16 * lane;
  const uint32_t xs = (uint32_t)__cvta_generic_to_shared(smem) + g * pitch + 16 * t4;
  const int part = warp % a.split, per_cta = kMvWarps / a.split;
  int tok[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) tok[n] = 8 * n + g < a.T;

  for (int64_t first = (int64_t)blockIdx.x * per_cta; first < a.groups; first += (int64_t)gridDim.x * per_cta) {
    const int64_t group = first + warp / a.split;
    const int64_t r0 = min(group, a.groups - 1) * (16 * NP);
    const uint8_t* q = a.q + r0 * a.row_bytes + 16 * t4;
    const uint16_t* s = a.s + r0 * a.row_scales;
    int row[2 * NP];  // rows behind the last read it again
#pragma unroll
    for (int i = 0; i < 2 * NP; ++i) row[i] = (int)min((int64_t)(8 * i + g), a.N - 1 - r0);
    float acc[NP][NT][4] = {};
    for (int64_t k0 = 0; k0 < a.K; k0 += a.kc) {
      const int kn = (int)min((int64_t)a.kc, a.K - k0);
      const int nb = (int)w4_blocks(kn);
      const int64_t b0 = k0 / kW4Block;
      const bool work = group < a.groups;
      uint2 sc[2 * NP], sn[2 * NP];  // scales, a block ahead
      auto fetch = [&](int b, int slot) {  // (a group without copies where there is no such block)
        if (work && b < nb)
#pragma unroll
          for (int i = 0; i < 2 * NP; ++i)
            copy16(mine + (slot * 2 * NP + i) * 512, q + row[i] * a.row_bytes + (b0 + b) * kW4BlockBytes);
        copy_commit();
      };
      auto fetch_scales = [&](int b) {
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) sn[i] = w4_block_scales(s + row[i] * a.row_scales, (int)(b0 + b), SHIFT);
      };
#pragma unroll
      for (int d = 0; d < kMvDepth - 1; ++d) fetch(part + d * a.split, d);
      if (work && part < nb) fetch_scales(part);
      if (a.kc < a.K || first == (int64_t)blockIdx.x * per_cta) {
        __syncthreads();  // every warp is done with the last chunk of x
        // x, zeros up to whole blocks; warp by warp, so that a thread's loads are all in flight
        const int cols = nb * kW4Block;
        const uint32_t x0 = (uint32_t)__cvta_generic_to_shared(smem);
        if (((reinterpret_cast<uintptr_t>(a.x) | (uint64_t)(2 * a.ldx)) & 15u) == 0 && kn % 8 == 0) {
          for (int t = 0; t < a.T; ++t) {
            const uint16_t* from = a.x + t * a.ldx + k0;
            for (int k = 8 * tid; k < cols; k += 8 * kMvThreads)
              copy16_or_zero(x0 + t * pitch + 2 * k, from + (k < kn ? k : 0), k < kn);
          }
          copy_commit();
          copy_wait<0>();
        } else {
          constexpr int batch = 8;
          for (int t = 0; t < a.T; ++t) {
            const uint16_t* from = a.x + t * a.ldx + k0;
            uint16_t* to = reinterpret_cast<uint16_t*>(smem + (size_t)t * pitch);
            for (int k = tid; k < cols; k += batch * kMvThreads) {
              uint16_t v[batch];
#pragma unroll
              for (int i = 0; i < batch; ++i)
                v[i] = k + i * kMvThreads < kn ? __ldg(from + k + i * kMvThreads) : (uint16_t)0;
#pragma unroll
              for (int i = 0; i < batch; ++i)
                if (k + i * kMvThreads < cols) to[k + i * kMvThreads] = v[i];
            }
          }
        }
        __syncthreads();
      }
      for (int b = part, slot = 0; b < nb; b += a.split, slot = (slot + 1) % kMvDepth) {
        fetch(b + (kMvDepth - 1) * a.split, (slot + kMvDepth - 1) % kMvDepth);
        copy_wait<kMvDepth - 1>();
        if (!work) continue;
        uint4 w[2 * NP];
#pragma unroll
        for (int i = 0; i < 2 * NP; ++i) {
          w[i] = lds_v4(mine + (slot * 2 * NP + i) * 512);
          sc[i] = sn[i];
        }
        if (b + a.split < nb) fetch_scales(b + a.split);
        mv_block<F16, SHIFT, NT, NP>(w, sc, xs + 256 * b, pitch, tok, acc);
      }
      copy_wait<0>();  // the next chunk starts with an empty ring
    }
    if (a.split == 1) {
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 8 * n + 2 * t4 + (i & 1);
            const int64_t row = r0 + 16 * p + 8 * (i >> 1) + g;
            if (group < a.groups && t < a.T && row < a.N) mv_store<F16>(a, t, row, acc[p][n][i] * kW4Unit<F16>);
          }
    } else {
      // the sums of a warp [row][NT * 8] take the place of its ring
      static_assert(16 * NP * 8 * NT * 4 <= ring, "");
      float* red = reinterpret_cast<float*>(behind + warp * ring);
#pragma unroll
      for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            *reinterpret_cast<float2*>(red + (16 * p + 8 * h + g) * (8 * NT) + 8 * n + 2 * t4) =
                make_float2(acc[p][n][2 * h], acc[p][n][2 * h + 1]);
      __syncthreads();
      const int rows = per_cta * 16 * NP;
      for (int o = tid; o < rows * a.T; o += kMvThreads) {
        const int t = o / rows, r = o - t * rows, w0 = r / (16 * NP) * a.split;
        const int64_t row = first * (16 * NP) + r;
        if (row >= a.N) continue;
        float v = 0.f;
        for (int w = 0; w < a.split; ++w)
          v += reinterpret_cast<const float*>(behind + (w0 + w) * ring)[r % (16 * NP) * (8 * NT) + t];
        mv_store<F16>(a, t, row, v * kW4Unit<F16>);
      }
      __syncthreads();  // red is read
    }
  }
}

template <bool F16, int SHIFT>
const void* mv_kernel(int nt, int np) {
  if (nt == 1) return np == 1 ? (const void*)matvec_w4_kernel<F16, SHIFT, 1, 1> : (const void*)matvec_w4_kernel<F16, SHIFT, 1, 2>;
  return np == 1 ? (const void*)matvec_w4_kernel<F16, SHIFT, 2, 1> : (const void*)matvec_w4_kernel<F16, SHIFT, 2, 2>;
}

}  // namespace

cudaError_t launch_matvec_w4(int T, int64_t N, int64_t K, int shift, const uint16_t* x, bool f16,
                             int64_t ldx, const uint8_t* q, const uint16_t* s, void* y, bool y_f32,
                             int64_t ldy, int sms, cudaStream_t st) {
  MvArgs a{x, ldx, q, s, y, ldy, N, K, 0, w4_row_bytes(K), w4_row_scales(K, 32 << shift), T, 0, 1, y_f32};
  const int nt = T > 8 ? 2 : 1;
  const int64_t most = kMvXBytes / (2 * T) / kW4Block * kW4Block;
  a.kc = (int)std::min(w4_blocks(K) * kW4Block, most);
  // 32 rows a group, 16 where that leaves SMs without one (32: 1 row by 65536 x 8192 73 us, 16: 84 us);
  // and so many warps a group (a power of two) that the
  // groups fill the device's warps once, fewer than two for a block
  const int np = N > (int64_t)sms * 32 ? 2 : 1;
  a.groups = (N + 16 * np - 1) / (16 * np);
  const int nb = (int)w4_blocks(a.kc);
  while (a.split < kMvWarps && a.split < nb && a.groups * a.split * 2 <= (int64_t)sms * kMvWarps) a.split *= 2;
  const int per_cta = kMvWarps / a.split;
  const int64_t ctas = (a.groups + per_cta - 1) / per_cta;
  const size_t smem = (size_t)T * (2 * a.kc + 64) + (size_t)kMvWarps * kMvDepth * 2 * np * 512;
  const void* fn = f16 ? (shift == 0 ? mv_kernel<true, 0>(nt, np) : shift == 1 ? mv_kernel<true, 1>(nt, np) : mv_kernel<true, 2>(nt, np))
                       : (shift == 0 ? mv_kernel<false, 0>(nt, np) : shift == 1 ? mv_kernel<false, 1>(nt, np) : mv_kernel<false, 2>(nt, np));
  static std::atomic<uint64_t> done[2][3][2][2];
  cudaError_t e = allow_smem(fn, 227 * 1024, done[f16][shift][nt - 1][np - 1]);
  if (e != cudaSuccess) return e;
  LaunchScope scope(MOE_K_OTHER, st);
  void* params[] = {&a};
  const unsigned grid = (unsigned)std::min<int64_t>(ctas, sms);
  e = cudaLaunchKernel(fn, dim3(grid), dim3(kMvThreads), params, smem, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

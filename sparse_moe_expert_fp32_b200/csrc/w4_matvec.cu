// w4_matvec.cu -- y = x W^T for 1 to 16 rows of x and a 4-bit matrix (format: w4.cuh).
//
//   y[t, n] = sum_k x[t, k] (c[n, k] - 8) s[n, k / group]
//
// Bound by the weight bytes, 1/2 + 2/group each. CTA b of the grid owns the matrix rows
// [b N / grid, (b + 1) N / grid) and takes them 32 at a time (four tiles of 8); its 16 warps
// split the row's 128-element blocks, so a CTA has no partner to wait for and small matrices
// still spread over all SMs. x is staged in shared memory once per K chunk. The codes enter
// the MMA as exact integers, a 32-element part at a time; its fp32 sum is multiplied by the
// part's scale and added to the running fp32 sums, so no product or weight is rounded.
#include <cuda_fp16.h>

#include <mutex>

#include "moe_internal.h"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kMvWarps = 16;
constexpr int kMvThreads = kMvWarps * 32;
constexpr int kMvRows = 32;
constexpr int kMvChunkRows = 512;  // most rows of a CTA when K is taken in chunks
constexpr int kMvXBytes = 131072;  // staged x, without the pitch's padding

struct MvArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* q;
  const uint16_t* s;
  void* y;
  int64_t ldy;
  int64_t N, K;
  int64_t row_bytes, row_scales;
  int T, shift, kc, y_f32;
};

template <bool F16, int NT>
__global__ void __launch_bounds__(kMvThreads)
matvec_w4_kernel(const MvArgs a) {
  extern __shared__ uint4 smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
  const int64_t n0 = blockIdx.x * a.N / gridDim.x, n1 = (blockIdx.x + 1) * a.N / gridDim.x;
  const int pitch = 2 * a.kc + 64;  // 64 mod 128: two tokens' 64-byte reads share no bank
  uint8_t* xs = reinterpret_cast<uint8_t*>(smem);
  float* red = reinterpret_cast<float*>(xs + (size_t)a.T * pitch);  // [warp][row][NT * 8]
  float* sums = red + kMvWarps * kMvRows * NT * 8;                  // [rows of the CTA][NT * 8], if K is chunked
  const bool chunked = a.K > a.kc;

  for (int64_t k0 = 0; k0 < a.K; k0 += a.kc) {
    const int kn = (int)min((int64_t)a.kc, a.K - k0);
    const int nb = (int)w4_blocks(kn);
    if (k0) __syncthreads();  // every warp is done with the last chunk of x
    for (int i = tid; i < a.T * nb * kW4Block; i += kMvThreads) {
      const int t = i / (nb * kW4Block), k = i - t * (nb * kW4Block);
      const uint16_t v = k < kn ? __ldg(a.x + t * a.ldx + k0 + k) : (uint16_t)0;
      *reinterpret_cast<uint16_t*>(xs + (size_t)t * pitch + 2 * k) = v;
    }
    __syncthreads();
    for (int64_t r0 = n0; r0 < n1; r0 += kMvRows) {
      const int nr = (int)min((int64_t)kMvRows, n1 - r0);
      float acc[4][4] = {};
      for (int b = warp; b < nb; b += kMvWarps) {
        const int64_t kb = k0 / kW4Block + b;
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          q[i] = ld_stream_v4(a.q + (r0 + min(g + 8 * i, nr - 1)) * a.row_bytes + kb * kW4BlockBytes + 16 * t4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (8 * i >= nr) break;
          const uint2 s0 = w4_block_scales(a.s + (r0 + min(8 * i + 2 * t4, nr - 1)) * a.row_scales, (int)kb, a.shift);
          const uint2 s1 = w4_block_scales(a.s + (r0 + min(8 * i + 2 * t4 + 1, nr - 1)) * a.row_scales, (int)kb, a.shift);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint8_t* xp = xs + (size_t)g * pitch + b * 256 + 64 * j + 16 * t4;
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            const uint4 x0 = g < a.T ? *reinterpret_cast<const uint4*>(xp) : zero;
            const uint4 x1 = g + 8 < a.T ? *reinterpret_cast<const uint4*>(xp + 8 * (size_t)pitch) : zero;
            float d[4];
            mma_cols<F16>(d, make_uint4(x0.x, x1.x, x0.y, x1.y), make_uint4(x0.z, x1.z, x0.w, x1.w),
                          w4_pairs<F16>((&q[i].x)[j]));
            acc[i][0] = fmaf(d[0], w4_scale(s0, j), acc[i][0]);
            acc[i][1] = fmaf(d[1], w4_scale(s1, j), acc[i][1]);
            acc[i][2] = fmaf(d[2], w4_scale(s0, j), acc[i][2]);
            acc[i][3] = fmaf(d[3], w4_scale(s1, j), acc[i][3]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (h == 0 || NT == 2) {
            float* at = red + ((size_t)warp * kMvRows + 8 * i + 2 * t4) * (NT * 8) + 8 * h + g;
            at[0] = acc[i][2 * h];
            at[NT * 8] = acc[i][2 * h + 1];
          }
      __syncthreads();
      for (int o = tid; o < kMvRows * NT * 8; o += kMvThreads) {
        const int r = o % kMvRows, t = o / kMvRows;
        if (r >= nr || t >= a.T) continue;
        float v = 0.f;
        for (int wi = 0; wi < kMvWarps; ++wi) v += red[((size_t)wi * kMvRows + r) * (NT * 8) + t];
        if (chunked) {
          float* at = sums + (size_t)(r0 - n0 + r) * (NT * 8) + t;
          if (k0) v += *at;
          *at = v;
        }
        if (k0 + a.kc >= a.K) {
          const int64_t at = t * a.ldy + r0 + r;
          if (a.y_f32) static_cast<float*>(a.y)[at] = v;
          else if constexpr (F16) static_cast<__half*>(a.y)[at] = __float2half_rn(v);
          else static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_rn(v);
        }
      }
      __syncthreads();
    }
  }
}

}  // namespace

cudaError_t launch_matvec_w4(int T, int64_t N, int64_t K, int shift, const uint16_t* x, bool f16,
                             int64_t ldx, const uint8_t* q, const uint16_t* s, void* y, bool y_f32,
                             int64_t ldy, int sms, cudaStream_t st) {
  MvArgs a{x, ldx, q, s, y, ldy, N, K, w4_row_bytes(K), w4_row_scales(K, 32 << shift), T, shift, 0, y_f32};
  const int nt = T > 8 ? 2 : 1;
  const int64_t most = kMvXBytes / (2 * T) / kW4Block * kW4Block;
  a.kc = (int)(w4_blocks(K) * kW4Block < most ? w4_blocks(K) * kW4Block : most);
  int64_t grid = N < sms ? N : sms;
  // a CTA keeps the sums of its rows in shared memory between K chunks
  if (K > a.kc && grid < (N + kMvChunkRows - 1) / kMvChunkRows) grid = (N + kMvChunkRows - 1) / kMvChunkRows;
  size_t smem = (size_t)T * (2 * a.kc + 64) + (size_t)kMvWarps * kMvRows * nt * 8 * sizeof(float);
  if (K > a.kc) smem += (size_t)((N + grid - 1) / grid) * nt * 8 * sizeof(float);
  if (smem > 227 * 1024) return cudaErrorInvalidValue;
  const void* kernels[2][2] = {
      {(const void*)matvec_w4_kernel<false, 1>, (const void*)matvec_w4_kernel<false, 2>},
      {(const void*)matvec_w4_kernel<true, 1>, (const void*)matvec_w4_kernel<true, 2>}};
  const void* fn = kernels[f16][nt - 1];
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024);
  if (e != cudaSuccess) return e;
  LaunchScope scope(MOE_K_OTHER, st);
  void* params[] = {&a};
  e = cudaLaunchKernel(fn, dim3((unsigned)grid), dim3(kMvThreads), params, smem, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe

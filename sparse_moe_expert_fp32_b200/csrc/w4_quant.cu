// w4_quant.cu -- the 4-bit weight pre-pass and its inverse (format: include/moe.h, w4.cuh).
//
//   scale = bf16(amax_group / 7)       code = clamp(round_half_even(w / scale), -8, 7) + 8
//
// Half a warp takes one storage block of 128 elements: lane 4 j + t reads elements
// 32 j + 8 t .. + 7 (16 bytes, in row order) and writes word 4 t + j, so a block is one
// 256-byte read and one 64-byte write, and a group's maximum is a shuffle over 4, 8 or 16
// lanes. Bound by HBM: 2 bytes read and 1/2 + 2/group written per weight.
//
// The quotient without a division: with 8-bit significands w / scale is either exactly half
// way between two integers or at least 2^-10 away from it (for |w / scale| >= 1/2 its
// distance is a nonzero multiple of 1/2 over twice an 8-bit integer). w times the rounded
// reciprocal is within 2^-20 of it (|w / scale| <= 7.1), so rounding the product to a
// multiple of 2^-12 first brings exact ties back and moves nothing else across a tie.
// Scales so small that the reciprocal leaves fp32's range divide instead.
#include "moe_internal.h"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;

// eight bf16 of a row at element e (zeros behind the row's end)
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int64_t e, int64_t K) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (VEC) {
    if (e < K) v = ld_stream_v4(row + e);
  } else {
    uint32_t* u = &v.x;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e + i < K) u[i >> 1] |= (uint32_t)__ldg(row + e + i) << (16 * (i & 1));
  }
  return v;
}

template <bool VEC>
__global__ void __launch_bounds__(kQuantThreads)
quantize_w4_kernel(const uint16_t* __restrict__ w, int64_t rows, int64_t K, int shift,
                   uint8_t* __restrict__ q, uint16_t* __restrict__ scales) {
  const int lane = threadIdx.x & 15, j = lane >> 2, t = lane & 3;
  const int64_t blocks = w4_blocks(K);
  const int64_t ns = w4_row_scales(K, 32 << shift);
  const int64_t vblocks = (ns << shift) >> 2;  // blocks with the scale padding's share, >= blocks
  const int64_t total = rows * vblocks;
  const int64_t stride = (int64_t)gridDim.x * (kQuantThreads / 16);
  const int lanes = 4 << shift;  // lanes of a group
  // every lane of a warp stays in the loop as long as one half has a block (the shuffles)
  for (int64_t v0 = (int64_t)blockIdx.x * (kQuantThreads / 16) + ((threadIdx.x >> 5) << 1); v0 < total;
       v0 += stride) {
    const int64_t vb = v0 + ((threadIdx.x >> 4) & 1);
    const bool in = vb < total;
    const int64_t row = in ? vb / vblocks : 0, b = in ? vb - row * vblocks : 0;
    const bool real = in && b < blocks;
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (real) v = load8<VEC>(w + row * K, b * kW4Block + 32 * j + 8 * t, K);
    // |w| as integers: infinities and NaN sort above every finite value
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                          __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    m = max(m & 0xffffu, m >> 16);
    for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    // a group with an infinity or a NaN gets a NaN scale, so that all of it reads back as NaN
    const uint16_t sb = m >= 0x7f80u ? (uint16_t)0x7fc0u
                                     : f32_to_bf16_rn(__fdiv_rn(__uint_as_float(m << 16), 7.f));
    const float s = __uint_as_float((uint32_t)sb << 16);
    const int64_t g = (b * 4 + j) >> shift;
    // a group has one writer: its first lane
    if (in && (lane & (lanes - 1)) == 0) scales[row * ns + g] = sb;
    if (!real) continue;
    const bool ok = s > 0.f, tiny = s < 0x1p-100f;
    const float inv = ok ? __frcp_rn(s) : 0.f;
    float f[8];
    unpack8(v, f);
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float r = 0.f;
      if (ok) {
        const float p = tiny ? __fdiv_rn(f[i], s) : f[i] * inv;
        // round to a multiple of 2^-12 (1.5 * 2^11 has that ulp), then to an integer
        const float snapped = __fadd_rn(__fadd_rn(p, 0x1.8p11f), -0x1.8p11f);
        r = fminf(fmaxf(rintf(snapped), -8.f), 7.f);
      }
      word |= (uint32_t)((int)r + 8) << (4 * ((i >> 1) + 4 * (i & 1)));
    }
    *reinterpret_cast<uint32_t*>(q + (row * blocks + b) * kW4BlockBytes + 16 * t + 4 * j) = word;
  }
}

// The inverse: (c - 8) s is exact in fp32 (4 by 8 significant bits); bf16 rounds it once.
template <bool VEC, bool BF16>
__global__ void __launch_bounds__(kQuantThreads)
dequantize_w4_kernel(const uint8_t* __restrict__ q, const uint16_t* __restrict__ scales,
                     int64_t rows, int64_t K, int shift, void* __restrict__ out) {
  const int lane = threadIdx.x & 15, j = lane >> 2, t = lane & 3;
  const int64_t blocks = w4_blocks(K);
  const int64_t ns = w4_row_scales(K, 32 << shift);
  const int64_t total = rows * blocks, stride = (int64_t)gridDim.x * (kQuantThreads / 16);
  for (int64_t vb = (int64_t)blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4); vb < total;
       vb += stride) {
    const int64_t row = vb / blocks, b = vb - row * blocks;
    const int64_t e = b * kW4Block + 32 * j + 8 * t;
    if (e >= K) continue;
    const uint32_t word =
        __ldg(reinterpret_cast<const uint32_t*>(q + vb * kW4BlockBytes + 16 * t + 4 * j));
    const float s = bf16lo(__ldg(scales + row * ns + ((b * 4 + j) >> shift)));
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      f[i] = (float)((int)((word >> (4 * ((i >> 1) + 4 * (i & 1)))) & 15u) - 8) * s;
    if constexpr (BF16) {
      uint16_t* o = static_cast<uint16_t*>(out) + row * K + e;
      if constexpr (VEC) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          u[i] = (uint32_t)f32_to_bf16_rn(f[2 * i]) | (uint32_t)f32_to_bf16_rn(f[2 * i + 1]) << 16;
        *reinterpret_cast<uint4*>(o) = make_uint4(u[0], u[1], u[2], u[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < K) o[i] = f32_to_bf16_rn(f[i]);
      }
    } else {
      float* o = static_cast<float*>(out) + row * K + e;
      if constexpr (VEC) {
        reinterpret_cast<float4*>(o)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(f[4], f[5], f[6], f[7]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (e + i < K) o[i] = f[i];
      }
    }
  }
}

int quant_blocks(int64_t items, int sms) {
  const int64_t per = kQuantThreads / 16;
  const int64_t need = (items + per - 1) / per, most = (int64_t)sms * 8;
  return (int)(need < most ? need : most);
}

}  // namespace

cudaError_t launch_quantize_w4(const uint16_t* w, int64_t rows, int64_t K, int shift, uint8_t* q,
                               uint16_t* scales, int sms, cudaStream_t st) {
  const int64_t items = rows * ((w4_row_scales(K, 32 << shift) << shift) >> 2);
  if (items == 0) return cudaSuccess;
  LaunchScope scope(MOE_K_OTHER, st);
  if (K % 8 == 0)
    quantize_w4_kernel<true><<<quant_blocks(items, sms), kQuantThreads, 0, st>>>(w, rows, K, shift, q, scales);
  else
    quantize_w4_kernel<false><<<quant_blocks(items, sms), kQuantThreads, 0, st>>>(w, rows, K, shift, q, scales);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_w4(const uint8_t* q, const uint16_t* scales, int64_t rows, int64_t K,
                                 int shift, void* out, bool bf16, int sms, cudaStream_t st) {
  const int64_t items = rows * w4_blocks(K);
  if (items == 0) return cudaSuccess;
  LaunchScope scope(MOE_K_OTHER, st);
  const int grid = quant_blocks(items, sms);
#define MOE_DEQ(VEC, BF) \
  dequantize_w4_kernel<VEC, BF><<<grid, kQuantThreads, 0, st>>>(q, scales, rows, K, shift, out)
  if (K % 8 == 0) {
    if (bf16) MOE_DEQ(true, true);
    else MOE_DEQ(true, false);
  } else {
    if (bf16) MOE_DEQ(false, true);
    else MOE_DEQ(false, false);
  }
#undef MOE_DEQ
  return cudaGetLastError();
}

}  // namespace moe

// w4_quant.cu -- the 4-bit weight pre-pass and its inverse (format: include/moe.h, w4.cuh).
//
//   scale = bf16(amax_group / 7)       code = clamp(round_half_even(w / scale), -8, 7) + 8
//
// Half a warp takes one storage block of 128 elements: lane 4 j + t reads elements
// 32 j + 8 t .. + 7 (16 bytes, in row order) and writes word 4 t + j, so a block is one
// 256-byte read and one 64-byte write, and a group's maximum is a shuffle over 4, 8 or 16
// lanes. Four blocks a half warp are in flight. 2 bytes read and 1/2 + 2/group
// written per weight. 40960 x 2560 in groups of 32: 65 us, 131072 x 2048 in groups of 128: 155 us
// (4.3 TB/s; the copy rate is 6.56), and back to fp32 104 us (4.6 TB/s), to bf16 114 us (5.9 TB/s).
// The way there is held back by its instructions: 126 (groups of 128) for a lane's eight weights, 2.96 of 4
// a clock, at 48 % of the DRAM rate. Back to fp32 by its stores: a lane writes its 32 bytes as two halves, so a
// store instruction covers half of each sector it touches (32 sectors where 16 hold the data); to bf16 by HBM.
// 32 CTAs an SM in turn are 5 to 15 % faster than the 8 that fit at once: no tail of slow ones.
//
// The quotient without a division: with 8-bit significands w / scale is either exactly half
// way between two integers or at least 2^-10 away from it (for |w / scale| >= 1/4 its
// distance is a multiple of 1/2 over twice an 8-bit integer). fma(w, 1 / scale, 2^11 + 2^10) is it
// to a multiple of 2^-12, off by less than that, so an exact tie is exact again and nothing
// else has crossed one; adding 2^23 + 2^22 + 8 - 2^11 - 2^10 rounds it to an integer, ties to even, and
// leaves code in the low bits. Scales so small that the reciprocal leaves fp32's range divide
// instead. amax / 7 has no such ties (7 divides no odd multiple of a half step), so a
// multiplication by 1/7 rounds to the same bf16.
#include "moe_internal.h"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kQuantThreads = 256;

// Eight bf16 of row r at element e, zeros behind the row's end. Where rows do not start on 16 bytes
// (VEC false) they come as the five aligned words that hold them, except at the matrix's two ends.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* w, uint32_t r, uint32_t e, uint32_t K, uint64_t total) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (e >= K) return v;
  const uint64_t at = (uint64_t)r * K + e;
  const uint16_t* p = w + at;
  if constexpr (VEC) {
    v = ld_stream_v4(p);
  } else {
    uint32_t* u = &v.x;
    const int n = (int)min(8u, K - e);
    if (at > 0 && at + 9 <= total) {
      const bool odd = (reinterpret_cast<uintptr_t>(p) & 2u) != 0;
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p - odd);
      uint32_t x[5];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __ldg(q + i);
      x[4] = odd ? __ldg(q + 4) : 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = odd ? __byte_perm(x[i], x[i + 1], 0x5432) : x[i];
        if (2 * i + 1 >= n) u[i] = 2 * i < n ? u[i] & 0xffffu : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) u[i >> 1] |= (uint32_t)__ldg(p + i) << (16 * (i & 1));
    }
  }
  return v;
}

// Blocks i, i + stride, ... of a matrix with `per_row` blocks a row, without a division a step.
// The numbers are 32-bit (at most 2^31 rows of 2^20 elements), so that an address is one wide
// multiplication.
struct BlockWalk {
  uint32_t row, b, per_row, row_step, b_step;
  __device__ BlockWalk(uint32_t first, uint32_t stride, uint32_t per_row)
      : row(first / per_row), b(first % per_row), per_row(per_row), row_step(stride / per_row), b_step(stride % per_row) {}
  __device__ void next() {
    row += row_step;
    b += b_step;
    if (b >= per_row) {
      b -= per_row;
      ++row;
    }
  }
};
constexpr int kQuantBatch = 4;

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The word of eight elements' codes.
__device__ __forceinline__ uint32_t codes8(const uint4& v, float s) {
  float f[8];
  unpack8(v, f);
  uint32_t c[8];
  if (s >= 0x1p-100f) {
    const float inv = __frcp_rn(s);
    const uint64_t inv2 = pack2(inv, inv), snap = pack2(0x1.8p11f, 0x1.8p11f), whole = pack2(12579848.f, 12579848.f);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t r = add2(fma2(pack2(f[i], f[i + 1]), inv2, snap), whole);
      c[i] = (uint32_t)r;
      c[i + 1] = (uint32_t)(r >> 32);
    }
  } else {
    const bool ok = s > 0.f;  // a zero or NaN scale: all codes 8
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = ok ? (uint32_t)((int)fminf(fmaxf(rintf(__fdiv_rn(f[i], s)), -8.f), 7.f) + 8) : 8u;
  }
  // low bytes of the even elements, then of the odd ones; two nibbles a byte
  const uint32_t e = __byte_perm(__byte_perm(c[0], c[2], 0x0040), __byte_perm(c[4], c[6], 0x0040), 0x5410);
  const uint32_t o = __byte_perm(__byte_perm(c[1], c[3], 0x0040), __byte_perm(c[5], c[7], 0x0040), 0x5410);
  return __byte_perm(e | (e >> 4), o | (o >> 4), 0x6420);
}

template <bool VEC, int SHIFT>
__global__ void __launch_bounds__(kQuantThreads)
quantize_w4_kernel(const uint16_t* __restrict__ w, uint32_t rows, int64_t K, uint8_t* __restrict__ q,
                   uint16_t* __restrict__ scales) {
  const int lane = threadIdx.x & 15, j = lane >> 2, t = lane & 3;
  const uint32_t blocks = (uint32_t)w4_blocks(K), ns = (uint32_t)w4_row_scales(K, 32 << SHIFT), k = (uint32_t)K;
  const uint32_t vblocks = (ns << SHIFT) >> 2;  // blocks with the scale padding's share, >= blocks
  const uint32_t stride = gridDim.x * (kQuantThreads / 16);
  constexpr int lanes = 4 << SHIFT;  // lanes of a group
  BlockWalk at(blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4), stride, vblocks);
  // both halves of a warp stay in the loop as long as one has a block (the shuffles)
  while (__any_sync(0xffffffffu, at.row < rows)) {
    uint4 v[kQuantBatch];
    uint32_t row[kQuantBatch], b[kQuantBatch];
#pragma unroll
    for (int u = 0; u < kQuantBatch; ++u) {
      row[u] = at.row;
      b[u] = at.b;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      if (at.row < rows && at.b < blocks)
        v[u] = load8<VEC>(w, at.row, at.b * kW4Block + 32 * j + 8 * t, k, (uint64_t)rows * k);
      at.next();
    }
#pragma unroll
    for (int u = 0; u < kQuantBatch; ++u) {
      // |w| as integers: infinities and NaN sort above every finite value
      uint32_t m = __vmaxu2(__vmaxu2(v[u].x & 0x7fff7fffu, v[u].y & 0x7fff7fffu),
                            __vmaxu2(v[u].z & 0x7fff7fffu, v[u].w & 0x7fff7fffu));
      m = max(m & 0xffffu, m >> 16);
#pragma unroll
      for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      // a group with an infinity or a NaN gets a NaN scale, so that all of it reads back as NaN
      const uint16_t sb =
          m >= 0x7f80u ? (uint16_t)0x7fc0u : f32_to_bf16_rn(__uint_as_float(m << 16) * (1.f / 7.f));
      if (row[u] >= rows) continue;
      // a group has one writer: its first lane
      if ((lane & (lanes - 1)) == 0) scales[(uint64_t)row[u] * ns + ((b[u] * 4 + j) >> SHIFT)] = sb;
      if (b[u] < blocks)
        *reinterpret_cast<uint32_t*>(q + ((uint64_t)row[u] * blocks + b[u]) * kW4BlockBytes + 16 * t + 4 * j) =
            codes8(v[u], __uint_as_float((uint32_t)sb << 16));
    }
  }
}

// A block of 128 values of a row to a place without alignment: through shared memory, so that the
// half warp's stores lie side by side. `n`: the values that are in the row.
__device__ __forceinline__ void store_block(float* buf, const uint4& v, uint16_t* o, int n, int lane, uint32_t mask) {
  uint32_t* b = reinterpret_cast<uint32_t*>(buf);
  reinterpret_cast<uint4*>(b)[lane] = v;
  __syncwarp(mask);
  const int odd = (int)((reinterpret_cast<uintptr_t>(o) >> 1) & 1u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = lane + 16 * i, e = 2 * k + odd;
    const uint32_t two = odd ? __byte_perm(b[k], b[min(k + 1, 63)], 0x5432) : b[k];
    if (e + 1 < n) *reinterpret_cast<uint32_t*>(o + e) = two;
    else if (e < n) o[e] = (uint16_t)two;
  }
  if (odd && lane == 0) o[0] = (uint16_t)b[0];
  __syncwarp(mask);
}
__device__ __forceinline__ void store_block(float* buf, const float (&f)[8], float* o, int n, int lane, uint32_t mask) {
#pragma unroll
  for (int i = 0; i < 8; ++i) buf[8 * lane + i] = f[i];
  __syncwarp(mask);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (lane + 16 * i < n) o[lane + 16 * i] = buf[lane + 16 * i];
  __syncwarp(mask);
}

// The inverse: (c - 8) s is exact in fp32 (4 by 8 significant bits); bf16 rounds it once.
template <bool VEC, bool BF16, int SHIFT>
__global__ void __launch_bounds__(kQuantThreads)
dequantize_w4_kernel(const uint8_t* __restrict__ q, const uint16_t* __restrict__ scales,
                     uint32_t rows, int64_t K, void* __restrict__ out) {
  const int lane = threadIdx.x & 15, j = lane >> 2, t = lane & 3;
  __shared__ __align__(16) float lines[VEC ? 1 : kQuantThreads / 16][kW4Block];
  float* buf = lines[VEC ? 0 : threadIdx.x >> 4];
  const uint32_t half = 0xffffu << (threadIdx.x & 16);
  const uint32_t blocks = (uint32_t)w4_blocks(K), ns = (uint32_t)w4_row_scales(K, 32 << SHIFT), k = (uint32_t)K;
  const uint32_t stride = gridDim.x * (kQuantThreads / 16);
  BlockWalk at(blockIdx.x * (kQuantThreads / 16) + (threadIdx.x >> 4), stride, blocks);
  while (at.row < rows) {
    uint32_t word[kQuantBatch], scale[kQuantBatch];
    uint32_t row[kQuantBatch], b[kQuantBatch];
#pragma unroll
    for (int u = 0; u < kQuantBatch; ++u) {
      row[u] = at.row;
      b[u] = at.b;
      word[u] = scale[u] = 0u;
      if (at.row < rows && at.b * kW4Block + 32 * j + 8 * t < k) {
        word[u] = __ldg(reinterpret_cast<const uint32_t*>(q + ((uint64_t)at.row * blocks + at.b) * kW4BlockBytes + 16 * t + 4 * j));
        scale[u] = __ldg(scales + (uint64_t)at.row * ns + ((at.b * 4 + j) >> SHIFT));
      }
      at.next();
    }
#pragma unroll
    for (int u = 0; u < kQuantBatch; ++u) {
      if (row[u] >= rows) continue;
      const uint4 c = w4_codes(word[u]);  // c - 8 as bf16, exactly
      const uint64_t at = (uint64_t)row[u] * k + b[u] * kW4Block;
      const int n = (int)min((uint32_t)kW4Block, k - b[u] * kW4Block);
      if constexpr (BF16) {
        uint16_t* o = static_cast<uint16_t*>(out) + at;
        const uint32_t s2 = scale[u] * 0x10001u;
        const uint4 r = make_uint4(mul_bf16x2(c.x, s2), mul_bf16x2(c.y, s2), mul_bf16x2(c.z, s2), mul_bf16x2(c.w, s2));
        if constexpr (!VEC) store_block(buf, r, o, n, lane, half);
        else if (8 * lane < n) reinterpret_cast<uint4*>(o)[lane] = r;
      } else {
        float* o = static_cast<float*>(out) + at;
        const float s = bf16lo(scale[u]);
        float f[8];
        unpack8(c, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= s;
        if constexpr (!VEC) {
          store_block(buf, f, o, n, lane, half);
        } else if (8 * lane < n) {
          reinterpret_cast<float4*>(o)[2 * lane] = make_float4(f[0], f[1], f[2], f[3]);
          reinterpret_cast<float4*>(o)[2 * lane + 1] = make_float4(f[4], f[5], f[6], f[7]);
        }
      }
    }
  }
}

int quant_blocks(int64_t items, int sms) {
  const int64_t per = kQuantThreads / 16;
  const int64_t need = (items + per - 1) / per, most = (int64_t)sms * 32;
  return (int)(need < most ? need : most);
}

}  // namespace

cudaError_t launch_quantize_w4(const uint16_t* w, int64_t rows, int64_t K, int shift, uint8_t* q,
                               uint16_t* scales, int sms, cudaStream_t st) {
  const int64_t items = rows * ((w4_row_scales(K, 32 << shift) << shift) >> 2);
  if (items == 0) return cudaSuccess;
  LaunchScope scope(MOE_K_OTHER, st);
  const int grid = quant_blocks(items, sms);
#define MOE_QUANT(VEC, SH) \
  quantize_w4_kernel<VEC, SH><<<grid, kQuantThreads, 0, st>>>(w, (uint32_t)rows, K, q, scales)
  if (K % 8 == 0) {
    if (shift == 0) MOE_QUANT(true, 0);
    else if (shift == 1) MOE_QUANT(true, 1);
    else MOE_QUANT(true, 2);
  } else {
    if (shift == 0) MOE_QUANT(false, 0);
    else if (shift == 1) MOE_QUANT(false, 1);
    else MOE_QUANT(false, 2);
  }
#undef MOE_QUANT
  return cudaGetLastError();
}

namespace {
template <bool VEC, bool BF16>
void dequantize(const uint8_t* q, const uint16_t* scales, int64_t rows, int64_t K, int shift, void* out, int grid,
                cudaStream_t st) {
  if (shift == 0) dequantize_w4_kernel<VEC, BF16, 0><<<grid, kQuantThreads, 0, st>>>(q, scales, (uint32_t)rows, K, out);
  else if (shift == 1) dequantize_w4_kernel<VEC, BF16, 1><<<grid, kQuantThreads, 0, st>>>(q, scales, (uint32_t)rows, K, out);
  else dequantize_w4_kernel<VEC, BF16, 2><<<grid, kQuantThreads, 0, st>>>(q, scales, (uint32_t)rows, K, out);
}
}  // namespace

cudaError_t launch_dequantize_w4(const uint8_t* q, const uint16_t* scales, int64_t rows, int64_t K,
                                 int shift, void* out, bool bf16, int sms, cudaStream_t st) {
  const int64_t items = rows * w4_blocks(K);
  if (items == 0) return cudaSuccess;
  LaunchScope scope(MOE_K_OTHER, st);
  const int grid = quant_blocks(items, sms);
  if (K % 8 == 0) {
    if (bf16) dequantize<true, true>(q, scales, rows, K, shift, out, grid, st);
    else dequantize<true, false>(q, scales, rows, K, shift, out, grid, st);
  } else {
    if (bf16) dequantize<false, true>(q, scales, rows, K, shift, out, grid, st);
    else dequantize<false, false>(q, scales, rows, K, shift, out, grid, st);
  }
  return cudaGetLastError();
}

}  // namespace moe

// w4.cuh -- the 4-bit weight format on the device, and the warp-level products that the
// few-token kernels build on.
//
// Format (include/moe.h): a weight is (c - 8) s with a code c in 0..15 and the bf16 scale s
// of its group. A row is stored in blocks of 128 elements = 64 bytes = 16 words; word
// 4 t + j holds elements 32 j + 8 t + i (i < 8), element i in nibble (i >> 1) + 4 (i & 1).
//
// Why this order. The products run on mma.sync.m16n8k16 with the weights as A (16 weight
// rows) and the tokens as B (8 tokens): a few tokens give each weight 8 columns of use at
// most, so the kernels are bound by the weight bytes and take the tensor instruction only
// for its cheap operand path; a tcgen05 tile would need the dequantised weights written back
// to shared memory first. In an A fragment lane 4 g + t holds elements of row g at K
// positions that depend on t alone, and the sum over K may run in any order. So lane t takes
// its 16-byte quarter of a block in one load: word j is its share (8 of 32 elements) of the
// j-th 32-element group, two whole MMAs of one scale group, and the nibble order makes
// ((word >> 4 m) & 0x000f000f) the element pair (2 m, 2 m + 1) as it lies in a row of x.
#pragma once

#include <stdint.h>

#include "device_common.cuh"

namespace moe {

constexpr int kW4Block = 128;      // elements of a storage block
constexpr int kW4BlockBytes = 64;

__host__ __device__ inline int64_t w4_blocks(int64_t K) { return (K + kW4Block - 1) / kW4Block; }
__host__ __device__ inline int64_t w4_row_bytes(int64_t K) { return w4_blocks(K) * kW4BlockBytes; }
// scales of a row, padded to whole 16-byte vectors
__host__ __device__ inline int64_t w4_row_scales(int64_t K, int group) {
  return ((K + group - 1) / group + 7) / 8 * 8;
}

// D += A B, m16n8k16, fp32 accumulators; A and B both bf16 or both fp16.
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9},"
        " {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 32 elements x 16 rows of one K block of 32: lane 4 g + t holds 16 bytes of row g (a) and
// of row g + 8 (b) at elements 8 t .. 8 t + 7, and of token g (x) at the same elements.
template <bool F16>
__device__ __forceinline__ void mma_k32(float (&d)[4], const uint4& a, const uint4& b,
                                        const uint4& x) {
  mma16816<F16>(d, a.x, b.x, a.y, b.y, x.x, x.y);
  mma16816<F16>(d, a.z, b.z, a.w, b.w, x.z, x.w);
}

__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
  return r;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// One word of codes -> the four pairs (2 m, 2 m + 1), m = 0..3, of c - 8: exact. A code in the
// low mantissa bits of 128 (bf16) or 1024 (fp16) is 128 + c or 1024 + c; fp16 has room for the
// code four bits higher too (1024 + 16 c), which saves a shift.
template <bool F16>
__device__ __forceinline__ uint4 w4_pairs(uint32_t w) {
  uint4 r;
  if constexpr (F16) {
    const uint32_t v = w >> 8;
    r.x = sub_f16x2(and_or(w, 0x000f000fu, 0x64006400u), 0x64086408u);              // - 1032
    r.y = fma_f16x2(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);  // /16 - 72
    r.z = sub_f16x2(and_or(v, 0x000f000fu, 0x64006400u), 0x64086408u);
    r.w = fma_f16x2(and_or(v, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
  } else {
    r.x = sub_bf16x2(and_or(w, 0x000f000fu, 0x43004300u), 0x43084308u);  // 128 + c - 136
    r.y = sub_bf16x2(and_or(w >> 4, 0x000f000fu, 0x43004300u), 0x43084308u);
    r.z = sub_bf16x2(and_or(w >> 8, 0x000f000fu, 0x43004300u), 0x43084308u);
    r.w = sub_bf16x2(and_or(w >> 12, 0x000f000fu, 0x43004300u), 0x43084308u);
  }
  return r;
}

// The scales of a block's four 32-element parts: group 32 << shift elements, `s` the row.
__device__ __forceinline__ void w4_block_scales(const uint16_t* s, int block, int shift, float (&f)[4]) {
  if (shift == 0) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(s + 4 * (int64_t)block));
    f[0] = bf16lo(v.x); f[1] = bf16hi(v.x);
    f[2] = bf16lo(v.y); f[3] = bf16hi(v.y);
  } else if (shift == 1) {
    const uint32_t v = __ldg(reinterpret_cast<const uint32_t*>(s + 2 * (int64_t)block));
    f[0] = f[1] = bf16lo(v);
    f[2] = f[3] = bf16hi(v);
  } else {
    f[0] = f[1] = f[2] = f[3] = bf16lo(__ldg(s + block));
  }
}

}  // namespace moe

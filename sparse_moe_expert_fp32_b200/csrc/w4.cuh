// w4.cuh -- the 4-bit weight format on the device, and the warp-level products that the
// few-token kernels build on.
//
// Format (include/moe.h): a weight is (c - 8) s with a code c in 0..15 and the bf16 scale s
// of its group. A row is stored in blocks of 128 elements = 64 bytes = 16 words; word
// 4 t + j holds elements 32 j + 8 t + i (i < 8), element i in nibble (i >> 1) + 4 (i & 1).
//
// Why this order. The products run on mma.sync.m16n8k16: a few tokens give each weight at most
// 16 uses, so the kernels are bound by the weight bytes, and a tensor instruction is only the
// cheapest way to spend them (a tcgen05 tile would need the dequantised weights written back to
// shared memory, four times the codes' bytes). Its operands are register quads (A) and pairs (B)
// that have to be consecutive, and a move costs as much as any other instruction, so they are taken
// as they come out of one load. A thread reads 16 bytes of one weight row: lane
// 4 g + t the quarter t of row g. Since a sum over K may run in any order, a word of codes, an
// eighth of a 32-element part of one scale group, becomes four consecutive pairs of elements.
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

// D = A B (+ D), m16n8k16, fp32 accumulators; A and B both bf16 or both fp16.
#define MOE_MMA_16816(T) "mma.sync.aligned.m16n8k16.row.col.f32." T "." T ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm(MOE_MMA_16816("f16") "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm(MOE_MMA_16816("bf16") "{%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool F16>
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm(MOE_MMA_16816("f16") "{%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm(MOE_MMA_16816("bf16") "{%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8 weight rows by 32 elements as A. Lane 4 g + t holds elements 8 t .. 8 t + 7 of row g, four
// registers in order, so MMA row g has the register pairs 0 and 2 and MMA row g + 8 the pairs 1 and 3
// of the same weight row. B gives columns 0-3 the elements that belong to the first (`x`: registers 0
// and 2 of a column's 16 bytes) and columns 4-7 those of the second (registers 1 and 3): four columns
// of x, d[0], d[1] of lanes t < 2 and d[2], d[3] of lanes t >= 2 hold the two halves of their sums,
// and the rest of D means nothing. See fold().
__device__ __forceinline__ void mma_rows(float (&d)[4], const uint4& w, const uint2& x) {
  mma16816<false>(d, w.x, w.y, w.z, w.w, x.x, x.y);
}

__device__ __forceinline__ uint32_t word(const uint4& v, int j) { return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w; }

// Shared memory by 32-bit address; the _if forms leave v as it is where p is 0.
__device__ __forceinline__ uint4 lds_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}
__device__ __forceinline__ void lds_v4_if(uint4& v, uint32_t at, int p) {
  asm volatile("{\n .reg .pred q;\n setp.ne.s32 q, %5, 0;\n @q ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n}\n"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
               : "r"(at), "r"(p));
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
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
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

// One word of codes -> the four pairs (2 m, 2 m + 1), m = 0..3, of (c - 8) / kW4Unit: exact, and
// without moving every code to the lowest bits. fp16: a code in the low mantissa bits of 1024 is
// 1024 + c, one four bits higher 1024 + 16 c (the method of Kim, Henry, Fahim and Hassan Awadalla, "Who
// Says Elephants Can't Run", 2022). bf16 has no such room, but taken as a bf16 by themselves
// (subnormal, or of the lowest binade, which goes on in the same steps) the code is c 2^-133 and the one
// four bits higher c 2^-129; a multiplication by 2^127 or 2^123 brings both to c / 64. The sums are
// multiplied by 64 at the end: exact, but for results below 2^-120, which were subnormal meanwhile.
// (4-bit layer, 5 tokens: 71 us, with every code in the lowest bits 74 us.)
template <bool F16>
constexpr float kW4Unit = F16 ? 1.f : 64.f;
template <bool F16>
__device__ __forceinline__ uint4 w4_pairs(uint32_t w) {
  uint4 r;
  const uint32_t v = w >> 8;
  if constexpr (F16) {
    r.x = sub_f16x2(and_or(w, 0x000f000fu, 0x64006400u), 0x64086408u);              // - 1032
    r.y = fma_f16x2(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);  // /16 - 72
    r.z = sub_f16x2(and_or(v, 0x000f000fu, 0x64006400u), 0x64086408u);
    r.w = fma_f16x2(and_or(v, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
  } else {
    r.x = fma_bf16x2(w & 0x000f000fu, 0x7f007f00u, 0xbe00be00u);  // 2^127, -1/8
    r.y = fma_bf16x2(w & 0x00f000f0u, 0x7d007d00u, 0xbe00be00u);  // 2^123
    r.z = fma_bf16x2(v & 0x000f000fu, 0x7f007f00u, 0xbe00be00u);
    r.w = fma_bf16x2(v & 0x00f000f0u, 0x7d007d00u, 0xbe00be00u);
  }
  return r;
}
// The same as bf16 pairs of c - 8 itself: 128 + c - 136.
__device__ __forceinline__ uint4 w4_codes(uint32_t w) {
  return make_uint4(sub_bf16x2(and_or(w, 0x000f000fu, 0x43004300u), 0x43084308u),
                    sub_bf16x2(and_or(w >> 4, 0x000f000fu, 0x43004300u), 0x43084308u),
                    sub_bf16x2(and_or(w >> 8, 0x000f000fu, 0x43004300u), 0x43084308u),
                    sub_bf16x2(and_or(w >> 12, 0x000f000fu, 0x43004300u), 0x43084308u));
}

// The scales of a block's four 32-element parts as four bf16: group 32 << shift elements, `s` the
// row's scales in global memory, `at` their address in shared memory.
__device__ __forceinline__ uint2 w4_spread1(uint32_t v) {
  return make_uint2(__byte_perm(v, v, 0x1010), __byte_perm(v, v, 0x3232));
}
__device__ __forceinline__ uint2 w4_block_scales(const uint16_t* s, int block, int shift) {
  if (shift == 0) return __ldg(reinterpret_cast<const uint2*>(s + 4 * (int64_t)block));
  if (shift == 1) return w4_spread1(__ldg(reinterpret_cast<const uint32_t*>(s + 2 * (int64_t)block)));
  const uint32_t v = __ldg(s + block) * 0x10001u;
  return make_uint2(v, v);
}
template <int SHIFT>
__device__ __forceinline__ uint2 w4_block_scales(uint32_t at, int block) {
  uint32_t v;
  if constexpr (SHIFT == 0) return lds_v2(at + 8 * block);
  if constexpr (SHIFT == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at + 4 * block));
    return w4_spread1(v);
  }
  asm volatile("{\n .reg .u16 h;\n ld.shared.u16 h, [%1];\n mov.b32 %0, {h, h};\n}\n" : "=r"(v) : "r"(at + 2 * block));
  return make_uint2(v, v);
}
__device__ __forceinline__ float w4_scale(const uint2& s, int j) {
  const uint32_t v = j & 2 ? s.y : s.x;
  return j & 1 ? bf16hi(v) : bf16lo(v);
}

}  // namespace moe

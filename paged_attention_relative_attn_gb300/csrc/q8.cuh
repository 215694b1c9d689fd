// The 8-bit block format of the paged K/V cache (kv8), shared by the kernels
// that write, read and attend over it.  Its definition is in
// include/inkling_rel_attn.h, "The 8-bit cache".
//
// A block (16 tokens of one page and KV head) stands for x * 2^e with e4m3
// numbers x and one exponent e.  A power of two as scale: x * 2^e has 4 significant
// bits and is a bf16 number, so nothing is rounded when a row is read back, and when
// a joining row raises e, the rows that are there change by an exact division
// unless they fall under e4m3's smallest normal number.
//
// Rows are stored in the order of their channels, in 16-byte units (8-byte ones for V
// rows of 64 channels) exchanged between rows so that the lanes of a warp, which
// take an operand's rows side by side, find theirs in different banks of shared memory.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"

namespace ira {

constexpr int kQ8Block = 16;      // tokens per block (the M of one MMA)
constexpr int kQ8MinExp = -60;    // the smallest exponent, of a block of zeros too
constexpr int kQ8MaxExp = 55;     // larger magnitudes than 448 * 2^55 count as it

// Bytes of a block: 16 rows of D bytes, then the scale (fp32), the NaN rows (16 bits) and zeros.
__host__ __device__ constexpr int q8_block_bytes(int D) { return kQ8Block * (D + 1); }
__host__ __device__ constexpr int q8_tail_off(int D) { return kQ8Block * D; }

// Where token `place` of a page keeps KV head `h`: byte offset of its block.
__device__ __forceinline__ size_t q8_block_at(int page, int h, int place, int H_kv, int P, int D) {
  return (((size_t)page * H_kv + h) * (P / kQ8Block) + place / kQ8Block) * q8_block_bytes(D);
}

// Byte of channels 8u .. 8u + 7 of row r in a block.
template <int D, bool IS_V>
__device__ __forceinline__ int q8_unit_at(int r, int u) {
  if (D == 128) return r * 128 + 16 * ((u >> 1) ^ (IS_V ? 2 * ((r >> 1) & 3) : 4 * (r & 1))) + 8 * (u & 1);
  if (!IS_V) return r * 64 + 8 * u;
  return (r >> 1) * 128 + 8 * (4 * ((2 * (r & 1) + (u >> 2)) ^ ((r >> 1) & 3)) + (u & 3));
}

// The first 8 bytes of a block's tail.
struct Q8Tail {
  uint32_t scale;  // 2^e, as fp32
  uint32_t nan;    // bit r: row r reads as NaN
};
__device__ __forceinline__ uint32_t q8_scale_bits(int e) { return (uint32_t)(e + 127) << 23; }
// Exponent of a scale; below kQ8MinExp when the block has not been begun (a pool starts as zeros).
__device__ __forceinline__ int q8_exp(uint32_t scale) {
  const int e = (int)(scale >> 23) - 127;
  return (scale & 0x807fffffu) == 0 && e >= kQ8MinExp && e <= kQ8MaxExp ? e : kQ8MinExp - 1;
}
// Smallest exponent with magnitude <= 448 * 2^e, within the range, from a bf16's bits: 448 = 1.75 * 2^8.
__device__ __forceinline__ int q8_exp_for(uint32_t magnitude_bits) {
  const int e = (int)((magnitude_bits + 0x1fu) >> 7) - 127 - 8;
  return min(max(e, kQ8MinExp), kQ8MaxExp);
}

// e4m3 pair -> fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_bytes) {
  uint32_t r;
  asm("{.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;}" : "=r"(r) : "r"(two_bytes));
  return r;
}
// Both pairs of a word, exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// Four fp32 to e4m3, to nearest even, magnitudes past 448 as 448.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 8 channels (8 x bf16) times f = 2^-e as e4m3.
__device__ __forceinline__ uint2 q8_quantise8(const uint4& v, float f) {
  return make_uint2(e4m3x4(bf16_lo(v.x) * f, bf16_hi(v.x) * f, bf16_lo(v.y) * f, bf16_hi(v.y) * f),
                    e4m3x4(bf16_lo(v.z) * f, bf16_hi(v.z) * f, bf16_lo(v.w) * f, bf16_hi(v.w) * f));
}

// 4 stored values times 2^-d (d >= 1), rounded again.  In fp16 the quotient is exact down to 2^-24,
// far below half of e4m3's smallest number.
__device__ __forceinline__ uint32_t q8_rescale4(uint32_t w, uint32_t factor_f16x2) {
  uint32_t lo, hi, r;
  e4m3x4_to_f16(w, lo, hi);
  asm("{.reg .b32 x, y;\n\t.reg .b16 a, b;\n\tmul.rn.f16x2 x, %1, %3;\n\tmul.rn.f16x2 y, %2, %3;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 a, x;\n\tcvt.rn.satfinite.e4m3x2.f16x2 b, y;\n\tmov.b32 %0, {a, b};}"
      : "=r"(r)
      : "r"(lo), "r"(hi), "r"(factor_f16x2));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_pow2_down(int d) {  // 2^-d twice; 0 from 25 on
  const uint32_t h = d <= 14 ? (uint32_t)(15 - d) << 10 : d <= 24 ? 1u << (24 - d) : 0u;
  return h | h << 16;
}

// The values of 4 stored bytes times the scale, as bf16 pairs: exact.
__device__ __forceinline__ uint2 q8_values4(uint32_t w, float s) {
  uint32_t lo, hi;
  e4m3x4_to_f16(w, lo, hi);
  float a, b, c, d;
  asm("{.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;}" : "=f"(a), "=f"(b) : "r"(lo));
  asm("{.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.f32.f16 %0, x;\n\tcvt.f32.f16 %1, y;}" : "=f"(c), "=f"(d) : "r"(hi));
  return make_uint2(__byte_perm(__float_as_uint(a * s), __float_as_uint(b * s), 0x7632),
                    __byte_perm(__float_as_uint(c * s), __float_as_uint(d * s), 0x7632));
}

}  // namespace ira

// The 4-bit row format of the paged K/V cache (kv4), shared by the kernels
// that write, read and attend over it.  Its definition is in
// include/inkling_rel_attn.h, "The 4-bit cache".
//
// A group (32 adjacent channels of a token's row of one KV head) stands for
// x * s with integers x in -7..7, stored as the nibble u = x + 8, and a scale s
// of 5 significant bits: x * s then has at most 8 and is a bf16 number, so
// nothing is rounded when a row is read back as bf16.
//
// The nibbles of a row are ordered for the tensor-core fragments: lane 4g + t
// of a warp needs, of a K row (an MMA row), 8 channels of every group, and of
// a V row (an MMA column of V^T) 4 channels of every group; both are stored
// side by side for all groups, so a lane takes them with one load.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "internal.h"

namespace ira {

constexpr int kQ4Group = 32;  // channels per scale
constexpr int kQ4Block = 16;  // tokens per block (the M of one MMA)

// Bytes of a block: 16 nibble rows of D / 2 bytes, then 16 scale rows of D / 32 bf16.
__host__ __device__ constexpr int q4_block_bytes(int D) { return kQ4Block * (D / 2 + D / 16); }
__host__ __device__ constexpr int q4_scale_off(int D) { return kQ4Block * (D / 2); }

// Where token `place` of a page keeps KV head `h`: byte offset of its block.
__device__ __forceinline__ size_t q4_block_at(int page, int h, int place, int H_kv, int P, int D) {
  return (((size_t)page * H_kv + h) * (P / kQ4Block) + place / kQ4Block) * q4_block_bytes(D);
}

// Quantise 8 channels (one 16-byte load) of a group held by 4 adjacent lanes.
// Returns the 8 nibbles (channel c at bits 4c) and the scale's bf16 bits.
//
// Both quotients are taken as products with a reciprocal made a little too small,
// and come out as exact arithmetic would give them:
//   s = amax / 7 rounded up to 5 significant bits.  amax has 8 significant bits,
//     so amax / 7 is a 5-bit number or more than 2^-9 away from one; the factor
//     (1 - 2^-18) moves an exact one below itself, from where it is rounded up to itself.
//   x = v / s to nearest, ties toward zero.  v * (1 / s) * (1 - 2^-18) is rounded to
//     an integer by adding 1.5 * 2^23; quotients of an 8-bit by a 5-bit number
//     that are no tie lie more than 2^-12 from one, so the factor (and the
//     approximate reciprocal's 2^-22) turns exact ties toward zero and nothing else.
// The sums 1.5 * 2^23 + 8 + x are gathered as integers, each 16 times the last:
// their constant parts add up to a constant, which is taken off once.
__device__ __forceinline__ uint32_t q4_quantise8(const uint4& raw, uint32_t& s_bits) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                        __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t amax = max(m & 0xffffu, m >> 16);  // bits of the largest magnitude
  constexpr uint32_t kTiny = 27u << 7;               // 2^-100: below it the group is stored as zeros
  constexpr uint32_t kMost = 0x7f00u;                // 2^127: larger magnitudes, infinities too, count as it
  float lim = 0x1p127f;                              // (7 s, up to 17/16 of the largest, stays finite)
  const float a = fminf(__uint_as_float(amax << 16), lim);
  const uint32_t sb = (__float_as_uint(a * ((1.f - 0x1p-18f) / 7.f)) + 0x7ffffu) & ~0x7ffffu;
  float r = __fdividef(1.f - 0x1p-18f, __uint_as_float(sb));
  s_bits = sb >> 16;
  if (amax < kTiny) {
    s_bits = 0;
    r = 0.f;
  }
  if (amax > 0x7f80u) {  // a NaN: the group reads as NaN
    s_bits = 0x7fc0u;
    r = 0.f;
    lim = 0.f;
  }
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  if (amax > kMost) {  // rare: clamp, turn NaN into 0 (fminf / fmaxf drop NaN operands)
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = fmaxf(fminf(f[i], lim), -lim);
  }
  constexpr uint32_t kMagic = 0x4b400008u;  // 1.5 * 2^23 + 8
  uint32_t out = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) out = out * 16u + __float_as_uint(fmaf(f[i], r, __uint_as_float(kMagic)));
  return out - kMagic * 0x11111111u + 0x88888888u;
}

// The values of the 8 nibbles of a word times the scale (bf16 bits), as bf16 pairs:
// a nibble set under the exponent of 128 is 128 + u, from which 136 is taken off;
// that difference and its product with the scale are bf16 numbers, so nothing is rounded.
__device__ __forceinline__ uint4 q4_values8(uint32_t w, uint32_t s_bits) {
  const uint32_t hi = w >> 4;
  const uint32_t s2 = __byte_perm(s_bits, 0, 0x1010);
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // byte i: the even nibble to the low half, the odd one to the high half
    uint32_t u = (__byte_perm(w, hi, i | (4 + i) << 8) & 0x000f000fu) | 0x43004300u;
    asm("{.reg .b32 x;\n\tsub.rn.bf16x2 x, %1, %2;\n\tmul.rn.bf16x2 %0, x, %3;}"
        : "=r"(out[i]) : "r"(u), "r"(0x43084308u), "r"(s2));
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

}  // namespace ira

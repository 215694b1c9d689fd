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
// s = amax / 7 rounded up to 5 significant bits: the division is correctly
// rounded and the next 5-bit number is at least 2^-9 away unless the quotient
// is one, so the bits decide as exact arithmetic would.  x = v / s to nearest,
// ties toward zero: v * (1 / s) * (1 - 2^-18) is rounded to an integer by adding
// 1.5 * 2^23; quotients of an 8-bit by a 5-bit number that are no tie lie more
// than 2^-12 from one, so the factor turns exact ties toward zero and nothing else.
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
  const uint32_t sb = (__float_as_uint(__fdiv_rn(a, 7.f)) + 0x7ffffu) & ~0x7ffffu;
  float r = __fdiv_rn(1.f, __uint_as_float(sb)) * (1.f - 0x1p-18f);
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
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
    if (amax > kMost) {  // rare: clamp, turn NaN into 0 (fminf / fmaxf drop NaN operands)
      lo = fmaxf(fminf(lo, lim), -lim);
      hi = fmaxf(fminf(hi, lim), -lim);
    }
    constexpr float kMagic = 12582912.f + 8.f;
    out |= (__float_as_uint(fmaf(lo, r, kMagic)) & 15u) << (8 * i);
    out |= (__float_as_uint(fmaf(hi, r, kMagic)) & 15u) << (8 * i + 4);
  }
  return out;
}

// The two values at nibbles 2i, 2i + 1 of a word times s, as a bf16 pair (exact).
__device__ __forceinline__ uint32_t q4_value2(uint32_t w, int i, float s) {
  const float lo = (float)((int)((w >> (8 * i)) & 15u) - 8) * s;
  const float hi = (float)((int)((w >> (8 * i + 4)) & 15u) - 8) * s;
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

}  // namespace ira

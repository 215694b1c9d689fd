// Expansion for prefill over a cache in blocks of 16 tokens (the 4-bit and the 8-bit
// one): the keys that any query of sequence b's chunk sees,
// [lo_b, L_b), go to bf16 pages of 64 tokens of the scratch pool, sequence b's
// from page b * pages_per_seq on.  Its first key is base_b = lo_b rounded down
// to 64, so the scratch sequence has length L_b - base_b; relative positions,
// all that the attention uses, stay the same.  The scratch lengths and page
// table are written for the attention that follows.  A sequence that the
// scratch cannot hold, or whose chunk is longer than it is, gets length 0,
// which the attention reports and skips.
#pragma once

#include <stdint.h>

#include "internal.h"
#include "plan.cuh"

namespace ira {

constexpr int kRowThreads = 256;

struct ExpandParams {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* page_table;
  const int32_t* cu;
  const int32_t* seq_lens;
  uint4* k_out;  // [B * pages_per_seq][64][H_kv][D / 8]
  uint4* v_out;
  int32_t* table_out;  // [B][pages_per_seq]
  int32_t* lens_out;   // [B]
  int32_t* dev_err;
  int B, H_kv, P, num_pages, pt_stride, window, pages_per_seq;
};

constexpr int kExpandTokens = 16;  // tokens per block of the grid
constexpr int kExpandBlocks = 2;   // blocks that share the heads of these tokens (4-bit, local chunk 302.0 -> 299.3 us)

// F::block_bytes(D), and F::read8<D>(kb, vb, have, r, i, k, v): the 8 K and 8 V channels from
// 8 i on of row r of the blocks at kb, vb, as bf16; all lanes of a warp call it together.
template <class F, int D>
__device__ __forceinline__ void expand_blocks(const ExpandParams& p) {
  constexpr int U = D / 8;
  const int b = blockIdx.y;
  const int q_len = p.cu[b + 1] - p.cu[b];
  const int L_in = p.seq_lens[b];
  const int L = min(max(L_in, 0), p.pt_stride * p.P);
  const int lo = p.window > 0 ? max(0, L - q_len - p.window + 1) : 0;
  const int base = lo & ~63;
  const bool fits = q_len > 0 && q_len <= L && L - base <= p.pages_per_seq * 64;
  if (blockIdx.x == 0 && blockIdx.z == 0) {
    if (threadIdx.x == 0) {
      p.lens_out[b] = fits ? L - base : 0;
      if (L_in > L || (q_len > 0 && q_len <= L && !fits)) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
    }
    for (int i = threadIdx.x; i < p.pages_per_seq; i += kRowThreads)
      p.table_out[(size_t)b * p.pages_per_seq + i] = b * p.pages_per_seq + i;
  }
  const int j0 = base + (int)blockIdx.x * kExpandTokens;  // all in one 16-token block of the cache
  if (!fits || j0 >= L || j0 + kExpandTokens <= lo) return;  // keys before lo are not attended to: their page may be gone
  const int lp = j0 / p.P;
  const int page = p.page_table[(size_t)b * p.pt_stride + lp];
  const bool ok = page >= 0 && page < p.num_pages;
  if (!ok && threadIdx.x == 0) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
  // thread: 8 channels of one row, head after head (with D = 64 half of the block has every other head)
  constexpr int kHeads = kRowThreads / (kExpandTokens * U);
  const int i = threadIdx.x % U, r = threadIdx.x / U % kExpandTokens;
  const bool in = r < L - j0;
  const size_t block = (size_t)(p.P / 16) * F::block_bytes(D);  // from one head's first block to the next's
  const size_t at = (((size_t)(ok ? page : 0) * p.H_kv) * (p.P / 16) + (j0 - lp * p.P) / 16) * F::block_bytes(D);
  const size_t dst = ((size_t)b * p.pages_per_seq * 64 + (j0 - base) + r) * p.H_kv * U + i;
#pragma unroll 4
  for (int h0 = kHeads * blockIdx.z; h0 < p.H_kv; h0 += kHeads * gridDim.z) {
    const int h = h0 + threadIdx.x / (kExpandTokens * U);
    const bool mine = in && h < p.H_kv;
    const size_t src = at + (size_t)h * block;
    uint4 k, v;
    F::template read8<D>(p.k_cache + src, p.v_cache + src, ok && mine, r, i, k, v);
    if (mine) {
      p.k_out[dst + (size_t)h * U] = k;
      p.v_out[dst + (size_t)h * U] = v;
    }
  }
}

inline ExpandParams expand_params(const ExpandCall& c) {
  ExpandParams p;
  p.k_cache = static_cast<const uint8_t*>(c.k_cache);
  p.v_cache = static_cast<const uint8_t*>(c.v_cache);
  p.page_table = c.page_table;
  p.cu = c.cu_seqlens_q;
  p.seq_lens = c.seq_lens;
  p.k_out = static_cast<uint4*>(c.k_out);
  p.v_out = static_cast<uint4*>(c.v_out);
  p.table_out = c.table_out;
  p.lens_out = c.lens_out;
  p.dev_err = c.dev_err;
  p.B = c.B;
  p.H_kv = c.H_kv;
  p.P = c.P;
  p.num_pages = c.num_pages;
  p.pt_stride = c.pt_stride;
  p.window = c.window;
  p.pages_per_seq = c.pages_per_seq;
  return p;
}
inline dim3 expand_grid(const ExpandCall& c) {
  return dim3((unsigned)(c.pages_per_seq * (64 / kExpandTokens)), (unsigned)c.B, kExpandBlocks);
}

}  // namespace ira

// The 4-bit cache's rows: quantising append, read-back, and the expansion of
// the visible part of a batch's sequences into bf16 pages for prefill.
//
// Operations: inkling_rel_attn_kv_append_q4, inkling_rel_attn_kv_read_q4 and
// the first step of inkling_rel_attn_prefill_q4 in include/inkling_rel_attn.h.
//
// All three move rows and are bound by HBM.  A thread owns 8 adjacent channels
// of K and the same 8 of V: 16 bytes each on the bf16 side, one 32-bit word
// each on the 4-bit side; 4 adjacent lanes share a group and its scale, D / 8
// lanes a row.  A block of the grid has one KV head of 2048 / D adjacent tokens:
// its rows follow from the thread's number without a division, and tokens that
// are neighbours in the cache, as a chunk's are, fill whole blocks of it.
// Append and read-back of 8192 tokens x 16 heads, D = 128: 30 us for 172 MB, 0.85 of
// the measured copy rate; what bounds them beside HBM is the quantiser's instructions.
#include <cuda_runtime.h>
#include <stdint.h>

#include "async.cuh"
#include "expand.cuh"
#include "internal.h"
#include "launch.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "q4.cuh"

namespace ira {

constexpr int kQ4Heads = 2;           // heads per thread of a large call (8192 tokens x 16 heads both ways: 30 us; 1: 33.7, 4: 31.9)
constexpr int kRowsFill = 4;          // such blocks per SM from which on it is taken

struct Q4RowsParams {
  uint4* k_rows;  // [T][H_kv][D / 8] of 8 x bf16
  uint4* v_rows;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int64_t* slots;
  int32_t* dev_err;
  uint64_t inv_P;  // 2^64 / P rounded up: slots below 2^31 * 256 divide by the high half of a product
  int T, H_kv, P, num_pages;
};

__device__ __forceinline__ size_t q4_slot_at(const Q4RowsParams& p, int64_t slot, int h, int D, int& r) {
  const int page = (int)__umul64hi((uint64_t)slot, p.inv_P);
  const int place = (int)(slot - (int64_t)page * p.P);
  r = place % kQ4Block;
  return q4_block_at(page, h, place, p.H_kv, p.P, D);
}

// Word of a V row that this lane stores: lane i (group j = i / 4, t = i % 4)
// holds the 16-bit units (g = 2t, j) and (2t + 1, j) of the row; a word has the
// units (g, j) and (g, j + 1), j even.  The lanes of groups j and j + 1 swap
// one unit each: the even one then has word (2t, j), the odd one (2t + 1, j - 1).
template <int D>
__device__ __forceinline__ int v_word(int j, int t) {
  constexpr int N = D / kQ4Group;
  return (N * (2 * t + (j & 1)) + (j & ~1)) >> 1;
}
__device__ __forceinline__ uint32_t v_swap(uint32_t units, int j) {
  const uint32_t other = __shfl_xor_sync(0xffffffffu, units, 4);
  return (j & 1) ? __byte_perm(other, units, 0x7632) : __byte_perm(units, other, 0x5410);
}

template <int D, int HEADS>
__global__ void __launch_bounds__(kRowThreads)
    kv_append_q4_kernel(const __grid_constant__ Q4RowsParams p) {
  await_previous_kernel();
  constexpr int N = D / kQ4Group;
  constexpr int U = D / 8;  // lanes per row
  const int t_row = blockIdx.x * (kRowThreads / U) + threadIdx.x / U, h0 = blockIdx.y * HEADS;
  const int i = threadIdx.x % U, j = i >> 2, t = i & 3;
  uint4 kr[HEADS], vr[HEADS];
  int64_t slot = -1;
  if (t_row < p.T) slot = p.slots[t_row];
#pragma unroll
  for (int x = 0; x < HEADS; ++x) {
    kr[x] = vr[x] = make_uint4(0, 0, 0, 0);
    if (t_row < p.T && h0 + x < p.H_kv) {
      const size_t idx = ((size_t)t_row * p.H_kv + h0 + x) * U + i;
      kr[x] = __ldcs(p.k_rows + idx);
      vr[x] = __ldcs(p.v_rows + idx);
    }
  }
  if (slot >= (int64_t)p.num_pages * p.P) {
    report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
    slot = -1;
  }
  int r = 0;
  size_t at = slot < 0 ? 0 : q4_slot_at(p, slot, h0, D, r);
  const size_t head = q4_block_at(0, 1, 0, 1, p.P, D);  // from a head's block to the next head's
#pragma unroll
  for (int x = 0; x < HEADS; ++x, at += head) {
    uint32_t ks, vs;
    const uint32_t kw = q4_quantise8(kr[x], ks);
    const uint32_t vw = v_swap(q4_quantise8(vr[x], vs), j);
    if (slot < 0 || h0 + x >= p.H_kv) continue;
    uint8_t* kb = p.k_cache + at;
    uint8_t* vb = p.v_cache + at;
    reinterpret_cast<uint32_t*>(kb + r * (D / 2))[N * t + j] = kw;
    reinterpret_cast<uint32_t*>(vb + r * (D / 2))[v_word<D>(j, t)] = vw;
    if (t == 0) {
      reinterpret_cast<uint16_t*>(kb + q4_scale_off(D))[r * N + j] = (uint16_t)ks;
      reinterpret_cast<uint16_t*>(vb + q4_scale_off(D))[r * N + j] = (uint16_t)vs;
    }
  }
}

// The 8 K and 8 V channels (group j, quarter t) of row r of the blocks at kb, vb, as bf16;
// zeros without a block.  All lanes of a warp call it together (V words are swapped).
template <int D>
__device__ __forceinline__ void q4_read8(const uint8_t* kb, const uint8_t* vb, bool have, int r, int j, int t,
                                         uint4& k, uint4& v) {
  constexpr int N = D / kQ4Group;
  uint32_t kw = 0, vw = 0, ks = 0, vs = 0;
  if (have) {
    kw = reinterpret_cast<const uint32_t*>(kb + r * (D / 2))[N * t + j];
    vw = reinterpret_cast<const uint32_t*>(vb + r * (D / 2))[v_word<D>(j, t)];
    ks = reinterpret_cast<const uint16_t*>(kb + q4_scale_off(D))[r * N + j];
    vs = reinterpret_cast<const uint16_t*>(vb + q4_scale_off(D))[r * N + j];
  }
  k = q4_values8(kw, ks);
  v = q4_values8(v_swap(vw, j), vs);
  if (!have) k = v = make_uint4(0, 0, 0, 0);
}

template <int D, int HEADS>
__global__ void __launch_bounds__(kRowThreads)
    kv_read_q4_kernel(const __grid_constant__ Q4RowsParams p) {
  await_previous_kernel();
  constexpr int U = D / 8;
  const int t_row = blockIdx.x * (kRowThreads / U) + threadIdx.x / U, h0 = blockIdx.y * HEADS;
  const int i = threadIdx.x % U;
  int64_t slot = t_row < p.T ? p.slots[t_row] : -1;
  if (slot >= (int64_t)p.num_pages * p.P) {
    report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
    slot = -1;
  }
  int r = 0;
  const size_t at = slot >= 0 ? q4_slot_at(p, slot, h0, D, r) : 0;
  const size_t head = q4_block_at(0, 1, 0, 1, p.P, D);
  uint4 k[HEADS], v[HEADS];
#pragma unroll
  for (int x = 0; x < HEADS; ++x)
    q4_read8<D>(p.k_cache + at + x * head, p.v_cache + at + x * head, slot >= 0 && h0 + x < p.H_kv, r, i >> 2, i & 3,
                k[x], v[x]);
  if (t_row >= p.T) return;
#pragma unroll
  for (int x = 0; x < HEADS; ++x) {
    if (h0 + x >= p.H_kv) return;
    const size_t idx = ((size_t)t_row * p.H_kv + h0 + x) * U + i;
    p.k_rows[idx] = k[x];
    p.v_rows[idx] = v[x];
  }
}

static Q4RowsParams rows_params(const RowsCall& c) {
  Q4RowsParams p;
  p.k_rows = static_cast<uint4*>(c.k_rows);
  p.v_rows = static_cast<uint4*>(c.v_rows);
  p.k_cache = static_cast<uint8_t*>(c.k_cache);
  p.v_cache = static_cast<uint8_t*>(c.v_cache);
  p.slots = c.slots;
  p.dev_err = c.dev_err;
  p.T = c.T;
  p.H_kv = c.H_kv;
  p.P = c.P;
  p.num_pages = c.num_pages;
  p.inv_P = ~0ull / (uint64_t)c.P + 1;  // P >= 16: exact for powers of two, rounded up for the others
  return p;
}

template <int D, int HEADS>
static bool rows_launch(const Q4RowsParams& p, bool append, cudaStream_t stream) {
  constexpr int kTokens = kRowThreads / (D / 8);
  const dim3 g((unsigned)(((int64_t)p.T + kTokens - 1) / kTokens), (unsigned)((p.H_kv + HEADS - 1) / HEADS));
  return append ? launch_dependent(kv_append_q4_kernel<D, HEADS>, g, kRowThreads, 0, p, stream)
                : launch_dependent(kv_read_q4_kernel<D, HEADS>, g, kRowThreads, 0, p, stream);
}

int launch_q4_rows(const RowsCall& c, bool append) {
  const Q4RowsParams p = rows_params(c);
  // Several heads per thread share its place in the cache; a call that could not fill
  // the GPU so is latency-bound and takes a head per thread.  Append and read, blocks at
  // one head a thread, 152 SMs (border 1216): 128 blocks 3.07 us with one head and 3.65
  // with two, 512: 4.2 and 4.5, 1024: 6.75 and 7.2, 2048: 10.7 and 10.7, 4096: 17.9 and 16.3.
  const bool many = (int64_t)c.T * c.H_kv * (c.D / 8) >= (int64_t)kQ4Heads * kRowThreads * kRowsFill * device_info().sms;
  const bool ok =
      c.D == 128
          ? (many ? rows_launch<128, kQ4Heads>(p, append, c.stream) : rows_launch<128, 1>(p, append, c.stream))
          : (many ? rows_launch<64, kQ4Heads>(p, append, c.stream) : rows_launch<64, 1>(p, append, c.stream));
  return ok ? INKLING_OK : INKLING_ERR_CUDA;
}

// ---------------------------------------------------------------------------
// Expansion for prefill (expand.cuh)
struct Q4ReadFormat {
  __host__ __device__ static constexpr int block_bytes(int D) { return q4_block_bytes(D); }
  template <int D>
  __device__ static __forceinline__ void read8(const uint8_t* kb, const uint8_t* vb, bool have, int r, int i, uint4& k,
                                               uint4& v) {
    q4_read8<D>(kb, vb, have, r, i >> 2, i & 3, k, v);
  }
};

template <int D>
__global__ void __launch_bounds__(kRowThreads)
    q4_expand_kernel(const __grid_constant__ ExpandParams p) {
  await_previous_kernel();
  expand_blocks<Q4ReadFormat, D>(p);
}

int launch_q4_expand(const ExpandCall& c) {
  const ExpandParams p = expand_params(c);
  const bool ok = c.D == 128 ? launch_dependent(q4_expand_kernel<128>, expand_grid(c), kRowThreads, 0, p, c.stream)
                             : launch_dependent(q4_expand_kernel<64>, expand_grid(c), kRowThreads, 0, p, c.stream);
  return ok ? INKLING_OK : INKLING_ERR_CUDA;
}

}  // namespace ira

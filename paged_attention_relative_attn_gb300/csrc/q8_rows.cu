// The 8-bit cache's rows: quantising append, read-back, and the expansion of
// the visible part of a batch's sequences into bf16 pages for prefill.
//
// Operations: inkling_rel_attn_kv_append_q8, inkling_rel_attn_kv_read_q8 and
// the first step of inkling_rel_attn_prefill_q8 in include/inkling_rel_attn.h.
//
// All three move rows and are bound by HBM.
//
// Append.  What is written together is a block: its exponent comes from all of its
// rows.  The tokens that join a block lie within 16 of the call; the first of them
// leads.  A warp looks at a window of tokens, the 16 before and the 16 behind it (two
// loads), and for each leader in the window takes its tokens' rows of one KV head of K
// or V: the rows into registers (16 bytes a lane), their largest magnitude by one
// reduction, the block's scale as it was, and out go 8 bytes a lane.  Nothing but the
// one warp touches a block, so no atomic is needed and the result does not depend on
// timing.  Rows that the block has already are read only when its exponent grows.
// 8192 tokens x 16 heads, D = 128: 20.8 us for 101 MB, 0.71 of the measured copy rate (K
// and V by one warp, which then holds twice the registers: 24.0).
#include <cuda_runtime.h>
#include <stdint.h>

#include "async.cuh"
#include "expand.cuh"
#include "internal.h"
#include "launch.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "q8.cuh"

namespace ira {

struct Q8RowsParams {
  uint4* k_rows;  // [T][H_kv][D / 8] of 8 x bf16
  uint4* v_rows;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int64_t* slots;
  int32_t* dev_err;
  uint64_t inv_P;  // 2^64 / P rounded up: slots below 2^31 * 256 divide by the high half of a product
  int T, H_kv, P, num_pages;
};

__device__ __forceinline__ size_t q8_slot_at(const Q8RowsParams& p, int64_t slot, int h, int D) {
  const int page = (int)__umul64hi((uint64_t)slot, p.inv_P);
  return q8_block_at(page, h, (int)(slot - (int64_t)page * p.P), p.H_kv, p.P, D);
}

// Rows of a run of tokens join the block at `blk` (K or V).  raw[i]: 16 bytes of row RP * i + lane / U
// of the run; place[i]: that row's place in the block; joins: all their places.
template <int D, bool IS_V>
__device__ __forceinline__ void q8_join(uint8_t* blk, const uint4 (&raw)[D / 16], const int (&place)[D / 16], int len,
                                        uint32_t joins) {
  constexpr int U = D / 8, RP = 32 / U, N = 16 / RP;  // lanes per row, rows per step, steps
  const int lane = threadIdx.x & 31, u = lane % U;
  const bool begins = joins & 1u;  // place 0 is among them
  const uint2 tail = begins ? make_uint2(0u, 0u) : *reinterpret_cast<const uint2*>(blk + q8_tail_off(D));
  // rows with a NaN, and the largest magnitude of the others
  uint32_t nan_rows = 0, most = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (RP * i >= len) break;
    const uint4 v = raw[i];
    const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                 __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    const uint32_t m = max(m2 & 0xffffu, m2 >> 16);
    const uint32_t bad = __ballot_sync(0xffffffffu, m > 0x7f80u);
    const bool row_bad = ((bad >> (lane - u)) & ((1u << (U - 1) << 1) - 1u)) != 0u;
    if (row_bad) nan_rows |= 1u << place[i];
    else most = max(most, m);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  nan_rows = __reduce_or_sync(0xffffffffu, nan_rows);
  const int e_old = begins ? kQ8MinExp - 1 : q8_exp(tail.x);
  const bool begun = e_old >= kQ8MinExp;
  const int e = max(q8_exp_for(most), e_old);
  const float f = __uint_as_float(q8_scale_bits(-e));
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (RP * i + lane / U >= len) continue;
    uint2 x = q8_quantise8(raw[i], f);
    if ((nan_rows >> place[i]) & 1u) x = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(blk + q8_unit_at<D, IS_V>(place[i], u)) = x;
  }
  if (begun && e > e_old) {  // the rows that are there: their values, rounded again
    const uint32_t down = f16x2_pow2_down(e - e_old);
#pragma unroll 4
    for (int r = lane / U; r < kQ8Block; r += RP) {
      if ((joins >> r) & 1u) continue;
      uint2* at = reinterpret_cast<uint2*>(blk + q8_unit_at<D, IS_V>(r, u));
      uint2 x = *at;
      x.x = q8_rescale4(x.x, down);
      x.y = q8_rescale4(x.y, down);
      *at = x;
    }
  }
  const uint32_t flags = (begun ? tail.y & 0xffffu & ~joins : 0u) | nan_rows;
  if (lane == 0 && (!begun || e > e_old || flags != tail.y))
    *reinterpret_cast<uint4*>(blk + q8_tail_off(D)) = make_uint4(q8_scale_bits(e), flags, 0u, 0u);
}

constexpr int kAppendThreads = 128;

// WIN: tokens whose leaders a warp looks after.
template <int D, int WIN, bool IS_V>
__device__ __forceinline__ void append_side(const Q8RowsParams& p, const uint4* rows, uint8_t* cache) {
  constexpr int U = D / 8, RP = 32 / U, N = 16 / RP;
  static_assert(N == D / 16, "steps of a block");
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const int64_t t0 = ((int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5)) * WIN;
  if (t0 >= p.T) return;
  // blocks of the 32 tokens that end with the window, and slots of the 32 that begin with it
  auto slot_of = [&](int64_t t, bool tell) {
    int64_t s = t >= 0 && t < p.T ? p.slots[t] : -1;
    if (s >= (int64_t)p.num_pages * p.P) {
      if (tell) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
      s = -1;
    }
    return s;
  };
  const int64_t back = slot_of(t0 + WIN - 32 + lane, false), slot = slot_of(t0 + lane, lane < WIN && h == 0 && !IS_V);
  // (a skipped token's slot is negative, and so is this number of its block)
  const uint32_t alike = __match_any_sync(0xffffffffu, back >> 4);
  uint32_t leaders = __ballot_sync(0xffffffffu, lane >= 32 - WIN && back >= 0 && __ffs(alike) - 1 == lane);
  while (leaders != 0u) {
    const int l = __ffs(leaders) - 1 - (32 - WIN);  // of the window's tokens
    leaders &= leaders - 1;
    const int64_t first = __shfl_sync(0xffffffffu, slot, l);
    uint32_t run = __ballot_sync(0xffffffffu, slot >> 4 == first >> 4);  // its tokens, from l on
    const uint32_t behind = run + (run & (0u - run));
    const bool dense = (run & behind) == 0u;  // next to each other
    const int len = min(__popc(run), kQ8Block);
    const uint32_t joins = __reduce_or_sync(0xffffffffu, (run >> lane) & 1u ? 1u << (slot & 15) : 0u);
    uint4 raw[N];
    int place[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int k = RP * i + lane / U;
      const int at_lane = k >= len ? l : dense ? l + k : (int)__fns(run, 0, k + 1);
      place[i] = (int)__shfl_sync(0xffffffffu, (int)(slot & 15), at_lane);
      raw[i] = make_uint4(0, 0, 0, 0);
      if (k < len) {
        const size_t at = ((size_t)(t0 + at_lane) * p.H_kv + h) * U + lane % U;
        raw[i] = __ldcs(rows + at);
      }
    }
    q8_join<D, IS_V>(cache + q8_slot_at(p, first, h, D), raw, place, len, joins);
  }
}

template <int D, int WIN>
__global__ void __launch_bounds__(kAppendThreads)
    kv_append_q8_kernel(const __grid_constant__ Q8RowsParams p) {
  await_previous_kernel();
  if (blockIdx.z == 0) append_side<D, WIN, false>(p, p.k_rows, p.k_cache);
  else append_side<D, WIN, true>(p, p.v_rows, p.v_cache);
}

// The 8 K and 8 V channels of unit u of row r of the blocks at kb, vb, as bf16; zeros without a block.
struct Q8ReadFormat {
  __host__ __device__ static constexpr int block_bytes(int D) { return q8_block_bytes(D); }
  template <int D, bool IS_V>
  __device__ static __forceinline__ uint4 side(const uint8_t* blk, bool have, int r, int u) {
    uint2 w = make_uint2(0, 0), tail = make_uint2(0, 0);
    if (have) {
      w = *reinterpret_cast<const uint2*>(blk + q8_unit_at<D, IS_V>(r, u));
      tail = *reinterpret_cast<const uint2*>(blk + q8_tail_off(D));
    }
    const float s = __uint_as_float(tail.x);
    const uint2 a = q8_values4(w.x, s), b = q8_values4(w.y, s);
    if ((tail.y >> r) & 1u) return make_uint4(0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  template <int D>
  __device__ static __forceinline__ void read8(const uint8_t* kb, const uint8_t* vb, bool have, int r, int u, uint4& k,
                                               uint4& v) {
    k = side<D, false>(kb, have, r, u);
    v = side<D, true>(vb, have, r, u);
  }
};

constexpr int kReadHeads = 2;  // of a large call (8192 tokens x 16 heads, D = 128: 17.6 us; 1: 18.4, 4: 19.8)

// HEADS: heads per thread, which share the token's place in the cache.
template <int D, int HEADS>
__global__ void __launch_bounds__(kRowThreads)
    kv_read_q8_kernel(const __grid_constant__ Q8RowsParams p) {
  await_previous_kernel();
  constexpr int U = D / 8;
  const int64_t t_row = (int64_t)blockIdx.x * (kRowThreads / U) + threadIdx.x / U;
  const int h0 = blockIdx.y * HEADS, u = threadIdx.x % U;
  if (t_row >= p.T) return;
  int64_t slot = p.slots[t_row];
  if (slot >= (int64_t)p.num_pages * p.P) {
    report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
    slot = -1;
  }
  const size_t at = slot >= 0 ? q8_slot_at(p, slot, h0, D) : 0;
  const size_t head = (size_t)(p.P / kQ8Block) * q8_block_bytes(D);  // from a head's block to the next head's
  uint4 k[HEADS], v[HEADS];
#pragma unroll
  for (int x = 0; x < HEADS; ++x)
    Q8ReadFormat::read8<D>(p.k_cache + at + x * head, p.v_cache + at + x * head, slot >= 0 && h0 + x < p.H_kv,
                           (int)(slot & 15), u, k[x], v[x]);
#pragma unroll
  for (int x = 0; x < HEADS; ++x) {
    if (h0 + x >= p.H_kv) return;
    const size_t to = ((size_t)t_row * p.H_kv + h0 + x) * U + u;
    p.k_rows[to] = k[x];
    p.v_rows[to] = v[x];
  }
}

template <int D>
static bool rows_launch(const Q8RowsParams& p, bool append, cudaStream_t stream) {
  if (!append) {
    constexpr int kTokens = kRowThreads / (D / 8);
    // one head and two, D = 128: 16384 rows 4.0 and 4.2 us, 32768: 6.1 and 6.0; 40960 of D = 64: 4.6 and 5.2
    const bool many = (int64_t)p.T * p.H_kv * (D / 8) >= 32768 * 16;
    const int heads = many ? kReadHeads : 1;
    const dim3 g((unsigned)(((int64_t)p.T + kTokens - 1) / kTokens), (unsigned)((p.H_kv + heads - 1) / heads));
    return many ? launch_dependent(kv_read_q8_kernel<D, kReadHeads>, g, kRowThreads, 0, p, stream)
                : launch_dependent(kv_read_q8_kernel<D, 1>, g, kRowThreads, 0, p, stream);
  }
  constexpr int kWarps = kAppendThreads / 32;
  auto grid = [&](int win) {
    const int64_t windows = ((int64_t)p.T + win - 1) / win;
    return dim3((unsigned)((windows + kWarps - 1) / kWarps), (unsigned)p.H_kv, 2);
  };
  // Wide windows leave few warps without a block of their own, but take single tokens, as a decode
  // step's are, one after the other.  us with windows of 1, 4, 8 tokens (152 SMs, D = 128): 512
  // (token, head) pairs of single tokens 3.0, 5.6, 9.8; 2048: 5.0, 7.1, 10.2; 8192: 16.2, 12.1, 16.1; of runs of
  // tokens 2048: 3.5, 3.0, 2.8; 8192: 6.4, 4.0, 4.0; 16384: 10.4, 6.4, 5.0; 131072: -, 24.4, 20.8.
  const int64_t pairs = (int64_t)p.T * p.H_kv;
  return pairs >= 16384  ? launch_dependent(kv_append_q8_kernel<D, 8>, grid(8), kAppendThreads, 0, p, stream)
         : pairs >= 4096 ? launch_dependent(kv_append_q8_kernel<D, 4>, grid(4), kAppendThreads, 0, p, stream)
                         : launch_dependent(kv_append_q8_kernel<D, 1>, grid(1), kAppendThreads, 0, p, stream);
}

int launch_q8_rows(const RowsCall& c, bool append) {
  Q8RowsParams p;
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
  const bool ok = c.D == 128 ? rows_launch<128>(p, append, c.stream) : rows_launch<64>(p, append, c.stream);
  return ok ? INKLING_OK : INKLING_ERR_CUDA;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads)
    q8_expand_kernel(const __grid_constant__ ExpandParams p) {
  await_previous_kernel();
  expand_blocks<Q8ReadFormat, D>(p);
}

int launch_q8_expand(const ExpandCall& c) {
  const ExpandParams p = expand_params(c);
  const bool ok = c.D == 128 ? launch_dependent(q8_expand_kernel<128>, expand_grid(c), kRowThreads, 0, p, c.stream)
                             : launch_dependent(q8_expand_kernel<64>, expand_grid(c), kRowThreads, 0, p, c.stream);
  return ok ? INKLING_OK : INKLING_ERR_CUDA;
}

}  // namespace ira

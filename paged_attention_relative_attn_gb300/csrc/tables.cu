// The tables of a serving step, built from request lengths.
//
// Operation: inkling_rel_attn_build_tables in include/inkling_rel_attn.h.
//
// Three prefix sums over the batch (new tokens, pages returned, pages taken)
// fix everything: where a request's tokens start, which part of the free stack
// its returned pages go to and which part its new pages come from.  Pages and
// slots follow without any atomic, so the result does not depend on timing.
//
// Latency-bound: a few KB are touched, so what counts is the number of memory
// round trips in a row.  A page taken in the step in which it came back is
// looked up in the row that returned it, not on the stack, so nothing reads
// what the step writes: after the sums, returned pages, taken pages and slots
// are independent.  A cluster of up to 8 blocks does the step.  Every block
// makes the sums for itself; block 0 moves the pages, the others share the
// slots.  One cluster barrier keeps the lengths, which may be updated in
// place, from changing before every block has read them.  128 decoding requests
// take 4.5 us (one block that went through the stack in memory: 7.9), 256 requests
// with 16384 slots 6.4 us (17.8).
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "async.cuh"
#include "internal.h"
#include "launch.h"
#include "plan.cuh"
#include "ptx.cuh"

namespace ira {

constexpr int kTabThreads = 1024;

struct TablesParams {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* page_table;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* kv_lens;
  int32_t* cu;
  int64_t* slot_map;
  int32_t* free_left;
  int32_t* step_lens;
  int32_t* dev_err;
  uint64_t inv_P;  // 2^64 / P rounded up: lengths divide by the high half of a product
  int B, pt_stride, P, num_pages, max_tokens;
};

// Sums stop at 2^31 - 1 (a batch may ask for any int32 each): there they are past
// every limit they are compared with, and which sums came first makes no difference.
struct Sum3 {
  uint32_t n, gone, need;
};
__device__ __forceinline__ uint32_t sat(uint32_t a, uint32_t b) { return min(a + b, 0x7fffffffu); }
__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) {
  return {sat(a.n, b.n), sat(a.gone, b.gone), sat(a.need, b.need)};
}

__device__ __forceinline__ int pages_of(const TablesParams& p, int tokens) {  // tokens <= stride * P < 2^31
  return (int)__umul64hi((uint64_t)((uint32_t)tokens + (uint32_t)p.P - 1), p.inv_P);
}

// What a request asks for.
struct Ask {
  int L, n;
  uint32_t gone, need;
  bool bad;  // its row cannot hold it: refused
};
__device__ __forceinline__ Ask ask_of(const TablesParams& p, int Lr, int n) {
  Ask a;
  const int cap = p.pt_stride * p.P;
  a.L = min(max(Lr, 0), cap);
  a.n = max(n, 0);
  const int had = pages_of(p, a.L);
  a.bad = n >= 0 && (Lr != a.L || a.n > cap - a.L);
  a.gone = n < 0 ? had : 0;
  a.need = n >= 0 && !a.bad ? pages_of(p, a.L + a.n) - had : 0;
  return a;
}

// Largest i < n with a[i] <= x; a does not decrease and a[0] <= x.
__device__ __forceinline__ int last_at_most(const int32_t* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// (1 block per SM: without it the compiler keeps to 32 registers and spills; 5.0 us instead of 4.55)
__global__ void __launch_bounds__(kTabThreads, 1)
    build_tables_kernel(const __grid_constant__ TablesParams p) {
  await_previous_kernel();
  extern __shared__ int32_t sm[];
  int32_t* cu = sm;                // [B + 1] first token of each request
  int32_t* back = cu + p.B + 1;    // [B] rank of its first returned page
  int32_t* first = back + p.B;     // [B] rank of its first new page; -1: refused
  int32_t* lens = first + p.B;     // [B] tokens before the step
  __shared__ uint4 wsum[32];
  __shared__ int s_used;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool mover = blockIdx.x == 0;  // moves pages and lengths; the other blocks make the slots

  // ---- prefix sums: each thread a run of requests, then over the block
  const int count = *p.free_count;
  const int per = (p.B + kTabThreads - 1) / kTabThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  const int warps = per == 0 ? 0 : (p.B + 32 * per - 1) / (32 * per);  // those that have requests
  Sum3 mine = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const Ask a = ask_of(p, p.seq_lens[b], p.new_lens[b]);
    mine = mine + Sum3{(uint32_t)a.n, a.gone, a.need};
  }
  Sum3 before = {0, 0, 0};  // of the warp's threads before this one
  if (warp < warps) {
    Sum3 incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const Sum3 o = {__shfl_up_sync(0xffffffffu, incl.n, off), __shfl_up_sync(0xffffffffu, incl.gone, off),
                      __shfl_up_sync(0xffffffffu, incl.need, off)};
      if (lane >= off) incl = incl + o;
    }
    before = {__shfl_up_sync(0xffffffffu, incl.n, 1), __shfl_up_sync(0xffffffffu, incl.gone, 1),
              __shfl_up_sync(0xffffffffu, incl.need, 1)};
    if (lane == 0) before = {0, 0, 0};
    if (lane == 31) wsum[warp] = make_uint4(incl.n, incl.gone, incl.need, 0);
  }
  if (tid == 0) s_used = 0;
  __syncthreads();
  Sum3 at = {0, 0, 0}, all = {0, 0, 0};
  for (int w = 0; w < warps; ++w) {
    if (w == warp) at = all;
    const uint4 s = wsum[w];
    all = all + Sum3{s.x, s.y, s.z};
  }
  at = at + before;
  const int F = min(max(count, 0), p.num_pages);
  const int top = (int)min((uint32_t)F + all.gone, (uint32_t)p.num_pages);  // the stack once pages have come back
  int used = 0;
  const bool packed = all.n < 0x7fffffffu;  // else offsets have stopped, and the slot map's length decides nothing
  for (int b = b0; b < b1; ++b) {
    const Ask a = ask_of(p, p.seq_lens[b], p.new_lens[b]);
    const bool room = !packed || a.n == 0 || at.n + a.n <= (uint32_t)p.max_tokens;  // a slot for each of its tokens
    // (requests after one without room have none either, so pages taken still are a prefix of those asked for)
    const bool served = !a.bad && room && (a.need == 0 || at.need + a.need <= (uint32_t)top);
    cu[b] = (int)at.n;
    back[b] = (int)at.gone;
    first[b] = served ? (int)min(at.need, (uint32_t)top) : -1;
    lens[b] = a.L;
    if (mover) {
      if (a.bad) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
      else if (room && !served) report(p.dev_err, INKLING_DEVERR_NO_PAGES);
    }
    at = at + Sum3{(uint32_t)a.n, a.gone, a.need};
    if (served && a.need > 0) used = (int)at.need;  // served requests that take pages are a prefix
  }
  if (used > 0) atomicMax(&s_used, used);
  if (tid == 0) {
    cu[p.B] = (int)all.n;
    if (mover && all.n > (uint32_t)p.max_tokens) report(p.dev_err, INKLING_DEVERR_BAD_CHUNK);
    if (mover && (uint32_t)F + all.gone > (uint32_t)p.num_pages) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
  }
  __syncthreads();
  cluster_arrive();  // this block has read the lengths

  // The page at place i of the stack: below F from the stack, above from the row that returns it.
  auto stack_page = [&](int i) {
    if (i < F) return p.free_pages[i];
    const int b = last_at_most(back, p.B, i - F);
    return p.page_table[(size_t)b * p.pt_stride + (i - F - back[b])];
  };

  if (mover) {
    // pages come back and are taken from the top: one warp per request
    for (int b = warp; b < p.B; b += kTabThreads / 32) {
      const int n_in = p.new_lens[b], L = lens[b], had = pages_of(p, L);
      int32_t* row = p.page_table + (size_t)b * p.pt_stride;
      if (n_in < 0) {
        for (int c = lane; c < had; c += 32) {
          const int64_t to = (int64_t)F + back[b] + c;
          if (to < p.num_pages) p.free_pages[to] = row[c];
        }
      } else if (first[b] >= 0) {
        const int need = pages_of(p, L + n_in) - had;
        for (int c = lane; c < need; c += 32) {
          const int page = stack_page(top - 1 - (first[b] + c));
          if (page < 0 || page >= p.num_pages) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
          row[had + c] = page;
        }
      }
    }
  }
  // the slot of each new token
  const int makers = max((int)gridDim.x - 1, 1), me = (int)blockIdx.x - (gridDim.x > 1);
  for (int64_t t = (int64_t)me * kTabThreads + tid; me >= 0 && t < p.max_tokens; t += makers * kTabThreads) {
    int64_t slot = -1;
    if (t < cu[p.B]) {
      const int b = last_at_most(cu, p.B, (int)t), i = (int)t - cu[b];
      if (first[b] >= 0 && i < p.new_lens[b]) {
        const int had = pages_of(p, lens[b]);
        const int pos = lens[b] + i, lp = (int)__umul64hi((uint64_t)pos, p.inv_P);
        const int page = lp < had ? p.page_table[(size_t)b * p.pt_stride + lp]
                                  : stack_page(top - 1 - (first[b] + lp - had));
        if (page >= 0 && page < p.num_pages) slot = (int64_t)page * p.P + (pos - lp * p.P);
        else report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
      }
    }
    p.slot_map[t] = slot;
  }
  cluster_wait();  // kv_lens may be seq_lens, free_left free_count: every block has read them
  if (!mover) return;
  for (int b = tid; b < p.B; b += kTabThreads) {
    const int n_in = p.new_lens[b];
    const int L_in = p.seq_lens[b];
    const bool served = first[b] >= 0;  // ended requests too
    const int after = n_in < 0 ? 0 : served ? L_in + n_in : L_in;
    p.kv_lens[b] = after;
    if (p.step_lens) p.step_lens[b] = served ? after : 0;
    p.cu[b] = cu[b];
  }
  if (tid == 0) {
    p.cu[p.B] = cu[p.B];
    *p.free_left = top - s_used;
  }
}

int launch_build_tables(const TablesCall& c) {
  TablesParams p;
  p.seq_lens = c.seq_lens;
  p.new_lens = c.new_lens;
  p.page_table = c.page_table;
  p.free_pages = c.free_pages;
  p.free_count = c.free_count;
  p.kv_lens = c.kv_lens;
  p.cu = c.cu_seqlens_q;
  p.slot_map = c.slot_map;
  p.free_left = c.free_left;
  p.step_lens = c.step_lens;
  p.dev_err = c.dev_err;
  p.B = c.B;
  p.pt_stride = c.pt_stride;
  p.P = c.P;
  p.num_pages = c.num_pages;
  p.max_tokens = c.max_tokens;
  p.inv_P = ~0ull / (uint64_t)c.P + 1;
  const int smem = (4 * c.B + 1) * 4;
  static std::atomic<int> limit_set[kMaxDevices];
  constexpr int kMost = (4 * kTablesMaxBatch + 1) * 4;
  if (!smem_limit_on_device(reinterpret_cast<const void*>(build_tables_kernel), kMost, limit_set))
    return INKLING_ERR_CUDA;
  // one block for the pages, and one for every kTabThreads tokens, as many as a cluster may have
  const unsigned blocks = (unsigned)std::min(8, 1 + (int)(((int64_t)c.max_tokens + kTabThreads - 1) / kTabThreads));
  return launch_dependent(build_tables_kernel, dim3(blocks), kTabThreads, smem, p, c.stream, blocks)
             ? INKLING_OK
             : INKLING_ERR_CUDA;
}

}  // namespace ira

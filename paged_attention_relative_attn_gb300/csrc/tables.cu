// The tables of a serving step, built from request lengths.
//
// Operation: inkling_rel_attn_build_tables in include/inkling_rel_attn.h.
//
// Three prefix sums over the batch (new tokens, pages returned, pages taken)
// fix everything: where a request's tokens start, which part of the free stack
// its returned pages go to and which part its new pages come from.  Pages and
// slots follow without any atomic, so the result does not depend on timing.
// Latency-bound: a few KB are touched; the work is one block's.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "plan.cuh"

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
  int32_t* dev_err;
  int B, pt_stride, P, num_pages, max_tokens;
};

struct Sum3 {
  int64_t n, gone, need;  // 64 bits: what a batch asks for may be any int32 each
};
__device__ __forceinline__ Sum3 operator+(const Sum3& a, const Sum3& b) {
  return {a.n + b.n, a.gone + b.gone, a.need + b.need};
}

// What a request asks for.
struct Ask {
  int L, n, had, gone, need;
  bool bad;  // its row cannot hold it: refused
};
__device__ __forceinline__ Ask ask_of(const TablesParams& p, int b) {
  Ask a;
  const int cap = p.pt_stride * p.P;
  const int Lr = p.seq_lens[b], n = p.new_lens[b];
  a.L = min(max(Lr, 0), cap);
  a.n = max(n, 0);
  a.had = (a.L + p.P - 1) / p.P;
  a.bad = n >= 0 && (Lr != a.L || a.n > cap - a.L);
  a.gone = n < 0 ? a.had : 0;
  a.need = n >= 0 && !a.bad ? (a.L + a.n + p.P - 1) / p.P - a.had : 0;
  return a;
}

__global__ void __launch_bounds__(kTabThreads)
    build_tables_kernel(const __grid_constant__ TablesParams p) {
  extern __shared__ int32_t sm[];
  int32_t* cu = sm;                // [B + 1] first token of each request
  int32_t* back = cu + p.B + 1;    // [B] rank of its first returned page
  int32_t* first = back + p.B;     // [B] rank of its first new page; -1: refused
  int32_t* lens = first + p.B;     // [B] tokens before the step
  __shared__ Sum3 wsum[32];
  __shared__ int s_used;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.B + kTabThreads - 1) / kTabThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);

  // ---- prefix sums: each thread a run of requests, then over the block
  Sum3 mine = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const Ask a = ask_of(p, b);
    mine = mine + Sum3{a.n, a.gone, a.need};
  }
  Sum3 incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Sum3 o = {__shfl_up_sync(0xffffffffu, incl.n, off), __shfl_up_sync(0xffffffffu, incl.gone, off),
                    __shfl_up_sync(0xffffffffu, incl.need, off)};
    if (lane >= off) incl = incl + o;
  }
  if (lane == 31) wsum[warp] = incl;
  if (tid == 0) s_used = 0;
  __syncthreads();
  Sum3 at = {incl.n - mine.n, incl.gone - mine.gone, incl.need - mine.need}, all = {0, 0, 0};
  for (int w = 0; w < kTabThreads / 32; ++w) {
    if (w < warp) at = at + wsum[w];
    all = all + wsum[w];
  }
  const int F = min(max(*p.free_count, 0), p.num_pages);
  const int top = (int)min(F + all.gone, (int64_t)p.num_pages);  // the stack's height once pages have come back
  int used = 0;
  for (int b = b0; b < b1; ++b) {
    const Ask a = ask_of(p, b);
    const bool served = !a.bad && (a.need == 0 || at.need + a.need <= top);
    cu[b] = (int)min(at.n, (int64_t)INT32_MAX);
    back[b] = (int)min(at.gone, (int64_t)p.num_pages);
    first[b] = served ? (int)min(at.need, (int64_t)top) : -1;
    lens[b] = a.L;
    if (a.bad) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
    else if (!served) report(p.dev_err, INKLING_DEVERR_NO_PAGES);
    at = at + Sum3{a.n, a.gone, a.need};
    if (served && a.need > 0) used = (int)at.need;  // served requests that take pages are a prefix
  }
  if (used > 0) atomicMax(&s_used, used);
  if (tid == 0) {
    cu[p.B] = (int)min(all.n, (int64_t)INT32_MAX);
    if (all.n > p.max_tokens || F + all.gone > p.num_pages)
      report(p.dev_err, all.n > p.max_tokens ? INKLING_DEVERR_BAD_CHUNK : INKLING_DEVERR_BAD_PAGE);
  }
  __syncthreads();

  // ---- pages come back: one warp per ended request
  for (int b = warp; b < p.B; b += kTabThreads / 32) {
    if (p.new_lens[b] >= 0) continue;
    const int n = (lens[b] + p.P - 1) / p.P;
    for (int c = lane; c < n; c += 32) {
      const int64_t to = (int64_t)F + back[b] + c;
      if (to < p.num_pages) p.free_pages[to] = p.page_table[(size_t)b * p.pt_stride + c];
    }
  }
  __syncthreads();

  // ---- pages are taken from the top, and lengths move on
  for (int b = warp; b < p.B; b += kTabThreads / 32) {
    const int n_in = p.new_lens[b], L = lens[b];
    const bool served = first[b] >= 0;
    if (n_in >= 0 && served) {
      const int had = (L + p.P - 1) / p.P, need = (L + n_in + p.P - 1) / p.P - had;
      for (int c = lane; c < need; c += 32) {
        const int page = p.free_pages[top - 1 - (first[b] + c)];
        if (page < 0 || page >= p.num_pages) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
        p.page_table[(size_t)b * p.pt_stride + had + c] = page;
      }
    }
  }

  // ---- the slot of each new token
  for (int t = tid; t < p.max_tokens; t += kTabThreads) {
    int64_t slot = -1;
    if (t < cu[p.B]) {
      int lo = 0, hi = p.B;  // cu[lo] <= t < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
      }
      if (first[lo] >= 0 && t - cu[lo] < p.new_lens[lo]) {
        const int L = lens[lo], had = (L + p.P - 1) / p.P;
        const int pos = L + t - cu[lo], lp = pos / p.P;
        const int page = lp < had ? p.page_table[(size_t)lo * p.pt_stride + lp]
                                  : p.free_pages[top - 1 - (first[lo] + lp - had)];
        if (page >= 0 && page < p.num_pages) slot = (int64_t)page * p.P + (pos - lp * p.P);
        else report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
      }
    }
    p.slot_map[t] = slot;
  }
  __syncthreads();  // kv_lens may be seq_lens, free_left free_count: every read is done
  for (int b = tid; b < p.B; b += kTabThreads) {
    const int n_in = p.new_lens[b];
    const int L_in = p.seq_lens[b];
    p.kv_lens[b] = n_in < 0 ? 0 : first[b] >= 0 ? L_in + n_in : L_in;
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
  p.dev_err = c.dev_err;
  p.B = c.B;
  p.pt_stride = c.pt_stride;
  p.P = c.P;
  p.num_pages = c.num_pages;
  p.max_tokens = c.max_tokens;
  const int smem = (4 * c.B + 1) * 4;
  static std::atomic<int> limit_set[kMaxDevices];
  constexpr int kMost = (4 * kTablesMaxBatch + 1) * 4;
  if (!smem_limit_on_device(reinterpret_cast<const void*>(build_tables_kernel), kMost, limit_set))
    return INKLING_ERR_CUDA;
  build_tables_kernel<<<1, kTabThreads, smem, c.stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? INKLING_OK : INKLING_ERR_CUDA;
}

}  // namespace ira

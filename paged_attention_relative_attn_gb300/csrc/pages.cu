// Pages of the cache shared between requests: forking, releasing, moving together, copying.
//
// Operations: inkling_rel_attn_fork_pages, inkling_rel_attn_release_pages,
// inkling_rel_attn_compact_pages and inkling_rel_attn_copy_pages in
// include/inkling_rel_attn.h.
//
// The first three move a few KB of whole numbers and are bound by their chains of memory
// round trips and barriers.  Prefix sums over the requests (or over the pages) fix every
// place, so no result depends on timing; the atomics on page_refs and bitmaps are sums,
// minima and unions, which come out the same in any order.  Each is one thread-block cluster or
// one block, since its steps wait for one another.
//
// copy_pages is bound by HBM: thread blocks take equal parts of pages, up to 32 KB each, in turn.
// 1.29 GB both ways, 4 pools of 131 KB pages: 215 us, 6.0 TB/s, 0.88 of the measured copy rate.  (16 KB
// at once 235; a grid of 8 blocks per SM, which leaves some with a part more than others, 226; a ring of bulk
// copies through shared memory 232.)
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "async.cuh"
#include "internal.h"
#include "launch.h"
#include "plan.cuh"
#include "ptx.cuh"

namespace ira {

constexpr int kPgThreads = 1024;
constexpr int kPgWarps = kPgThreads / 32;

struct PagesParams {
  const int32_t* source;    // fork
  const int32_t* seq_lens;
  const int32_t* new_lens;  // release
  int32_t* page_table;
  int32_t* page_refs;       // compact: may be null
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* kv_lens;
  int32_t* src;  // pages to copy, and where to
  int32_t* dst;
  int32_t* count;  // compact: moves; fork, release: the stack's height
  int32_t* dev_err;
  uint64_t inv_P;  // 2^64 / P rounded up: lengths divide by the high half of a product
  int B, pt_stride, P, num_pages;
};

__device__ __forceinline__ int pages_of(const PagesParams& p, int tokens) {  // tokens <= stride * P < 2^31
  return (int)__umul64hi((uint64_t)((uint32_t)tokens + (uint32_t)p.P - 1), p.inv_P);
}
__device__ __forceinline__ bool page_ok(const PagesParams& p, int page) { return page >= 0 && page < p.num_pages; }

// Sum of x over the threads before this one, and over all; scratch: kPgWarps + 1 words.  All threads call it.
__device__ __forceinline__ int scan_block(int x, int* scratch, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += v;
  }
  __syncthreads();  // the scratch of a scan before
  if (lane == 31) scratch[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int v = scratch[lane];
    int s = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, s, off);
      if (lane >= off) s += o;
    }
    scratch[lane] = s - v;
    if (lane == 31) scratch[kPgWarps] = s;
  }
  __syncthreads();
  total = scratch[kPgWarps];
  return scratch[warp] + incl - x;
}

// ---------------------------------------------------------------------------
// Fork.  Rows are shared out over the cluster's warps, which look at the pages of each fork's
// source first: a fork with one that is none becomes a fork of no tokens.  Then every block makes the
// ranks of the requests that need a page, and the rows are written.  3 forks of a short prompt take 3.1 us, 128 of 16
// prompts of 4096 tokens 4.2 (2.8 and 3.4 without the look at the sources).
__device__ __forceinline__ uint32_t cluster_addr(const void* local, uint32_t block) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(local)), "r"(block));
  return r;
}
// Every block's copy of a word of shared memory; a warp calls it.
__device__ __forceinline__ void set_in_cluster(const int32_t* word, int value) {
  const uint32_t block = threadIdx.x & 31;
  if (block < gridDim.x)
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr(word, block)), "r"(value) : "memory");
}

__global__ void __launch_bounds__(kPgThreads, 1) fork_pages_kernel(const __grid_constant__ PagesParams p) {
  extern __shared__ int32_t sm[];
  int32_t* refused = sm;             // [B] not 0: its source has a page that is none
  int32_t* lens = refused + p.B;     // [B] tokens it gets; -1: no fork
  int32_t* source = lens + p.B;      // [B]
  int32_t* page_for = source + p.B;  // [B] the page that it takes; -1: none needed; -2: not served
  __shared__ int scratch[kPgWarps + 1];
  __shared__ int s_used;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w0 = (int)blockIdx.x * kPgWarps + warp, dw = (int)gridDim.x * kPgWarps;
  const bool first = blockIdx.x == 0;
  for (int b = tid; b < p.B; b += kPgThreads) refused[b] = 0;
  if (tid == 0) s_used = 0;
  cluster_arrive();  // waited for where another block's copy is written
  await_previous_kernel();
  const int F = min(max(*p.free_count, 0), p.num_pages), cap = p.pt_stride * p.P;
  const int per = (p.B + kPgThreads - 1) / kPgThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  for (int b = b0; b < b1; ++b) {
    const int from = p.source[b];
    int n = -1;
    if (from >= 0) {
      const bool bad = from >= p.B || p.seq_lens[b] != 0;
      const int L = bad ? 0 : p.seq_lens[from];
      const bool long_ = L > cap;
      if (first && bad) report(p.dev_err, INKLING_DEVERR_BAD_SLOT);
      if (first && long_) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
      if (!bad && !long_) n = max(L, 0);
    }
    lens[b] = n;
    source[b] = from;
  }
  cluster_wait();
  __syncthreads();
  for (int b = w0; b < p.B; b += dw) {
    const int n = lens[b];
    if (n <= 0) continue;
    const int32_t* parent = p.page_table + (size_t)source[b] * p.pt_stride;
    bool none = false;
    const int held = pages_of(p, n);
#pragma unroll 4
    for (int c = lane; c < held; c += 32) none |= !page_ok(p, parent[c]);
    if (!__any_sync(0xffffffffu, none)) continue;
    if (lane == 0) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
    set_in_cluster(refused + b, 1);
  }
  cluster_arrive();  // this block has read the lengths that kv_lens may replace, and the stack's height
  cluster_wait();
  int need = 0;
  for (int b = b0; b < b1; ++b) {
    if (refused[b]) lens[b] = 0;
    need += lens[b] > 0 && lens[b] % p.P != 0 ? 1 : 0;
  }
  int all;
  int at = scan_block(need, scratch, all);
  int used = 0;
  for (int b = b0; b < b1; ++b) {
    page_for[b] = -1;
    if (lens[b] <= 0 || lens[b] % p.P == 0) continue;
    int page = -2;
    if (at < F) {
      used = at + 1;
      page = p.free_pages[F - 1 - at];
      if (!page_ok(p, page)) {  // it leaves the stack all the same
        if (first) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
        page = -2;
      }
    } else if (first) {
      report(p.dev_err, INKLING_DEVERR_NO_PAGES);
    }
    page_for[b] = page;
    ++at;
  }
  if (used > 0) atomicMax(&s_used, used);
  __syncthreads();
  for (int b = w0; b < p.B; b += dw) {
    const int n = lens[b], dst = page_for[b];
    int src = -1;
    if (n > 0 && dst != -2) {
      const int32_t* parent = p.page_table + (size_t)source[b] * p.pt_stride;
      int32_t* row = p.page_table + (size_t)b * p.pt_stride;
      const int full = pages_of(p, n - p.P + 1);  // n / P (n - P + 1 + P - 1 = n)
      for (int c = lane; c < full; c += 32) {
        const int page = parent[c];
        row[c] = page;
        atomicAdd(p.page_refs + page, 1);
      }
      if (dst >= 0) {
        src = parent[full];
        if (lane == 0) row[full] = dst;
      }
    }
    if (lane == 0) {
      p.src[b] = src;
      p.dst[b] = src < 0 ? -1 : dst;
    }
  }
  if (!first) return;
  for (int b = tid; b < p.B; b += kPgThreads)
    p.kv_lens[b] = lens[b] < 0 ? p.seq_lens[b] : page_for[b] == -2 ? 0 : lens[b];
  if (tid == 0) *p.count = F - s_used;
}

// ---------------------------------------------------------------------------
// Release.  Four steps over the entries of the ended rows: the owners of each page are
// counted down; of a page without owners the last entry (the highest, one alone even if a row holds
// the page twice) is found by a minimum over marks in its counter; each row counts the pages
// that it gives back; they go to their places on the stack and their counters to 0.
constexpr int kMark = 1 << 30;  // past every count of entries, at most kReleaseMaxEntries
__device__ __forceinline__ int mark_of(const PagesParams& p, int b, int c) { return -kMark - (b * p.pt_stride + c); }

__global__ void __launch_bounds__(kPgThreads, 1) release_pages_kernel(const __grid_constant__ PagesParams p) {
  await_previous_kernel();
  extern __shared__ int32_t sm[];
  int32_t* back = sm;  // [B] pages that a row gives back, then those before it
  __shared__ int scratch[kPgWarps + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int w0 = (int)blockIdx.x * kPgWarps + warp, dw = (int)gridDim.x * kPgWarps;
  const int F = min(max(*p.free_count, 0), p.num_pages), cap = p.pt_stride * p.P;
  for (int b = tid; b < p.B; b += kPgThreads) back[b] = 0;
  auto held = [&](int b) {  // pages of an ended row
    return p.new_lens[b] < 0 ? pages_of(p, min(max(p.seq_lens[b], 0), cap)) : 0;
  };
  for (int b = w0; b < p.B; b += dw) {
    const int n = held(b);
    if (n > 0 && lane == 0 && p.seq_lens[b] > cap) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
    for (int c = lane; c < n; c += 32) {
      const int page = p.page_table[(size_t)b * p.pt_stride + c];
      if (page_ok(p, page)) atomicSub(p.page_refs + page, 1);
      else report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
    }
  }
  cluster_arrive();
  cluster_wait();
  for (int b = w0; b < p.B; b += dw) {
    const int n = held(b);
    for (int c = lane; c < n; c += 32) {
      const int page = p.page_table[(size_t)b * p.pt_stride + c];
      if (!page_ok(p, page) || __ldcg(p.page_refs + page) >= 0) continue;
      const int was = atomicMin(p.page_refs + page, mark_of(p, b, c));
      if (was > -kMark && was < -1) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);  // more rows than owners
    }
  }
  cluster_arrive();
  cluster_wait();
  for (int b = w0; b < p.B; b += dw) {
    const int n = held(b);
    int mine = 0;
    for (int c = lane; c < n; c += 32) {
      const int page = p.page_table[(size_t)b * p.pt_stride + c];
      mine += page_ok(p, page) && __ldcg(p.page_refs + page) == mark_of(p, b, c) ? 1 : 0;
    }
    mine = __reduce_add_sync(0xffffffffu, mine);
    if (n > 0) set_in_cluster(back + b, mine);
  }
  cluster_arrive();
  cluster_wait();
  const int per = (p.B + kPgThreads - 1) / kPgThreads, b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += back[b];
  int all;
  int at = scan_block(sum, scratch, all);
  for (int b = b0; b < b1; ++b) {
    const int n = back[b];
    back[b] = at;
    at += n;
  }
  __syncthreads();
  for (int b = w0; b < p.B; b += dw) {
    const int n = held(b);
    int to = F + back[b];
    for (int c0 = 0; c0 < n; c0 += 32) {
      const int c = c0 + lane;
      const int page = c < n ? p.page_table[(size_t)b * p.pt_stride + c] : -1;
      const bool mine = page_ok(p, page) && __ldcg(p.page_refs + page) == mark_of(p, b, c);
      const uint32_t who = __ballot_sync(0xffffffffu, mine);
      if (mine) {
        const int place = to + __popc(who & ((1u << lane) - 1u));
        if (place < p.num_pages) p.free_pages[place] = page;
        p.page_refs[page] = 0;
      }
      to += __popc(who);
    }
  }
  cluster_arrive();
  cluster_wait();  // kv_lens may be seq_lens, the height free_count: every block has read them
  if (blockIdx.x != 0) return;
  for (int b = tid; b < p.B; b += kPgThreads) p.kv_lens[b] = p.new_lens[b] < 0 ? 0 : p.seq_lens[b];
  if (tid == 0) {
    if (F + all > p.num_pages) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
    *p.count = min(F + all, p.num_pages);
  }
}

// ---------------------------------------------------------------------------
// Compaction.  Bitmaps of the live and the free pages in shared memory.  Of the M pages of
// either kind the n_live lowest are to be the live ones; `border` is the page with rank
// n_live.  Live pages from the border on move to the free ones before it, both in
// ascending order: the rank of a moving page is a count of bits.
__global__ void __launch_bounds__(kPgThreads, 1) compact_pages_kernel(const __grid_constant__ PagesParams p) {
  await_previous_kernel();
  extern __shared__ uint32_t bits[];
  const int words = (p.num_pages + 31) / 32;
  uint32_t* live = bits;
  uint32_t* spare = bits + words;
  uint32_t* before = spare + words;  // [words] holes and moving pages before a word
  __shared__ int scratch[kPgWarps + 1];
  __shared__ int s_border;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int F = min(max(*p.free_count, 0), p.num_pages), cap = p.pt_stride * p.P;
  for (int w = tid; w < 2 * words; w += kPgThreads) bits[w] = 0u;
  if (tid == 0) s_border = p.num_pages;
  __syncthreads();
  auto held = [&](int b) { return pages_of(p, min(max(p.seq_lens[b], 0), cap)); };
  for (int b = warp; b < p.B; b += kPgWarps) {
    const int n = held(b);
    if (lane == 0 && p.seq_lens[b] > cap) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
    for (int c = lane; c < n; c += 32) {
      const int page = p.page_table[(size_t)b * p.pt_stride + c];
      if (page_ok(p, page)) atomicOr(live + page / 32, 1u << page % 32);
      else report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
    }
  }
  for (int i = tid; i < F; i += kPgThreads) {
    const int page = p.free_pages[i];
    if (page == -1) continue;  // a place without a page, which an earlier compaction has told of
    if (!page_ok(p, page) || (atomicOr(spare + page / 32, 1u << page % 32) >> page % 32 & 1u))
      report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
  }
  __syncthreads();
  // a thread's words; pages of either kind before them
  const int per = (words + kPgThreads - 1) / kPgThreads, w0 = min(tid * per, words), w1 = min(w0 + per, words);
  int n_live = 0, known = 0;
  for (int w = w0; w < w1; ++w) {
    if (live[w] & spare[w]) {  // a page that is in use is on the stack: it stays in use
      report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
      spare[w] &= ~live[w];
    }
    n_live += __popc(live[w]);
    known += __popc(live[w] | spare[w]);
  }
  int all_live, all_known;
  scan_block(n_live, scratch, all_live);
  const int known0 = scan_block(known, scratch, all_known);
  if (known0 <= all_live && all_live < known0 + known) {  // the border is among this thread's words
    int r = known0;
    for (int w = w0; w < w1; ++w) {
      uint32_t m = live[w] | spare[w];
      const int n = __popc(m);
      if (r + n > all_live) {
        for (; r < all_live; ++r) m &= m - 1;
        s_border = 32 * w + __ffs(m) - 1;
        break;
      }
      r += n;
    }
  }
  __syncthreads();
  const int border = s_border;
  auto below = [&](int w) {  // bits of word w before the border
    return 32 * w + 32 <= border ? 0xffffffffu : 32 * w >= border ? 0u : (1u << (border - 32 * w)) - 1u;
  };
  int moving = 0;
  for (int w = w0; w < w1; ++w) moving += __popc((spare[w] & below(w)) | (live[w] & ~below(w)));
  int both;
  int at = scan_block(moving, scratch, both);
  const int moves = both / 2;  // as many holes as moving pages; the holes come first
  // places of the stack without a page (it held one twice, a live one or none): at the bottom, and no page's id,
  // so that build_tables and fork_pages tell whoever gets one and never hand out a live page
  for (int i = tid; i < F - (all_known - all_live); i += kPgThreads) p.free_pages[i] = -1;
  int r = known0;
  for (int w = w0; w < w1; ++w) {
    before[w] = (uint32_t)at;
    const uint32_t low = below(w);
    for (uint32_t m = spare[w] & low; m != 0u; m &= m - 1) p.dst[at++] = 32 * w + __ffs(m) - 1;
    for (uint32_t m = live[w] & ~low; m != 0u; m &= m - 1) p.src[at++ - moves] = 32 * w + __ffs(m) - 1;
    // the stack: the pages from the border on, the lowest on top
    const uint32_t k = live[w] | spare[w];
    for (uint32_t m = k; m != 0u; m &= m - 1, ++r)
      if (r >= all_live) p.free_pages[F - 1 - (r - all_live)] = 32 * w + __ffs(m) - 1;
  }
  for (int i = moves + tid; i < p.num_pages; i += kPgThreads) p.src[i] = p.dst[i] = -1;
  if (tid == 0) *p.count = moves;
  __syncthreads();
  // a moving page's new place: the hole with its rank
  auto moved = [&](int page) -> int {
    const int w = page / 32;
    if (page < border || !((live[w] >> page % 32) & 1u)) return page;
    const uint32_t low = below(w);
    const uint32_t m = (spare[w] & low) | (live[w] & ~low & ((1u << page % 32) - 1u));
    return p.dst[(int)before[w] + __popc(m) - moves];
  };
  for (int b = warp; b < p.B; b += kPgWarps) {
    const int n = held(b);
    int32_t* row = p.page_table + (size_t)b * p.pt_stride;
    for (int c = lane; c < n; c += 32) {
      const int page = row[c];
      if (!page_ok(p, page)) continue;
      const int to = moved(page);
      if (to != page) row[c] = to;
    }
  }
  if (p.page_refs)
    for (int i = tid; i < moves; i += kPgThreads) {
      const int from = p.src[i];
      p.page_refs[p.dst[i]] = p.page_refs[from];
      p.page_refs[from] = 0;
    }
}

// ---------------------------------------------------------------------------
// Copy.
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 4;                                  // 16-byte loads of a thread's step
constexpr int kCopyStep = kCopyThreads * kCopyVec;           // 16-byte words of a block's step
constexpr int kCopyChunk = 2 * kCopyStep * 16;               // bytes a block takes at once
constexpr int kCopyGrid = 64;                                // blocks per SM of the grid, 8 of which run at a time
constexpr int kCopyPools = 256;                              // of a launch (its parameters)

struct CopyParams {
  uint8_t* pools[kCopyPools];
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;
  int32_t* dev_err;
  int64_t page_bytes;
  int n_pools, n, num_pages, chunks;
  int chunk_bytes;  // of a page, equal parts of at most kCopyChunk
};

// A step's loads go out before the stores of the step before.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const __grid_constant__ CopyParams p) {
  await_previous_kernel();
  const int pairs = p.count ? min(max(*p.count, 0), p.n) : p.n;
  const int64_t per_pair = (int64_t)p.n_pools * p.chunks, units = pairs * per_pair;
  for (int64_t x = blockIdx.x; x < units; x += gridDim.x) {
    const int i = (int)(x / per_pair), rest = (int)(x - i * per_pair);
    const int from = p.src[i], to = p.dst[i];
    if (from < 0 || to < 0 || from == to) continue;
    if (from >= p.num_pages || to >= p.num_pages) {
      if (rest == 0 && threadIdx.x == 0) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
      continue;
    }
    const int pool = rest / p.chunks;
    const int64_t at = (int64_t)(rest - pool * p.chunks) * p.chunk_bytes;
    const int n = (int)min((int64_t)p.chunk_bytes, p.page_bytes - at) / 16;
    const uint4* a = reinterpret_cast<const uint4*>(p.pools[pool] + from * p.page_bytes + at) + threadIdx.x;
    uint4* b = reinterpret_cast<uint4*>(p.pools[pool] + to * p.page_bytes + at) + threadIdx.x;
    uint4 v[2][kCopyVec];
    auto load = [&](uint4 (&r)[kCopyVec], int k0) {
#pragma unroll
      for (int k = 0; k < kCopyVec; ++k)
        if ((int)threadIdx.x + k0 + k * kCopyThreads < n) r[k] = a[k0 + k * kCopyThreads];
    };
    auto store = [&](const uint4 (&r)[kCopyVec], int k0) {
#pragma unroll
      for (int k = 0; k < kCopyVec; ++k)
        if ((int)threadIdx.x + k0 + k * kCopyThreads < n) b[k0 + k * kCopyThreads] = r[k];
    };
    load(v[0], 0);
#pragma unroll
    for (int s = 0; s < kCopyChunk / 16 / kCopyStep; ++s) {
      if (s + 1 < kCopyChunk / 16 / kCopyStep) load(v[(s + 1) & 1], (s + 1) * kCopyStep);
      store(v[s & 1], s * kCopyStep);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side

static PagesParams pages_params(const PagesCall& c) {
  PagesParams p;
  p.source = c.source;
  p.seq_lens = c.seq_lens;
  p.new_lens = c.new_lens;
  p.page_table = c.page_table;
  p.page_refs = c.page_refs;
  p.free_pages = c.free_pages;
  p.free_count = c.free_count;
  p.kv_lens = c.kv_lens;
  p.src = c.src;
  p.dst = c.dst;
  p.count = c.count;
  p.dev_err = c.dev_err;
  p.inv_P = ~0ull / (uint64_t)c.P + 1;
  p.B = c.B;
  p.pt_stride = c.pt_stride;
  p.P = c.P;
  p.num_pages = c.num_pages;
  return p;
}

// Blocks of a cluster whose warps share the rows.
static unsigned row_blocks(int B) { return (unsigned)std::min(8, (B + kPgWarps - 1) / kPgWarps); }

int launch_fork_pages(const PagesCall& c) {
  static std::atomic<int> limit_set[kMaxDevices];
  if (!smem_limit_on_device(reinterpret_cast<const void*>(fork_pages_kernel), 16 * kTablesMaxBatch, limit_set))
    return INKLING_ERR_CUDA;
  const unsigned blocks = row_blocks(c.B);
  return launch_dependent(fork_pages_kernel, dim3(blocks), kPgThreads, 16 * c.B, pages_params(c), c.stream, blocks)
             ? INKLING_OK
             : INKLING_ERR_CUDA;
}

int launch_release_pages(const PagesCall& c) {
  static std::atomic<int> limit_set[kMaxDevices];
  if (!smem_limit_on_device(reinterpret_cast<const void*>(release_pages_kernel), 4 * kTablesMaxBatch, limit_set))
    return INKLING_ERR_CUDA;
  const unsigned blocks = row_blocks(c.B);
  return launch_dependent(release_pages_kernel, dim3(blocks), kPgThreads, 4 * c.B, pages_params(c), c.stream, blocks)
             ? INKLING_OK
             : INKLING_ERR_CUDA;
}

int launch_compact_pages(const PagesCall& c) {
  static std::atomic<int> limit_set[kMaxDevices];
  constexpr int kMost = kCompactMaxPages / 32 * 12;
  if (!smem_limit_on_device(reinterpret_cast<const void*>(compact_pages_kernel), kMost, limit_set))
    return INKLING_ERR_CUDA;
  const int smem = (c.num_pages + 31) / 32 * 12;
  return launch_dependent(compact_pages_kernel, dim3(1), kPgThreads, smem, pages_params(c), c.stream)
             ? INKLING_OK
             : INKLING_ERR_CUDA;
}

int launch_copy_pages(const CopyPagesCall& c) {
  CopyParams p;
  p.src = c.src;
  p.dst = c.dst;
  p.count = c.count;
  p.dev_err = c.dev_err;
  p.page_bytes = c.page_bytes;
  p.n = c.n;
  p.num_pages = c.num_pages;
  p.chunks = (int)((c.page_bytes + kCopyChunk - 1) / kCopyChunk);
  p.chunk_bytes = (int)(((c.page_bytes + p.chunks - 1) / p.chunks + 15) & ~15ll);
  for (int at = 0; at < c.n_pools; at += kCopyPools) {
    p.n_pools = std::min(c.n_pools - at, kCopyPools);
    for (int i = 0; i < kCopyPools; ++i) p.pools[i] = i < p.n_pools ? static_cast<uint8_t*>(c.pools[at + i]) : nullptr;
    const int64_t units = (int64_t)c.n * p.n_pools * p.chunks;
    const unsigned grid = (unsigned)std::min<int64_t>(units, (int64_t)c.sms * kCopyGrid);
    if (!launch_dependent(copy_pages_kernel, dim3(grid), kCopyThreads, 0, p, c.stream)) return INKLING_ERR_CUDA;
  }
  return INKLING_OK;
}

}  // namespace ira

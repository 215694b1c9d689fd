// Decode attention with the relative-position bias over a cache in blocks of 16
// tokens: what the 4-bit and the 8-bit cache share (decode_q4.cu, decode_q8.cu).
//
// Work.  An item is a (sequence, KV head, token group, head group); its rows are the
// group's (token, query head) pairs, at most 8, and its keys the visible range in
// tiles of two 16-token blocks.  (More rows in two MMA columns would read K and V
// once for them, but need twice the accumulators: over the 4-bit cache 64 query heads
// over 4 KV heads took 116 us so and 95 us as two items.)  The items of a head come one
// after the other, each over all its keys: a later one finds K and V in L2 where what the
// thread blocks read between its visits to a key stays within it, as with a window of 512 keys,
// and reads them from HBM again over long ranges (8-bit, 32 sequences to 32768 keys, 6 query
// heads per KV head: 181 us for one token, 343 for 2, 678 for 4, each an item of its own).
// All tiles of the batch, in (sequence, head, group, key) order, are cut into one
// equal run per thread block of a grid that fills the GPU, so every one streams the
// same bytes whatever the lengths are.  An item inside a run is finished there; the
// parts of one that is cut go to the workspace as (m, l, O), at most two per thread
// block, and a second kernel joins them.  The cuts depend on the lengths alone, not
// on page ids or timing.
//
// A thread block has two producer warps and four consumer warps.  One producer
// walks the run, looks pages up and brings each tile's K and V (a block's bytes are
// contiguous) into a ring of slots by bulk copy, a lane per tile; the ring runs
// across items, so the next one streams in while the current one is finished.  The
// other prepares the items (q as operands, bias pointers and positions per lane),
// three ahead; the 8-bit cache has a third for the sums of items of several tokens.
// Consumer warp w takes the ring's tiles w, w + 4, ... with an online
// softmax of its own; at the item's end it leaves (m, l, O) in one of two
// shared-memory buffers and goes on, and the preparing warp adds the parts up.  (One
// producer, and the last consumer to leave its part adding them up: over the 4-bit
// cache 64 sequences of 512 visible keys took 36.9 us instead of 31.9, for the copies
// stalled at every item and the slowest consumer was held up further.)
// Four warps load the SM's four schedulers alike (six, which give two of them two
// thirds of the work, took 195 us where four took 182), and a consumer's loop has
// no second copy for masked tiles (instruction fetches count in a short call).
//
// A format F says what a block is:
//   block_bytes(D)   bytes of a block of K or of V, a multiple of 16
//   key_of(g)        key of a block that row g < 8 of its first operand stands for; row g + 8: 8 more
//   zero_block       a block that reads as zeros, at two places of shared memory (K, V)
//   prepare          q of an item's rows as operands, and up to 4 words beside (RunPrep::extra)
//   kGroup           tiles whose copies go out together (those of a long ring)
//   kJoiner          whether a third producer warp fits the registers
//   Consumer         the products S^T = K Q^T (16 keys x rows) and O^T += V^T P^T of a warp;
//                    mark: what rows get from keys with a NaN that they see
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <cstring>

#include "async.cuh"
#include "internal.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "tc.cuh"

namespace ira {

constexpr int kRunItemSlots = 3;      // items published ahead
constexpr int kRunMinRun = 2;         // tiles of a run at least (4-bit, 2 sequences of 2 heads: 7.4 us, with 8 13.9)
constexpr int kRunSmemPerSm = 222 * 1024;
constexpr float kRunSlack = 5.5f;     // scores may exceed the exponent base by e^5.5 before it moves
constexpr int kRunW = 4;              // consumer warps
constexpr int kRunCtas = 2;           // thread blocks per SM
// Items of several tokens have up to 8 rows to add up, a warp's work of its own where the registers
// allow it (8-bit, 64 sequences of 4 drafts: 57.3 us, by the preparing warp 62.5, both before Q8Format::mark; items
// of one token, with 3 rows, 36.6 and 35.7).
template <class F, bool MULTI>
constexpr bool run_joiner() {
  return F::kJoiner && MULTI;
}
template <class F, bool MULTI>
constexpr int run_threads() {
  return 32 * (kRunW + (run_joiner<F, MULTI>() ? 3 : 2));
}
constexpr int kRunMergeWarps = 4;     // of the joining kernel's blocks: a thread per channel in all
constexpr int kRunU = 2;              // 16-token blocks per tile
constexpr int kRunTile = 16 * kRunU;  // keys per tile
static_assert(kRunU == 2, "a tile's first and last block");
constexpr int kRunRows = 8;           // rows of an item at most: the N of an MMA

struct DecodeBlocksParams {
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* rel;
  __nv_bfloat16* out;
  float* lse_out;
  float* part_o;    // [grid][2][NR][D]
  float2* part_ml;  // [grid][2][NR]
  int4* cut;        // [grid]: a cut item's first packed row, tokens, parts, heads; parts 0: none
  int32_t* dev_err;
  int B, pt_stride, H_q, H_kv, G, P, num_pages, R, window;
  int QL, TG;  // query tokens per sequence, per item
  int HI, HG;  // query heads of a KV head per item, items for all of them
  int NT, NR;  // token groups of a sequence; rows of an item at most
  int inv_G;   // 256 / G, rounded up (items of several tokens have all G <= 4 heads): rows divide by a product
  uint32_t inv_P;      // 2^32 / P, rounded up
  int slots;           // ring slots
  int bias_prefetch;   // rel_logits rows are 16-byte aligned
  float scale;         // what the format multiplies its products by
};

// Part of an item: tiles tile0 .. tile0 + ntile - 1 of the item's sequence.
struct RunItem {
  int row0;  // packed row (token * H_q + head) of its first token and head
  int tn, heads, pos0;
  int tile0, ntile;
  int part;  // -1: the whole item; else its part number of this thread block
};

// What the producer prepares of an item, per lane of a consumer.
struct RunPrep {
  const float* bias[2];  // of score columns 2t, 2t + 1: the element at the position of MMA row g's key 0
  float far[2];          // bias at and past the table's end
  int pos[2];
  uint32_t extra[4];     // what the format needs beside
};  // 48 bytes; the q fragments (16 bytes for 32 channels) follow

// Shared memory (byte offsets from a 128-byte aligned base).
struct RunSmem {
  int slot_bytes, item_bytes, prep_off, frag_off, item_off, comb_off, comb_floats, bar_off, total;
  __host__ __device__ RunSmem(int block_bytes, int D, int NR, int slots) {
    slot_bytes = 2 * kRunU * block_bytes;     // K of the blocks, V of the blocks
    prep_off = 64;                                   // [3][32] of 16 bytes
    frag_off = prep_off + 32 * 48;                   // [D / 32][32] of 16 bytes
    item_bytes = frag_off + (D / 32) * 32 * 16;
    item_off = (slots * slot_bytes + 127) & ~127;
    comb_off = item_off + kRunItemSlots * item_bytes;
    comb_floats = kRunW * NR * (D + 4) + 2 * kRunW * kRunRows;
    bar_off = comb_off + 2 * comb_floats * 4;
    total = bar_off + (2 * slots + 2 * kRunItemSlots + 4) * 8 + 16;
  }
};

// A plain load, not one of the read-only path (launch.h), that the compiler may still move
// among the arithmetic around it (as an ordinary load, which stays in its place, drafts
// took 57.6 us instead of 54.5).  Its address comes from shared memory written after the
// wait for the kernel before, so it cannot move ahead of that.
__device__ __forceinline__ float load_bias(const float* at) {
  float v;
  asm("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(at));
  return v;
}

// Positions and tiles of the items of token group tg of a sequence of length L >= QL.
struct GroupRange {
  int tn, pos0, tile0, ntile;
};
__device__ __forceinline__ GroupRange group_range(const DecodeBlocksParams& p, int L, int tg) {
  GroupRange r;
  const int first = tg * p.TG;
  r.tn = min(p.TG, p.QL - first);
  r.pos0 = L - p.QL + first;
  const int lo = p.window > 0 ? max(0, r.pos0 - p.window + 1) : 0;
  r.tile0 = lo / kRunTile;
  r.ntile = (r.pos0 + r.tn - 1) / kRunTile - r.tile0 + 1;
  return r;
}
__device__ __forceinline__ int clamped_len(const DecodeBlocksParams& p, int b) {
  return min(max(p.seq_lens[b], 0), p.pt_stride * p.P);
}
// Tiles of one KV head of a sequence of length L (all its items); 0 when it has fewer keys than new tokens.
__device__ __forceinline__ int head_tiles(const DecodeBlocksParams& p, int L) {
  if (L < p.QL) return 0;
  int n = 0;
  for (int tg = 0; tg < p.NT; ++tg) n += group_range(p, L, tg).ntile;
  return n * p.HG;
}

// Numbers of tiles nearly always fit 32 bits, whose division is several times shorter.
__device__ __forceinline__ int64_t div_tiles(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Page and place of a key.  The product with 2^32 / P rounded up is at most one too large.
__device__ __forceinline__ int2 page_place(const DecodeBlocksParams& p, int key) {
  int q = (int)__umulhi((uint32_t)key, p.inv_P), r = key - q * p.P;
  if (r < 0) {
    --q;
    r += p.P;
  }
  return make_int2(q, r);
}

// MULTI: items of several tokens, so rows of several positions.
// (The whole is the kernel itself: as a function that two kernels inline it took 59.4 us
// instead of 55.2 for 64 sequences of 4 drafts over the 4-bit cache, the compiler having
// treated the parameters as memory before it inlined.)
template <class F, int D, bool MULTI>
__global__ void __launch_bounds__(run_threads<F, MULTI>(), kRunCtas)
    decode_blocks_kernel(const __grid_constant__ DecodeBlocksParams p) {
  constexpr int W = kRunW, U = kRunU, TK = kRunTile;
  constexpr int HP = kRunRows;
  constexpr int OP = D + 4;
  constexpr bool JOINER = run_joiner<F, MULTI>();
  constexpr int BLK = F::block_bytes(D);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int NR = p.NR, slots = p.slots;
  const RunSmem S(BLK, D, NR, slots);
  // the warps' parts of an item, two buffers in turn: O [W][NR][D + 4], m [W][HP], l [W][HP]
  auto comb_o = [&](int s) { return reinterpret_cast<float*>(smem + S.comb_off) + s * S.comb_floats; };
  auto comb_m = [&](int s) { return comb_o(s) + W * NR * OP; };
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S.bar_off);  // ring slots
  uint64_t* empty = full + slots;
  uint64_t* ifull = empty + slots;           // items: published,
  uint64_t* iempty = ifull + kRunItemSlots;  // taken by every consumer
  uint64_t* cfull = iempty + kRunItemSlots;  // parts of an item: left by every consumer,
  uint64_t* cempty = cfull + 2;              // added up
  volatile int* abort_flag = reinterpret_cast<int*>(cempty + 2);
  auto item_at = [&](int s) { return smem + S.item_off + s * S.item_bytes; };
  auto item_rec = [&](int s) { return reinterpret_cast<RunItem*>(item_at(s)); };
  // token of an item's row r, and its packed row
  auto token_of = [&](int r) { return MULTI ? (r * p.inv_G) >> 8 : 0; };
  auto row_of = [&](const RunItem& it, int r) {
    const int i = token_of(r);
    return (size_t)it.row0 + (size_t)i * p.H_q + (r - i * it.heads);
  };
  const int key_g = F::key_of(g);  // key of a block that MMA row g stands for (and g + 8: 8 more)

  for (int i = tid; i < slots; i += run_threads<F, MULTI>()) {
    mbar_init(smem_u32(full + i), 1);
    mbar_init(smem_u32(empty + i), 1);
  }
  if (tid == 0) {
    for (int i = 0; i < kRunItemSlots; ++i) {
      mbar_init(smem_u32(ifull + i), 1);
      mbar_init(smem_u32(iempty + i), W + (JOINER ? 1 : 0));
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(cfull + i), W);
      mbar_init(smem_u32(cempty + i), 1);
    }
    *abort_flag = 0;
  }
  fence_mbar_init();
  __syncthreads();
  await_previous_kernel();

  // =================================================================== producers
  // ---- the sum of the warps' parts of an item
  // lane W * r + w makes the factor of warp w's part of row r, and leaves it where the part's
  // maximum was.  No shuffles: beside waiting and computing warps one takes some 280 cycles
  // here, and the four a row were what held the items up (64 sequences of 4 drafts over the
  // 8-bit cache).  (Short code: this warp shares the instruction cache with
  // the consumers' loop; unrolled by 4, 11 us more for 64 sequences of 4 drafts.)
  auto join = [&](const RunItem& it, int cb) {
    static_assert(W * HP == 32, "a lane per row and warp");
    constexpr int LR = D / 4;  // lanes per row
    const float* co = comb_o(cb);
    float* cm = comb_m(cb);
    const int rows = it.tn * it.heads, d = 4 * (lane % LR), row = lane / W;
    float m[W], M = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      m[w] = cm[w * HP + row];
      M = fmaxf(M, m[w]);
    }
    const float base = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < W; ++w) l = fmaf(ex2((m[w] - base) * kLog2e), cm[(W + w) * HP + row], l);
    __syncwarp();
    float f = ex2((cm[lane % W * HP + row] - base) * kLog2e);
    const bool mine = lane % W == 0 && row < rows;
    if (it.part < 0) {
      f = l == 0.f ? -1.f : f * __fdividef(1.f, l);  // every score -inf: an empty row, whatever its values
      if (mine && p.lse_out) p.lse_out[row_of(it, row)] = M + logf(l);
    } else if (mine) {
      p.part_ml[((size_t)blockIdx.x * 2 + it.part) * NR + row] = make_float2(M, l);
    }
    cm[lane % W * HP + row] = f;
    __syncwarp();
#pragma unroll 1
    for (int r0 = 0; r0 < rows; r0 += 32 / LR) {
      const int r = r0 + lane / LR;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      bool empty = false;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float fw = cm[w * HP + min(r, rows - 1)];
        if (w == 0) empty = fw < 0.f;
        const float4 v = *reinterpret_cast<const float4*>(co + (w * NR + min(r, rows - 1)) * OP + d);
        a.x = fmaf(fw, v.x, a.x);
        a.y = fmaf(fw, v.y, a.y);
        a.z = fmaf(fw, v.z, a.z);
        a.w = fmaf(fw, v.w, a.w);
      }
      if (r >= rows) continue;
      if (empty) a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (it.part < 0)
        *reinterpret_cast<uint2*>(p.out + row_of(it, r) * D + d) =
            make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
      else
        *reinterpret_cast<float4*>(p.part_o + (((size_t)blockIdx.x * 2 + it.part) * NR + r) * D + d) = a;
    }
  };
  if (JOINER && warp == W + 2) {  // adds the parts of every item up
    bool ok = true;
    for (int k = 0;; ++k) {
      const int is = k % kRunItemSlots, cb = k & 1;
      ok = waitw(smem_u32(ifull + is), (k / kRunItemSlots) & 1, abort_flag);
      if (!ok) break;
      const RunItem it = *item_rec(is);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(iempty + is));
      if (it.ntile == 0) break;
      ok = waitw(smem_u32(cfull + cb), (k >> 1) & 1, abort_flag);
      if (!ok) break;
      join(it, cb);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(cempty + cb));
    }
    if (!ok && lane == 0) report(p.dev_err, INKLING_DEVERR_TIMEOUT);
    return;
  }
  // Both walk the run: warp W sends the tiles, warp W + 1 prepares the items.
  if (warp >= W) {
    const bool copier = warp == W;
    // ---- this thread block's run [x, x1) of the batch's tiles.  A lane has four sequences
    // of 128, whose lengths are asked for together; up to 128 are read once.
    int tiles[4];  // of one KV head
    auto read = [&](int b0, bool tell) {
      int len[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int b = b0 + 4 * lane + k;
        len[k] = b < p.B ? p.seq_lens[b] : -1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int cap = p.pt_stride * p.P;
        tiles[k] = head_tiles(p, min(len[k], cap));
        if (tell && b0 + 4 * lane + k < p.B) {
          if (len[k] > cap) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
          if (p.QL > 1 && len[k] < p.QL) report(p.dev_err, INKLING_DEVERR_BAD_CHUNK);
        }
      }
      return (int64_t)p.H_kv * ((int64_t)tiles[0] + tiles[1] + tiles[2] + tiles[3]);
    };
    int64_t total = 0, mine = 0;
    for (int b0 = 0; b0 < p.B; b0 += 128) {
      mine = read(b0, copier && blockIdx.x == 0);
      total += mine;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    const int64_t runs = min((int64_t)gridDim.x, max((total + kRunMinRun - 1) / kRunMinRun, (int64_t)1));
    int64_t x = total, x1 = total;
    if (blockIdx.x < runs) {  // total * i / runs, rounded down
      const int64_t each = div_tiles(total, runs);
      const uint32_t left = (uint32_t)(total - each * runs), r = (uint32_t)runs, i = blockIdx.x;
      x = each * i + left * i / r;
      x1 = each * (i + 1) + left * (i + 1) / r;
    }
    // ---- the item at x
    int b = 0, hkv = 0, tg = 0, hg = 0, off = 0, L = 0;
    if (x < x1) {
      int64_t carry = 0;
      for (int b0 = 0;; b0 += 128) {
        if (p.B > 128) mine = read(b0, false);
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, carry + incl > x);
        if (past) {
          const int src = __ffs(past) - 1;
          int64_t at = x - (carry + __shfl_sync(0xffffffffu, incl - mine, src));
          int nb = 0;  // tiles per head of sequence b
          b = b0 + 4 * src;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            nb = __shfl_sync(0xffffffffu, tiles[k], src);
            if (at < (int64_t)p.H_kv * nb) break;
            at -= (int64_t)p.H_kv * nb;
            ++b;
          }
          hkv = (int)div_tiles(at, nb);
          off = (int)(at - (int64_t)hkv * nb);
          break;
        }
        carry += __shfl_sync(0xffffffffu, incl, 31);
      }
      L = clamped_len(p, b);
      for (;;) {  // items of a head: token groups, head groups within them
        const int n = group_range(p, L, tg).ntile;
        if (off < n) break;
        off -= n;
        if (++hg == p.HG) {
          hg = 0;
          ++tg;
        }
      }
    }

    int ki = 0, kb = 0;  // items published, tiles sent
    const int blocks_per_page = p.P / 16;
    const int batch = min(32, slots);
    uint32_t sent = 0;  // on a time-out: the copies of the batch at kb that went out
    int4 cut = make_int4(0, 0, 0, 0);
    bool ok = true;
    auto prepare = [&](const RunItem& it, int is) {
      const int rows = it.tn * it.heads;
      RunPrep pr;
      // q as operands: row min(g, rows - 1), zeros past the last row
      F::template prepare<D>(p, reinterpret_cast<const uint4*>(p.q + row_of(it, min(g, rows - 1)) * D), g < rows,
                             reinterpret_cast<uint4*>(item_at(is) + S.frag_off) + lane, pr);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = min(2 * t + x, rows - 1);
        pr.pos[x] = it.pos0 + token_of(r);
        const float* row = p.rel + row_of(it, r) * p.R;
        pr.bias[x] = row + (pr.pos[x] - key_g);
        pr.far[x] = it.pos0 + it.tn - 1 - TK * it.tile0 >= p.R ? row[p.R - 1] : 0.f;
      }
      uint4* dst = reinterpret_cast<uint4*>(item_at(is) + S.prep_off) + lane;
      const uint4* src = reinterpret_cast<const uint4*>(&pr);
#pragma unroll
      for (int i = 0; i < 3; ++i) dst[32 * i] = src[i];
    };
    auto join_item = [&](int k) -> bool {
      const int cb = k & 1;
      if (!waitw(smem_u32(cfull + cb), (k >> 1) & 1, abort_flag)) return false;
      const RunItem it = *item_rec(k % kRunItemSlots);
      join(it, cb);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(cempty + cb));
      return true;
    };
    auto publish = [&](const RunItem& it) -> bool {
      const int s = ki % kRunItemSlots;
      bool good = true;
      if (ki >= kRunItemSlots && lane == 0)
        good = wait1(smem_u32(iempty + s), ((ki / kRunItemSlots) - 1) & 1, abort_flag);
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) return false;
      if (it.ntile > 0) prepare(it, s);
      if (lane == 0) *item_rec(s) = it;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(ifull + s));
      ++ki;
      return true;
    };
    while (x < x1 && ok) {
      const GroupRange r = group_range(p, L, tg);
      RunItem it;
      const int h0 = hg * p.HI;  // its first head of the KV head's
      it.row0 = (b * p.QL + tg * p.TG) * p.H_q + hkv * p.G + h0;
      it.tn = r.tn;
      it.heads = min(p.HI, p.G - h0);
      it.pos0 = r.pos0;
      it.tile0 = r.tile0 + off;
      it.ntile = (int)min((int64_t)(r.ntile - off), x1 - x);
      it.part = -1;
      if (it.ntile < r.ntile) {
        it.part = off > 0 ? 0 : 1;
        if (off == 0) {  // the thread block with an item's first part has the record of its cut
          const int64_t e = x + r.ntile - 1;
          const int last = (int)div_tiles((e + 1) * runs - 1, total);
          cut = make_int4(it.row0, it.tn, last - (int)blockIdx.x + 1, it.heads);
        }
      }
      if (!copier && p.bias_prefetch && lane < it.tn * it.heads) {  // this row's bias for the part's keys
        const int pr = it.pos0 + token_of(lane);
        const int far = pr - TK * it.tile0, near = pr - (TK * (it.tile0 + it.ntile) - 1);
        const int dlo = min(max(near, 0), p.R - 1) & ~3;
        const int dhi = min(min(max(far, 0), p.R - 1) + 4, p.R) & ~3;
        const float* row = p.rel + row_of(it, lane) * p.R;
        if (dhi > dlo) bulk_prefetch_l2(row + dlo, (uint32_t)(dhi - dlo) * 4);
      }
      // (the record of item ki - 2 is in the slot of the item after this one)
      if (!copier) ok = publish(it) && (JOINER || ki < 3 || join_item(ki - 3));
      if (!ok) break;
      // ---- its tiles: a lane each, a batch of at most 32 (and of the ring's slots: no
      // two lanes share one) at a time.  A lane's copies go out as soon as its slot is
      // free; page ids are read a batch ahead.
      const int32_t* pt_row = p.page_table + (size_t)b * p.pt_stride;
      // Blocks of a tile that no row sees are not looked up: their pages may be gone.  A
      // tile has a key that is seen, so its first block can lie before the window only, and
      // its last past the last key only.  (Where pages hold whole tiles the first block's is
      // the last one's, and both come in one copy.)
      const int pos1 = it.pos0 + it.tn - 1;
      const int before = (p.window > 0 && p.P % TK != 0 ? max(0, it.pos0 - p.window + 1) : 0) - 15;
      auto seen = [&](int key, int u) { return u == 0 ? key >= before : key <= pos1; };
      auto page_of = [&](int i, int u) -> int {  // page of block u of tile i; -1: not seen
        const int key = (it.tile0 + i) * TK + 16 * u;
        return copier && lane < batch && i < it.ntile && seen(key, u) ? pt_row[page_place(p, key).x] : -1;
      };
      int page[U], next[U];
#pragma unroll
      for (int u = 0; u < U; ++u) next[u] = page_of(lane, u);
#pragma unroll 1
      for (int i0 = 0; copier && i0 < it.ntile; i0 += batch) {
        const int i = i0 + lane, key0 = (it.tile0 + i) * TK;
        int place[U];
        bool fine[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          page[u] = next[u];
          next[u] = page_of(i + batch, u);
          fine[u] = page[u] >= 0 && page[u] < p.num_pages;
          place[u] = page_place(p, key0 + 16 * u).y;
        }
        bool todo = lane < batch && i < it.ntile;
        const uint32_t all = __ballot_sync(0xffffffffu, todo);
        const uint32_t n = (uint32_t)(kb + lane), turn = n / (uint32_t)slots;
        const uint32_t sl = n - turn * (uint32_t)slots;
        uint8_t* dst = smem + sl * S.slot_bytes;
        const uint32_t fb = smem_u32(full + sl), eb = smem_u32(empty + sl);
        // Waits (suspended) for the slot of a pending lane a few tiles on, then every
        // lane whose slot is free sends.
        for (uint32_t left = all; left != 0; left = __ballot_sync(0xffffffffu, todo)) {
          // (of a pending lane: a slot already sent to may be a phase further by now)
#pragma unroll
          for (int u = 0; u < F::kGroup - 1; ++u) left = (left & (left - 1)) ? left & (left - 1) : left;
          const int at_lane = __ffs(left) - 1;
          // (a slot's first turn waits for the phase before the first, which counts as complete)
          ok = waitw(__shfl_sync(0xffffffffu, eb, at_lane), (__shfl_sync(0xffffffffu, turn, at_lane) - 1) & 1,
                     abort_flag);
          if (!ok) break;
          if (todo && mbar_try_wait(eb, (turn - 1) & 1)) {
            todo = false;
            int live = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
              live += fine[u] ? 1 : 0;
              // a bad page reads as zeros; of a block that no row sees nothing is needed
              if (!fine[u] && seen(key0 + 16 * u, u)) {
                F::template zero_block<D>(dst + u * BLK, dst + (U + u) * BLK);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
              }
            }
            if (live > 0) mbar_arrive_expect_tx(fb, 2 * BLK * live);
            else mbar_arrive(fb);
            // blocks of a page are contiguous: one copy where the tile lies in one
            const bool whole = U > 1 && live == U && place[U - 1] == place[0] + 16 * (U - 1);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (!fine[u] || (whole && u > 0)) continue;
              const size_t at = (((size_t)page[u] * p.H_kv + hkv) * blocks_per_page + place[u] / 16) * BLK;
              const uint32_t bytes = whole ? U * BLK : BLK;
              bulk_load(smem_u32(dst) + u * BLK, p.k_cache + at, bytes, fb);
              bulk_load(smem_u32(dst) + (U + u) * BLK, p.v_cache + at, bytes, fb);
            }
          }
        }
        if (!ok) {
          sent = all & ~__ballot_sync(0xffffffffu, todo);
          break;
        }
        kb += min(batch, it.ntile - i0);
      }
      if (!ok) break;
      // ---- the next item
      x += it.ntile;
      off = 0;
      if (++hg == p.HG) {
        hg = 0;
        ++tg;
      }
      if (tg == p.NT) {
        tg = 0;
        if (++hkv == p.H_kv) {
          hkv = 0;
          do {
            ++b;
          } while (b < p.B && clamped_len(p, b) < p.QL);
          if (b < p.B) L = clamped_len(p, b);
        }
      }
    }
    if (!copier) {
      if (ok) {
        RunItem end;
        memset(&end, 0, sizeof(end));
        const int n = ki;
        ok = publish(end) && (JOINER || ((n < 2 || join_item(n - 2)) && (n < 1 || join_item(n - 1))));  // ntile = 0: no more items
      }
      if (lane == 0) p.cut[blockIdx.x] = cut;
      if (!ok && lane == 0) report(p.dev_err, INKLING_DEVERR_TIMEOUT);
      return;
    }
    ok = __all_sync(0xffffffffu, ok && *abort_flag == 0);
    if (!ok) {  // drain: each slot's last copy in flight, which nobody reads
      for (int j = lane; j < slots; j += 32) {
        int n = kb - kb % slots + j;  // the slot's tile in [kb, kb + slots), or before
        if (n < kb) n += slots;
        if (n - kb >= 32 || !((sent >> (n - kb)) & 1u)) n -= slots;
        if (n >= 0) mbar_wait_drain(smem_u32(full + j), (n / slots) & 1);
      }
    }
    if (!ok && lane == 0) report(p.dev_err, INKLING_DEVERR_TIMEOUT);
    // ---- sequences with nothing to attend to
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      if (clamped_len(p, b) >= p.QL) continue;
      const int rows = p.QL * p.H_q;
      const size_t r0 = (size_t)b * rows;
      for (int i = lane; i < rows * (D / 8); i += 32)
        reinterpret_cast<uint4*>(p.out + r0 * D)[i] = make_uint4(0, 0, 0, 0);
      if (p.lse_out)
        for (int i = lane; i < rows; i += 32) p.lse_out[r0 + i] = -INFINITY;
    }
    return;
  }

  // =================================================================== consumers
  typename F::template Consumer<D, MULTI> c(g, t, lane);

  int kb_w = 0;       // tiles of the items before this one, modulo W
  int s_slot = warp;  // this warp's next slot (it owns warp, warp + W, ...) and its phase
  uint32_t s_phase = 0;
  bool ok = true;
  for (int ki = 0;; ++ki) {
    const int is = ki % kRunItemSlots;
    if (!waitw(smem_u32(ifull + is), (ki / kRunItemSlots) & 1, abort_flag)) {
      ok = false;
      break;
    }
    const RunItem it = *item_rec(is);
    if (it.ntile == 0) break;
    RunPrep pr;
    const uint4* src = reinterpret_cast<const uint4*>(item_at(is) + S.prep_off) + lane;
    c.load_q(reinterpret_cast<const uint4*>(item_at(is) + S.frag_off) + lane);
#pragma unroll
    for (int i = 0; i < 3; ++i) reinterpret_cast<uint4*>(&pr)[i] = src[32 * i];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(iempty + is));
    const int pos0 = it.pos0, pos1 = it.pos0 + it.tn - 1;

    float m_run[2], l_run[2];
    m_run[0] = m_run[1] = -INFINITY;
    l_run[0] = l_run[1] = 0.f;
    c.begin(pr);

    // ---- this warp's tiles of the item
    int i = warp - kb_w;
    if (i < 0) i += W;
    kb_w = (kb_w + it.ntile) % W;
    for (int turn = 1;; i += W, ++turn) {
      const bool last = i >= it.ntile;
      if (last || (turn & 7) == 0) {
        c.settle();
        if (last) break;
      }
      const int key0 = (it.tile0 + i) * TK;
      // ---- bias, on its way while the tile is awaited and K multiplied
      const bool inside = key0 + TK - 1 <= pos0 && (p.window <= 0 || pos1 - key0 < p.window);
      float bv[U][4];
      uint32_t hidden = 0;  // bit 4 u + x: the row of score x does not see its key, whatever the bias
      const bool far = inside && pos0 - (key0 + TK - 1) >= p.R - 1;
      if (!far && inside && pos1 - key0 < p.R) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) bv[u][x] = load_bias(pr.bias[x & 1] - key0 - 16 * u - 8 * (x >> 1));
      } else if (!far) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = key0 + 16 * u + 8 * (x >> 1), dist = pr.pos[x & 1] - key_g - key;
            const float v = load_bias(pr.bias[x & 1] - key + (min(max(dist, 0), p.R - 1) - dist));
            const bool seen = dist >= 0 && (p.window <= 0 || dist < p.window);
            bv[u][x] = seen ? v : -INFINITY;
            hidden |= seen ? 0u : 1u << (4 * u + x);
          }
      }
      if (!waitw(smem_u32(full + s_slot), s_phase, abort_flag)) {
        ok = false;
        break;
      }
      uint8_t* ring_slot = smem + s_slot * S.slot_bytes;
      const uint32_t eb = smem_u32(empty + s_slot);
      s_slot += W;
      if (s_slot >= slots) {
        s_slot = warp;
        s_phase ^= 1;
      }
      if (!inside) {  // keys that no row sees: their places may hold anything
        c.hide(ring_slot, key0, p.window > 0 ? pos0 - p.window + 1 : 0, pos1);
        fence_proxy_async_smem();  // before the slot's next copy
        __syncwarp();
      }
      // ---- scores of 16 keys x rows
      float sc[U][4];
      c.scores(p, ring_slot, sc);
      if (far) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[u][x] = c.score(p, u, x, sc[u][x], pr.far[x & 1], false);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[u][x] = c.score(p, u, x, sc[u][x], bv[u][x], hidden >> (4 * u + x) & 1u);
      }
      // ---- running maximum and sum.  The maximum, the exponents' base, is
      // taken anew over the warp only when a score passes it by kRunSlack;
      // until then a weight is at most e^kRunSlack and nothing is rescaled.
      float mx[2] = {fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[0][1], sc[0][3])};
#pragma unroll
      for (int u = 1; u < U; ++u) {
        mx[0] = fmaxf(mx[0], fmaxf(sc[u][0], sc[u][2]));
        mx[1] = fmaxf(mx[1], fmaxf(sc[u][1], sc[u][3]));
      }
      const bool v_up = c.v_scales(ring_slot);  // (the format's base for V moves; the same in all lanes)
      if (__any_sync(0xffffffffu, mx[0] > m_run[0] + kRunSlack || mx[1] > m_run[1] + kRunSlack) || v_up) {
        const float vf = c.v_rebase();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], off));
          const float mn = fmaxf(m_run[x], mx[x]);
          const float al = mn == -INFINITY ? 1.f : ex2((m_run[x] - mn) * kLog2e);
          l_run[x] *= al;
          m_run[x] = mn;
          c.rescale(x, al * vf);
        }
      }
      // the difference first: s * log2 e alone would lose it under a bias like -1e30
      const uint64_t l2e = f2_pack(kLog2e, kLog2e);
      const uint64_t mbase = f2_pack(m_run[0] == -INFINITY ? 0.f : -m_run[0],
                                     m_run[1] == -INFINITY ? 0.f : -m_run[1]);
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int x = 0; x < 4; x += 2) {
          float a0, a1;
          f2_unpack(f2_mul(f2_add(f2_pack(sc[u][x], sc[u][x + 1]), mbase), l2e), a0, a1);
          sc[u][x] = ex2(a0);
          sc[u][x + 1] = ex2(a1);
        }
        l_run[0] += sc[u][0] + sc[u][2];
        l_run[1] += sc[u][1] + sc[u][3];
      }
      // (whether the row of weight x sees its key: by position and window, whatever the bias)
      c.mark(ring_slot, sc, l_run, [&](int u, int x) {
        const int dist = pr.pos[x & 1] - key_g - (key0 + 16 * u + 8 * (x >> 1));
        return dist >= 0 && (p.window <= 0 || dist < p.window);
      });
      // ---- O^T += V^T P^T; hands the slot back
      c.values(ring_slot, eb, sc, hidden);
    }
    if (!ok) break;

    // ---- this warp's part of the item
    const int cb = ki & 1;
    if (ki >= 2 && !waitw(smem_u32(cempty + cb), ((ki >> 1) - 1) & 1, abort_flag)) {
      ok = false;
      break;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float l = l_run[x];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      const int r = 2 * t + x;
      if (g == 0) {
        comb_m(cb)[warp * HP + r] = m_run[x];
        comb_m(cb)[(W + warp) * HP + r] = l;
      }
      if (r < it.tn * it.heads) c.store(x, comb_o(cb) + (warp * NR + r) * OP);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(cfull + cb));
  }
  if (!ok && lane == 0) report(p.dev_err, INKLING_DEVERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Joins the parts of cut items: block (c, r) has row r of the item that thread
// block c's run cuts first.  Its parts are c's second and the first of c + 1 .. ;
// the block's warps take them in turn, D / 32 channels per lane.
template <int D>
__global__ void __launch_bounds__(32 * kRunMergeWarps)
    merge_blocks_kernel(const __grid_constant__ DecodeBlocksParams p) {
  await_previous_kernel();
  constexpr int C = D / 32;
  const int4 cut = p.cut[blockIdx.x];
  const int r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float s_o[kRunMergeWarps][D];
  __shared__ float2 s_ml[kRunMergeWarps];
  auto part_row = [&](int k) {
    return ((size_t)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * p.NR + r;
  };
  // a warp's first part is asked for along with the record that says whether there is
  // one (its place in the workspace exists in any case)
  float M = -INFINITY, l = 0.f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
  if (blockIdx.x + warp < gridDim.x) {
    const size_t row = part_row(warp);
    const float2 ml = p.part_ml[row];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = p.part_o[row * D + lane + 32 * c];
    M = ml.x;
    l = ml.y;
  }
  if (cut.z == 0 || r >= cut.y * cut.w) return;
  if (warp >= cut.z) {
    M = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = 0.f;
  }
#pragma unroll 4
  for (int k = warp + kRunMergeWarps; k < cut.z; k += kRunMergeWarps) {
    const size_t row = part_row(k);
    const float2 ml = p.part_ml[row];
    float v[C];
#pragma unroll
    for (int c = 0; c < C; ++c) v[c] = p.part_o[row * D + lane + 32 * c];
    const float mn = fmaxf(M, ml.x), base = mn == -INFINITY ? 0.f : mn;
    const float fa = ex2((M - base) * kLog2e), fb = ex2((ml.x - base) * kLog2e);
    l = fmaf(l, fa, ml.y * fb);
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = fmaf(acc[c], fa, v[c] * fb);
    M = mn;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) s_o[warp][lane + 32 * c] = acc[c];
  if (lane == 0) s_ml[warp] = make_float2(M, l);
  __syncthreads();
  if (threadIdx.x >= D) return;
  const int d = threadIdx.x;
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kRunMergeWarps; ++w) M = fmaxf(M, s_ml[w].x);
  const float base = M == -INFINITY ? 0.f : M;
  float o = 0.f;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kRunMergeWarps; ++w) {
    const float f = ex2((s_ml[w].x - base) * kLog2e);
    l = fmaf(s_ml[w].y, f, l);
    o = fmaf(s_o[w][d], f, o);
  }
  const int i = r / cut.w;
  const size_t row = (size_t)cut.x + (size_t)i * p.H_q + (r - i * cut.w);
  p.out[row * D + d] = __float2bfloat16(l == 0.f ? 0.f : o / l);
  if (d == 0 && p.lse_out) p.lse_out[row] = M + logf(l);
}

// ---------------------------------------------------------------------------
// Host side


struct RunPlan {
  int G, TG, HI, HG, NT, NR, grid;
  size_t ml, cut, total;  // workspace offsets: parts first
  RunPlan(int32_t QL, int32_t H_q, int32_t H_kv, int32_t D, int32_t sms) {
    G = H_q / H_kv;
    HG = (G + kRunRows - 1) / kRunRows;
    HI = (G + HG - 1) / HG;
    TG = std::min(QL, std::max(1, kRunRows / G));
    NT = (QL + TG - 1) / TG;
    NR = TG * HI;
    grid = sms * kRunCtas;
    ml = align256((size_t)grid * 2 * NR * D * sizeof(float));
    cut = ml + align256((size_t)grid * 2 * NR * sizeof(float2));
    total = cut + align256((size_t)grid * sizeof(int4));
  }
};

// Parameters and workspace of a call; the scale is the format's matter.
inline DecodeBlocksParams run_params(const DecodeBlocksCall& c, const RunPlan& plan) {
  DecodeBlocksParams p;
  memset(&p, 0, sizeof(p));
  char* ws = static_cast<char*>(c.workspace);
  p.q = static_cast<const __nv_bfloat16*>(c.q);
  p.k_cache = static_cast<const uint8_t*>(c.k_cache);
  p.v_cache = static_cast<const uint8_t*>(c.v_cache);
  p.page_table = c.page_table;
  p.seq_lens = c.seq_lens;
  p.rel = c.rel;
  p.out = static_cast<__nv_bfloat16*>(c.out);
  p.lse_out = c.lse_out;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.ml);
  p.cut = reinterpret_cast<int4*>(ws + plan.cut);
  p.dev_err = c.dev_err;
  p.B = c.B;
  p.pt_stride = c.pt_stride;
  p.H_q = c.H_q;
  p.H_kv = c.H_kv;
  p.G = plan.G;
  p.P = c.P;
  p.num_pages = c.num_pages;
  p.R = c.R;
  p.window = c.window;
  p.QL = c.QL;
  p.TG = plan.TG;
  p.HI = plan.HI;
  p.HG = plan.HG;
  p.NT = plan.NT;
  p.inv_G = 255 / plan.G + 1;
  p.inv_P = (uint32_t)(0xffffffffu / (uint32_t)c.P) + 1;
  p.NR = plan.NR;
  p.bias_prefetch = c.R % 4 == 0 && (reinterpret_cast<uintptr_t>(c.rel) & 15) == 0;
  return p;
}

// Whether a head's tiles, over all its items, can be counted in 32 bits.
inline bool run_countable(const DecodeBlocksCall& c, const RunPlan& plan) {
  return ((int64_t)c.pt_stride * c.P / kRunTile + 2) * plan.NT * plan.HG <= INT32_MAX;
}

// Ring slots of a thread block: a multiple of the warps, so a slot always belongs to the
// same one, which so waits for every phase of its barrier.
constexpr int kRunSmemBudget = kRunSmemPerSm / kRunCtas - 1024;
inline int run_slots(int block_bytes, int D, int NR) {
  int slots = 8 * kRunW;
  while (slots > kRunW && RunSmem(block_bytes, D, NR, slots).total > kRunSmemBudget) slots -= kRunW;
  return slots;
}

// Dispatch over head size and rows of several tokens.  L::launch<D, MULTI>(c, p, plan, smem) sends the
// two kernels; scale: what the format multiplies its products by.
template <class F, class L>
int launch_blocks(const DecodeBlocksCall& c, float scale) {
  const RunPlan plan(c.QL, c.H_q, c.H_kv, c.D, c.sms);
  if (!run_countable(c, plan)) return INKLING_ERR_ARG;
  DecodeBlocksParams p = run_params(c, plan);
  p.scale = scale;
  const int block_bytes = F::block_bytes(c.D);
  p.slots = run_slots(block_bytes, c.D, plan.NR);
  const int smem = RunSmem(block_bytes, c.D, plan.NR, p.slots).total;
  bool ok;
  if (c.D == 128)
    ok = plan.TG == 1 ? L::template launch<128, false>(c, p, plan, smem) : L::template launch<128, true>(c, p, plan, smem);
  else
    ok = plan.TG == 1 ? L::template launch<64, false>(c, p, plan, smem) : L::template launch<64, true>(c, p, plan, smem);
  return ok ? INKLING_OK : INKLING_ERR_CUDA;
}

}  // namespace ira

// Decode attention with the relative-position bias over the 4-bit cache.
//
// Operation: inkling_rel_attn_decode_q4 in include/inkling_rel_attn.h.
//
// Work.  An item is a (sequence, KV head, token group, head group); its rows are the
// group's (token, query head) pairs, at most 8, and its keys the visible range in
// tiles of two 16-token blocks.  (More rows in two MMA columns would read K and V
// once for them, but need twice the accumulators: 64 query heads over 4 KV heads
// took 116 us so and 95 us as two items, the second of which finds K and V in L2.)
// All tiles of the batch, in (sequence, head, group, key) order, are cut into one
// equal run per thread block of a grid that fills the GPU, so every one streams the
// same bytes whatever the lengths are.  An item inside a run is finished there; the
// parts of one that is cut go to the workspace as (m, l, O), at most two per thread
// block, and a second kernel joins them.  The cuts depend on the lengths alone, not
// on page ids or timing.
//
// A thread block has two producer warps and four consumer warps.  One producer
// walks the run, looks pages up and brings each tile's K and V (9 D bytes per block
// each, contiguous) into a ring of slots by bulk copy, a lane per tile; the ring runs
// across items, so the next one streams in while the current one is finished.  The
// other prepares the items (q as operands, bias pointers and positions per lane),
// three ahead.  Consumer warp w takes the ring's tiles w, w + 4, ... with an online
// softmax of its own; at the item's end it leaves (m, l, O) in one of two
// shared-memory buffers and goes on, and the preparing warp adds the parts up.  (One
// producer, and the last consumer to leave its part adding them up: 64 sequences of
// 512 visible keys 36.9 us instead of 31.9, for the copies stalled at every item
// and the slowest consumer was held up further.)
// Four warps load the SM's four schedulers alike (six, which give two of them two
// thirds of the work, took 195 us where four took 182), and a consumer's loop has
// no second copy for masked tiles (instruction fetches count in a short call).
// 32 sequences of 4096 .. 32768 keys, 48 heads over 8, D = 128: 144 us, 4.8 TB/s; 64
// sequences with 512 visible keys, 48 over 16: 30.4 us; without any arithmetic the
// two take 109 and 21 us, so the first is bound by the consumers' instructions, the
// second by what an item of 17 tiles costs beside them.
//
// Per block a warp forms S^T = K Q^T (16 keys x rows) and O^T += V^T P^T with
// mma.sync (rows are the N side, so 3 or 6 heads waste no M):
//  * a nibble is a bf16 operand where it stands (q4_expand): one logic instruction
//    for two values;
//  * the excess 8 over x = u - 8 is taken out by products: of the scales and
//    -8 sum(q) for K (one more product for all groups), and of a constant -8 and the
//    same rounded P for V, put together every few blocks;
//  * a group's scale is a factor of its own accumulator for K, in fp32, and of
//    P for V, before P is rounded to bf16 (the operand type of the product; 2^-8
//    of a weight at most, as the bf16 cache's decode rounds it).
// (8-bit products would need fewer operands, but mma.sync makes them of 16-bit ones.)
// Hidden keys get the bias -inf, so P = 0, and scales of 0: a page's unused places
// may hold anything.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "async.cuh"
#include "internal.h"
#include "launch.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "q4.cuh"
#include "tc.cuh"

namespace ira {

constexpr int kDq4ItemSlots = 3;      // items published ahead
constexpr int kDq4MinRun = 2;         // tiles of a run at least (2 sequences of 2 heads: 7.4 us, with 8 13.9)
constexpr int kDq4SmemPerSm = 222 * 1024;
constexpr float kDq4Slack = 5.5f;     // scores may exceed the exponent base by e^5.5 before it moves
constexpr int kDq4W = 4;              // consumer warps
constexpr int kDq4Ctas = 2;           // thread blocks per SM
constexpr int kDq4Threads = 32 * (kDq4W + 2);
constexpr int kDq4MergeWarps = 4;     // of the joining kernel's blocks: a thread per channel in all
constexpr int kDq4U = 2;              // 16-token blocks per tile
constexpr int kDq4Tile = 16 * kDq4U;  // keys per tile
static_assert(kDq4U == 2, "a tile's first and last block");
constexpr int kDq4Rows = 8;           // rows of an item at most: the N of an MMA

struct DecodeQ4Params {
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
  int slots;           // ring slots
  int bias_prefetch;   // rel_logits rows are 16-byte aligned
  float scale;         // of the products, which are 1 / kDown of <q, k>
};

// Part of an item: tiles tile0 .. tile0 + ntile - 1 of the item's sequence.
struct Dq4Item {
  int row0;  // packed row (token * H_q + head) of its first token and head
  int tn, heads, pos0;
  int tile0, ntile;
  int part;  // -1: the whole item; else its part number of this thread block
};

// What the producer prepares of an item, per lane of a consumer.
struct Dq4Prep {
  const float* bias[2];  // of score columns 2t, 2t + 1: the element at the position of MMA row g's key 0
  float far[2];          // bias at and past the table's end
  int pos[2];
  uint32_t qs[2];        // B fragment of -8 sum(q): k = N * part + group, three bf16 parts
  uint32_t pad[2];
};  // 48 bytes; the q fragments (16 bytes a group) follow

// Shared memory (byte offsets from a 128-byte aligned base).
struct Dq4Smem {
  int slot_bytes, item_bytes, prep_off, frag_off, item_off, comb_off, comb_floats, bar_off, total;
  __host__ __device__ Dq4Smem(int D, int NR, int slots) {
    slot_bytes = 2 * kDq4U * q4_block_bytes(D);      // K of the blocks, V of the blocks
    prep_off = 64;                                   // [3][32] of 16 bytes
    frag_off = prep_off + 32 * 48;                   // [D / 32][32] of 16 bytes
    item_bytes = frag_off + (D / 32) * 32 * 16;
    item_off = (slots * slot_bytes + 127) & ~127;
    comb_off = item_off + kDq4ItemSlots * item_bytes;
    comb_floats = kDq4W * NR * (D + 4) + 2 * kDq4W * kDq4Rows;
    bar_off = comb_off + 2 * comb_floats * 4;
    total = bar_off + (2 * slots + 2 * kDq4ItemSlots + 4) * 8 + 16;
  }
};

// Nibble n (0..3) of both halves of w, in place: bits 0..3 (n = 0, 2) or 4..7
// (n = 1, 3) of a half read as bf16 are u or 16 u times 2^-133 exactly, since a
// bf16's bits below 2^8 are linear in its value (its subnormals and the first
// octave above).  One logic instruction for two values, a shift for every four.
template <int n>
__device__ __forceinline__ uint32_t q4_expand(uint32_t w) {
  return (n >= 2 ? w >> 8 : w) & ((n & 1) ? 0x00f000f0u : 0x000f000fu);
}
// The other operand (q, P) carries 2^60, so the products lie at 2^-73 of their
// value, in the middle of fp32's range; for odd n q carries 2^56, and an output of V
// is 16 times its value instead.  Scales of V from 2^-40 to 2^55 and q up to 2^60
// leave everything in range.
constexpr float kDown = 0x1p73f;
constexpr uint32_t kMinus8 = 0x80088008u, kMinus128 = 0x80808080u;  // -8 and -128, in the same units
template <int e>
__device__ __forceinline__ uint32_t times_pow2(uint32_t bf16_pair) {  // exact
  constexpr uint32_t k = (uint32_t)(127 + e) << 7;
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(bf16_pair), "r"(k | k << 16));
  return r;
}

// mma_16816 into a new accumulator.
__device__ __forceinline__ void mma_16816_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

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
struct Dq4Range {
  int tn, pos0, tile0, ntile;
};
__device__ __forceinline__ Dq4Range group_range(const DecodeQ4Params& p, int L, int tg) {
  Dq4Range r;
  const int first = tg * p.TG;
  r.tn = min(p.TG, p.QL - first);
  r.pos0 = L - p.QL + first;
  const int lo = p.window > 0 ? max(0, r.pos0 - p.window + 1) : 0;
  r.tile0 = lo / kDq4Tile;
  r.ntile = (r.pos0 + r.tn - 1) / kDq4Tile - r.tile0 + 1;
  return r;
}
__device__ __forceinline__ int clamped_len(const DecodeQ4Params& p, int b) {
  return min(max(p.seq_lens[b], 0), p.pt_stride * p.P);
}
// Tiles of one KV head of sequence b (all its items); 0 when it has fewer keys than new tokens.
__device__ __forceinline__ int head_tiles(const DecodeQ4Params& p, int b) {
  const int L = clamped_len(p, b);
  if (L < p.QL) return 0;
  int n = 0;
  for (int tg = 0; tg < p.NT; ++tg) n += group_range(p, L, tg).ntile;
  return n * p.HG;
}

// MULTI: items of several tokens, so rows of several positions.
template <int D, bool MULTI>
__global__ void __launch_bounds__(kDq4Threads, kDq4Ctas)
    decode_q4_kernel(const __grid_constant__ DecodeQ4Params p) {
  constexpr int W = kDq4W, U = kDq4U, TK = kDq4Tile;
  constexpr int N = D / kQ4Group;  // groups of a row
  constexpr int HP = kDq4Rows;
  constexpr int OP = D + 4;
  constexpr int BLK = q4_block_bytes(D);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int NR = p.NR, slots = p.slots;
  const Dq4Smem S(D, NR, slots);
  // the warps' parts of an item, two buffers in turn: O [W][NR][D + 4], m [W][HP], l [W][HP]
  auto comb_o = [&](int s) { return reinterpret_cast<float*>(smem + S.comb_off) + s * S.comb_floats; };
  auto comb_m = [&](int s) { return comb_o(s) + W * NR * OP; };
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S.bar_off);  // ring slots
  uint64_t* empty = full + slots;
  uint64_t* ifull = empty + slots;           // items: published,
  uint64_t* iempty = ifull + kDq4ItemSlots;  // taken by every consumer
  uint64_t* cfull = iempty + kDq4ItemSlots;  // parts of an item: left by every consumer,
  uint64_t* cempty = cfull + 2;              // added up
  volatile int* abort_flag = reinterpret_cast<int*>(cempty + 2);
  auto item_at = [&](int s) { return smem + S.item_off + s * S.item_bytes; };
  auto item_rec = [&](int s) { return reinterpret_cast<Dq4Item*>(item_at(s)); };
  // token of an item's row r, and its packed row
  auto token_of = [&](int r) { return MULTI ? (r * p.inv_G) >> 8 : 0; };
  auto row_of = [&](const Dq4Item& it, int r) {
    const int i = token_of(r);
    return (size_t)it.row0 + (size_t)i * p.H_q + (r - i * it.heads);
  };
  // Key of a block that MMA row g (and g + 8: 8 more) stands for: rows 2t, 2t + 1
  // are keys t, 4 + (t ^ 1), so that the 64-byte rows read together lie in both halves
  // of the shared-memory banks, for K (rows 2t, 2t + 1 at once) and V (t = 0..3 at once).
  const int key_g = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;

  for (int i = tid; i < slots; i += kDq4Threads) {
    mbar_init(smem_u32(full + i), 1);
    mbar_init(smem_u32(empty + i), 1);
  }
  if (tid == 0) {
    for (int i = 0; i < kDq4ItemSlots; ++i) {
      mbar_init(smem_u32(ifull + i), 1);
      mbar_init(smem_u32(iempty + i), W);
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
  // Both walk the run: warp W sends the tiles, warp W + 1 prepares the items.
  if (warp >= W) {
    const bool copier = warp == W;
    // ---- this thread block's run [x, x1) of the batch's tiles
    int64_t total = 0;
    for (int b = lane; b < p.B; b += 32) {
      total += (int64_t)p.H_kv * head_tiles(p, b);
      if (copier && blockIdx.x == 0) {
        const int Lr = p.seq_lens[b];
        if (Lr > p.pt_stride * p.P) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
        if (p.QL > 1 && Lr < p.QL) report(p.dev_err, INKLING_DEVERR_BAD_CHUNK);
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    const int64_t runs = min((int64_t)gridDim.x, max((total + kDq4MinRun - 1) / kDq4MinRun, (int64_t)1));
    int64_t x = total, x1 = total;
    if (blockIdx.x < runs) {
      x = total * blockIdx.x / runs;
      x1 = total * (blockIdx.x + 1) / runs;
    }
    // ---- the item at x
    int b = 0, hkv = 0, tg = 0, hg = 0, nb = 0, off = 0, L = 0;  // nb: tiles per head of sequence b
    if (x < x1) {
      int64_t carry = 0;
      for (int b0 = 0;; b0 += 32) {
        const int bb = b0 + lane;
        const int mine = bb < p.B ? head_tiles(p, bb) : 0;
        int64_t incl = (int64_t)p.H_kv * mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, carry + incl > x);
        if (past) {
          const int src = __ffs(past) - 1;
          b = b0 + src;
          nb = __shfl_sync(0xffffffffu, mine, src);
          const int64_t at = x - (carry + __shfl_sync(0xffffffffu, incl, src) - (int64_t)p.H_kv * nb);
          hkv = (int)(at / nb);
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
    // ---- q operands of an item (channel order of the K rows), and -8 sum(q) of every
    // group as an operand of one more product, with the block's scales:
    // sum_j s_j (-8 sum_j(q)).
    auto prepare = [&](const Dq4Item& it, int is) {
      const int rows = it.tn * it.heads;
      const uint4* qr = reinterpret_cast<const uint4*>(p.q + row_of(it, min(g, rows - 1)) * D) + t;
      float sum[N];
      uint4 qw[N];
#pragma unroll
      for (int j = 0; j < N; ++j) qw[j] = qr[4 * j];  // channels 32j + 8t + 0..7
      uint4* frag = reinterpret_cast<uint4*>(item_at(is) + S.frag_off) + lane;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        uint4 w = qw[j];
        if (g >= rows) w = make_uint4(0, 0, 0, 0);
        uint4 f;  // c, c + 4 for c = 0..3
        f.x = times_pow2<60>(__byte_perm(w.x, w.z, 0x5410));
        f.y = times_pow2<56>(__byte_perm(w.x, w.z, 0x7632));
        f.z = times_pow2<60>(__byte_perm(w.y, w.w, 0x5410));
        f.w = times_pow2<56>(__byte_perm(w.y, w.w, 0x7632));
        frag[32 * j] = f;
        float c[4];
        mma_16816_new(c, kMinus8, kMinus8, kMinus128, kMinus128, f.x, f.y);
        mma_16816(c, kMinus8, kMinus8, kMinus128, kMinus128, f.z, f.w);
        // every row of c is the same; this lane takes column g
        const float c0 = __shfl_sync(0xffffffffu, c[0], g >> 1), c1 = __shfl_sync(0xffffffffu, c[1], g >> 1);
        sum[j] = (g & 1) ? c1 : c0;
      }
      // k = 2t, 2t + 1 and 2t + 8, 2t + 9 of column g
      auto part = [&](float v, int i) {  // part i of v's three bf16 parts
        float h = __bfloat162float(__float2bfloat16(v));
        if (i == 0) return h;
        v -= h;
        h = __bfloat162float(__float2bfloat16(v));
        return i == 1 ? h : v - h;
      };
      const float lo_ = N == 2 || !(t & 1) ? sum[0] : sum[N - 2], hi_ = N == 2 || !(t & 1) ? sum[1] : sum[N - 1];
      const int p0 = N == 2 ? t : t >> 1;  // of k = 2t; k = 2t + 8 is two further on
      Dq4Prep pr;
      pr.pad[0] = pr.pad[1] = 0u;
      pr.qs[0] = p0 < 3 ? pack_bf16(part(lo_, p0), part(hi_, p0)) : 0u;
      pr.qs[1] = N == 4 && t < 2 ? pack_bf16(part(lo_, 2), part(hi_, 2)) : 0u;
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
    // ---- the sum of the warps' parts of an item
    // lane W * r + w makes the factor of warp w's part of row r.  (Short code: this warp
    // shares the instruction cache with the consumers' loop; unrolled by 4, 11 us more
    // for 64 sequences of 4 drafts.)
    auto join = [&](const Dq4Item& it, int cb) {
      static_assert(W * HP == 32, "a lane per row and warp");
      constexpr int LR = D / 4;  // lanes per row
      const float* co = comb_o(cb);
      const float* cm = comb_m(cb);
      const int rows = it.tn * it.heads, d = 4 * (lane % LR);
      const float m = cm[lane % W * HP + lane / W];
      float M = m;
#pragma unroll
      for (int off = 1; off < W; off <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      float f = ex2((m - (M == -INFINITY ? 0.f : M)) * kLog2e);
      float l = f * cm[(W + lane % W) * HP + lane / W];
#pragma unroll
      for (int off = 1; off < W; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      const bool mine = lane % W == 0 && lane / W < rows;
      if (it.part < 0) {
        f *= l == 0.f ? 0.f : __fdividef(1.f, l);  // every score -inf: an empty row
        if (mine && p.lse_out) p.lse_out[row_of(it, lane / W)] = M + logf(l);
      } else if (mine) {
        p.part_ml[((size_t)blockIdx.x * 2 + it.part) * NR + lane / W] = make_float2(M, l);
      }
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += 32 / LR) {
        const int r = r0 + lane / LR;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float fw = __shfl_sync(0xffffffffu, f, min(W * r + w, 31));
          const float4 v = *reinterpret_cast<const float4*>(co + (w * NR + min(r, rows - 1)) * OP + d);
          a.x = fmaf(fw, v.x, a.x);
          a.y = fmaf(fw, v.y, a.y);
          a.z = fmaf(fw, v.z, a.z);
          a.w = fmaf(fw, v.w, a.w);
        }
        if (r >= rows) continue;
        if (it.part < 0)
          *reinterpret_cast<uint2*>(p.out + row_of(it, r) * D + d) =
              make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
        else
          *reinterpret_cast<float4*>(p.part_o + (((size_t)blockIdx.x * 2 + it.part) * NR + r) * D + d) = a;
      }
    };
    auto join_item = [&](int k) -> bool {
      const int cb = k & 1;
      if (!waitw(smem_u32(cfull + cb), (k >> 1) & 1, abort_flag)) return false;
      const Dq4Item it = *item_rec(k % kDq4ItemSlots);
      join(it, cb);
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(cempty + cb));
      return true;
    };
    auto publish = [&](const Dq4Item& it) -> bool {
      const int s = ki % kDq4ItemSlots;
      bool good = true;
      if (ki >= kDq4ItemSlots && lane == 0)
        good = wait1(smem_u32(iempty + s), ((ki / kDq4ItemSlots) - 1) & 1, abort_flag);
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
      const Dq4Range r = group_range(p, L, tg);
      Dq4Item it;
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
          const int last = (int)(((e + 1) * runs - 1) / total);
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
      if (!copier) ok = publish(it) && (ki < 3 || join_item(ki - 3));
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
        return copier && lane < batch && i < it.ntile && seen(key, u) ? pt_row[key / p.P] : -1;
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
          place[u] = (key0 + 16 * u) % p.P;
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
          for (int u = 0; u < 3; ++u) left = (left & (left - 1)) ? left & (left - 1) : left;
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
              // a bad page reads as zeros: scale 0 (16 * N bf16 of K and of V); of a block that
              // no row sees nothing is needed
              if (!fine[u] && seen(key0 + 16 * u, u)) {
#pragma unroll 1
                for (int w = 0; w < 8 * N; ++w) {
                  reinterpret_cast<uint32_t*>(dst + u * BLK + q4_scale_off(D))[w] = 0u;
                  reinterpret_cast<uint32_t*>(dst + (U + u) * BLK + q4_scale_off(D))[w] = 0u;
                }
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
        Dq4Item end;
        memset(&end, 0, sizeof(end));
        const int n = ki;
        ok = publish(end) && (n < 2 || join_item(n - 2)) && (n < 1 || join_item(n - 1));  // ntile = 0: no more items
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
  // Constant operands of V's offset: rows g (m8[0]) or rows g + 8 (m8[1]) of the
  // product take -8 sum(P) of a group; kept in registers.
  uint32_t m8[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm volatile("mov.b32 %0, %1;" : "=r"(m8[0][i]) : "r"((i & 1) ? 0u : kMinus8));
    asm volatile("mov.b32 %0, %1;" : "=r"(m8[1][i]) : "r"((i & 1) ? kMinus8 : 0u));
  }
  const int row_k = key_g * (D / 2) + 4 * N * t;                 // this lane's part of a K row
  const int row_v0 = t * (D / 2) + 2 * N * g, row_v1 = (4 + (t ^ 1)) * (D / 2) + 2 * N * g;  // and of V rows
  const int row_s = q4_scale_off(D) + key_g * (2 * N);           // and of the scales

  int kb_w = 0;       // tiles of the items before this one, modulo W
  int s_slot = warp;  // this warp's next slot (it owns warp, warp + W, ...) and its phase
  uint32_t s_phase = 0;
  bool ok = true;
  for (int ki = 0;; ++ki) {
    const int is = ki % kDq4ItemSlots;
    if (!waitw(smem_u32(ifull + is), (ki / kDq4ItemSlots) & 1, abort_flag)) {
      ok = false;
      break;
    }
    const Dq4Item it = *item_rec(is);
    if (it.ntile == 0) break;
    uint4 qf[N];
    Dq4Prep pr;
    const uint4* frag = reinterpret_cast<const uint4*>(item_at(is) + S.frag_off) + lane;
    const uint4* src = reinterpret_cast<const uint4*>(item_at(is) + S.prep_off) + lane;
#pragma unroll
    for (int j = 0; j < N; ++j) qf[j] = frag[32 * j];
#pragma unroll
    for (int i = 0; i < 3; ++i) reinterpret_cast<uint4*>(&pr)[i] = src[32 * i];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(iempty + is));
    const int pos0 = it.pos0, pos1 = it.pos0 + it.tn - 1;

    // O and, for groups 2i (x = 0, 1) and 2i + 1 (x = 2, 3), -8 sum(P s): O holds u, not
    // u - 8, until the two are put together
    float m_run[2], l_run[2], o[N][2][4], co[N / 2][4];
    m_run[0] = m_run[1] = -INFINITY;
    l_run[0] = l_run[1] = 0.f;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
#pragma unroll
      for (int j = 0; j < N; ++j) o[j][0][x] = o[j][1][x] = 0.f;
#pragma unroll
      for (int j = 0; j < N / 2; ++j) co[j][x] = 0.f;
    }

    // ---- this warp's tiles of the item
    int i = warp - kb_w;
    if (i < 0) i += W;
    kb_w = (kb_w + it.ntile) % W;
    for (int turn = 1;; i += W, ++turn) {
      const bool last = i >= it.ntile;
      if (last || (turn & 7) == 0) {
        // put O and its offset together: at the end, and often enough that the offset's
        // rounding does not add up (rows of odd nibbles hold 16 times their value)
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float& c = co[j >> 1][2 * (j & 1) + x];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              o[j][h][x] += c;
              o[j][h][x + 2] = fmaf(c, 16.f, o[j][h][x + 2]);
            }
            c = 0.f;
          }
        if (last) break;
      }
      const int key0 = (it.tile0 + i) * TK;
      // ---- bias, on its way while the tile is awaited and K multiplied
      const bool inside = key0 + TK - 1 <= pos0 && (p.window <= 0 || pos1 - key0 < p.window);
      float bv[U][4];
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
            bv[u][x] = dist >= 0 && (p.window <= 0 || dist < p.window) ? v : -INFINITY;
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
      if (!inside) {  // keys that no row sees get scales of 0: their places may hold NaN
        const int key = key0 + lane, first = p.window > 0 ? pos0 - p.window + 1 : 0;
        if (lane < TK && (key > pos1 || key < first)) {
          uint8_t* sk = ring_slot + (lane >> 4) * BLK + q4_scale_off(D) + (lane & 15) * (2 * N);
#pragma unroll
          for (int j = 0; j < N / 2; ++j) {
            reinterpret_cast<uint32_t*>(sk)[j] = 0u;
            reinterpret_cast<uint32_t*>(sk + U * BLK)[j] = 0u;
          }
        }
        fence_proxy_async_smem();  // before the slot's next copy
        __syncwarp();
      }
      // scales of rows g (x = 0) and g + 8, two groups to a word
      auto load_scales = [&](const uint8_t* blk, uint32_t (&sc)[2][N / 2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t* at = blk + row_s + x * 16 * N;
          if constexpr (N == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(at);
            sc[x][0] = v.x;
            sc[x][N / 2 - 1] = v.y;
          } else {
            sc[x][0] = *reinterpret_cast<const uint32_t*>(at);
          }
        }
      };
      auto scale_of = [&](const uint32_t (&sc)[2][N / 2], int x, int j) {
        return __uint_as_float((j & 1) ? sc[x][j >> 1] & 0xffff0000u : sc[x][j >> 1] << 16);
      };
      // ---- scores of 16 keys x rows, from sum_j s_j (-8 sum_j(q)) on
      float sc[U][4];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint8_t* kp = ring_slot + u * BLK;
        uint32_t kw[2][N], ksc[2][N / 2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint8_t* kr = kp + row_k + x * 4 * D;
          if constexpr (N == 4) {
            const uint4 a = *reinterpret_cast<const uint4*>(kr);
            kw[x][0] = a.x;
            kw[x][1] = a.y;
            kw[x][N - 2] = a.z;
            kw[x][N - 1] = a.w;
          } else {
            const uint2 a = *reinterpret_cast<const uint2*>(kr);
            kw[x][0] = a.x;
            kw[x][1] = a.y;
          }
        }
        load_scales(kp, ksc);
        const int w = N == 4 ? t & 1 : 0;  // scales of groups 2w, 2w + 1 against k = 2t, 2t + 1 (and + 8)
        const uint32_t z0 = w ? ksc[0][N / 2 - 1] : ksc[0][0], z1 = w ? ksc[1][N / 2 - 1] : ksc[1][0];
        mma_16816_new(sc[u], z0, z1, z0, z1, pr.qs[0], pr.qs[1]);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t a0 = q4_expand<0>(kw[0][j]), a1 = q4_expand<0>(kw[1][j]), a2 = q4_expand<1>(kw[0][j]),
                         a3 = q4_expand<1>(kw[1][j]);
          const uint32_t b0 = q4_expand<2>(kw[0][j]), b1 = q4_expand<2>(kw[1][j]), b2 = q4_expand<3>(kw[0][j]),
                         b3 = q4_expand<3>(kw[1][j]);
          const float s0 = scale_of(ksc, 0, j), s8 = scale_of(ksc, 1, j);
          float c[4];
          mma_16816_new(c, a0, a1, a2, a3, qf[j].x, qf[j].y);
          mma_16816(c, b0, b1, b2, b3, qf[j].z, qf[j].w);
          sc[u][0] = fmaf(c[0], s0, sc[u][0]);
          sc[u][1] = fmaf(c[1], s0, sc[u][1]);
          sc[u][2] = fmaf(c[2], s8, sc[u][2]);
          sc[u][3] = fmaf(c[3], s8, sc[u][3]);
        }
      }
      if (far) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[u][x] = fmaf(sc[u][x], p.scale, pr.far[x & 1]);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            sc[u][x] = fmaf(sc[u][x], p.scale, bv[u][x]);
            if constexpr (MULTI) sc[u][x] = bv[u][x] == -INFINITY ? -INFINITY : sc[u][x];  // its scale may be NaN
          }
      }
      // ---- running maximum and sum.  The maximum, the exponents' base, is
      // taken anew over the warp only when a score passes it by kDq4Slack;
      // until then a weight is at most e^kDq4Slack and nothing is rescaled.
      float mx[2] = {fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[0][1], sc[0][3])};
#pragma unroll
      for (int u = 1; u < U; ++u) {
        mx[0] = fmaxf(mx[0], fmaxf(sc[u][0], sc[u][2]));
        mx[1] = fmaxf(mx[1], fmaxf(sc[u][1], sc[u][3]));
      }
      if (__any_sync(0xffffffffu, mx[0] > m_run[0] + kDq4Slack || mx[1] > m_run[1] + kDq4Slack)) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], off));
          const float mn = fmaxf(m_run[x], mx[x]);
          const float al = mn == -INFINITY ? 1.f : ex2((m_run[x] - mn) * kLog2e);
          l_run[x] *= al;
          m_run[x] = mn;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            co[j >> 1][2 * (j & 1) + x] *= al;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              o[j][h][x] *= al;
              o[j][h][x + 2] *= al;
            }
          }
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
      // ---- O^T += V^T P^T
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint8_t* vp = ring_slot + (U + u) * BLK;
        uint32_t vw[4][N / 2], vsc[2][N / 2];
        load_scales(vp, vsc);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint8_t* vr = vp + ((x & 1) ? row_v1 : row_v0) + (x >> 1) * 4 * D;
          if constexpr (N == 4) {
            const uint2 v = *reinterpret_cast<const uint2*>(vr);
            vw[x][0] = v.x;
            vw[x][N / 2 - 1] = v.y;
          } else {
            vw[x][0] = *reinterpret_cast<const uint32_t*>(vr);
          }
        }
        if (u == U - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(eb);  // the tile is in registers
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int j = 0; j < N / 2; ++j) vsc[x][j] = times_pow2<60>(vsc[x][j]);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const float s0 = scale_of(vsc, 0, j), s8 = scale_of(vsc, 1, j);
          uint32_t pb[2];
          float w[4] = {sc[u][0] * s0, sc[u][1] * s0, sc[u][2] * s8, sc[u][3] * s8};
          if constexpr (MULTI) {  // a key hidden from some of the rows: its scale may be NaN
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = sc[u][x] == 0.f ? 0.f : w[x];
          }
          pb[0] = movmatrix_t(pack_bf16(w[0], w[1]));
          pb[1] = movmatrix_t(pack_bf16(w[2], w[3]));
          const uint32_t sel = (j & 1) ? 0x7632 : 0x5410;
          const uint32_t w0 = __byte_perm(vw[0][j >> 1], vw[1][j >> 1], sel);
          const uint32_t w8 = __byte_perm(vw[2][j >> 1], vw[3][j >> 1], sel);
          const uint32_t a0 = q4_expand<0>(w0), a1 = q4_expand<1>(w0), a2 = q4_expand<0>(w8), a3 = q4_expand<1>(w8);
          const uint32_t b0 = q4_expand<2>(w0), b1 = q4_expand<3>(w0), b2 = q4_expand<2>(w8), b3 = q4_expand<3>(w8);
          mma_16816(co[j >> 1], m8[j & 1][0], m8[j & 1][1], m8[j & 1][2], m8[j & 1][3], pb[0], pb[1]);
          mma_16816(o[j][0], a0, a1, a2, a3, pb[0], pb[1]);
          mma_16816(o[j][1], b0, b1, b2, b3, pb[0], pb[1]);
        }
      }
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
      if (r < it.tn * it.heads) {
#pragma unroll
        for (int j = 0; j < N; ++j)  // channels 32j + 4g + 0..3
          *reinterpret_cast<float4*>(comb_o(cb) + (warp * NR + r) * OP + 32 * j + 4 * g) =
              make_float4(o[j][0][x] * kDown, o[j][0][x + 2] * (kDown / 16), o[j][1][x] * kDown,
                          o[j][1][x + 2] * (kDown / 16));
      }
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
__global__ void __launch_bounds__(32 * kDq4MergeWarps) merge_q4_kernel(const __grid_constant__ DecodeQ4Params p) {
  await_previous_kernel();
  constexpr int C = D / 32;
  const int4 cut = p.cut[blockIdx.x];
  const int r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float s_o[kDq4MergeWarps][D];
  __shared__ float2 s_ml[kDq4MergeWarps];
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
  for (int k = warp + kDq4MergeWarps; k < cut.z; k += kDq4MergeWarps) {
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
  for (int w = 0; w < kDq4MergeWarps; ++w) M = fmaxf(M, s_ml[w].x);
  const float base = M == -INFINITY ? 0.f : M;
  float o = 0.f;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kDq4MergeWarps; ++w) {
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

struct Dq4Plan {
  int G, TG, HI, HG, NT, NR, grid;
  size_t ml, cut, total;  // workspace offsets: parts first
  Dq4Plan(int32_t QL, int32_t H_q, int32_t H_kv, int32_t D, int32_t sms) {
    G = H_q / H_kv;
    HG = (G + kDq4Rows - 1) / kDq4Rows;
    HI = (G + HG - 1) / HG;
    TG = std::min(QL, std::max(1, kDq4Rows / G));
    NT = (QL + TG - 1) / TG;
    NR = TG * HI;
    grid = sms * kDq4Ctas;
    ml = align256((size_t)grid * 2 * NR * D * sizeof(float));
    cut = ml + align256((size_t)grid * 2 * NR * sizeof(float2));
    total = cut + align256((size_t)grid * sizeof(int4));
  }
};

size_t decode_q4_workspace_bytes(int32_t, int32_t QL, int32_t H_q, int32_t H_kv, int32_t D, int32_t sms) {
  return Dq4Plan(QL, H_q, H_kv, D, sms).total;
}

template <int D, bool MULTI>
static int launch_decode_q4_t(const DecodeQ4Call& c, DecodeQ4Params prm, const Dq4Plan& plan) {
  const int budget = kDq4SmemPerSm / kDq4Ctas - 1024;
  // a multiple of the warps: a slot always belongs to the same one, which so waits for
  // every phase of its barrier
  int slots = 8 * kDq4W;
  while (slots > kDq4W && Dq4Smem(D, plan.NR, slots).total > budget) slots -= kDq4W;
  prm.slots = slots;
  const int smem = Dq4Smem(D, plan.NR, slots).total;
  auto kern = decode_q4_kernel<D, MULTI>;
  static std::atomic<int> limit_set[kMaxDevices];
  if (!smem_limit_on_device(reinterpret_cast<const void*>(kern), budget, limit_set)) return INKLING_ERR_CUDA;
  if (!launch_dependent(kern, dim3(plan.grid), kDq4Threads, smem, prm, c.stream)) return INKLING_ERR_CUDA;
  if (!launch_dependent(merge_q4_kernel<D>, dim3(plan.grid, plan.NR), 32 * kDq4MergeWarps, 0, prm, c.stream))
    return INKLING_ERR_CUDA;
  return INKLING_OK;
}

int launch_decode_q4(const DecodeQ4Call& c) {
  const Dq4Plan plan(c.QL, c.H_q, c.H_kv, c.D, c.sms);
  // a head's tiles, over all its items, are counted in 32 bits
  if (((int64_t)c.pt_stride * c.P / kDq4Tile + 2) * plan.NT * plan.HG > INT32_MAX) return INKLING_ERR_ARG;
  DecodeQ4Params p;
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
  p.NR = plan.NR;
  p.bias_prefetch = c.R % 4 == 0 && (reinterpret_cast<uintptr_t>(c.rel) & 15) == 0;
  p.scale = c.scale * kDown;
  if (c.D == 128)
    return plan.TG == 1 ? launch_decode_q4_t<128, false>(c, p, plan) : launch_decode_q4_t<128, true>(c, p, plan);
  return plan.TG == 1 ? launch_decode_q4_t<64, false>(c, p, plan) : launch_decode_q4_t<64, true>(c, p, plan);
}

}  // namespace ira

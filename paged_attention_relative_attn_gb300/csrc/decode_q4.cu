// Decode attention with the relative-position bias over the 4-bit cache.
//
// Operation: inkling_rel_attn_decode_q4 in include/inkling_rel_attn.h.
//
// Work.  An item is a (sequence, KV head, token group); its rows are the group's
// (token, query head) pairs, at most 16, and its keys the 16-token blocks of the
// visible range.  All blocks of the batch, in (sequence, head, group, key) order,
// are cut into one equal run per thread block of a grid that fills the GPU, so
// every one streams the same bytes whatever the lengths are.  An item inside a
// run is finished there; the parts of one that is cut go to the workspace as
// (m, l, O), at most two per thread block, and a second kernel joins them.
// The cuts depend on the lengths alone, not on page ids or timing.
//
// A thread block has one producer warp and W consumer warps.  The producer walks
// the run, looks pages up and brings each block's K and V (9 D bytes each,
// contiguous) into a ring of slots by bulk copy; the ring runs across items, so
// the next item streams in while the current one is finished.  It also
// publishes each item's record and q rows and prefetches its bias rows into L2.
// Consumer warp w takes the ring's blocks w, w + W, ... each on its own, with an
// online softmax of its own, and the warps are joined at the item's end.
//
// Per block a warp forms S^T = K Q^T (16 keys x rows) and O^T += V^T P^T with
// mma.sync m16n8k16 in bf16 (rows are the N side, so 3 or 6 heads waste no M):
//  * a nibble u becomes the bf16 number 128 + u by or-ing it into the mantissa
//    of 128 -- one instruction for two values; the excess 136 over x = u - 8 is
//    taken out by products: of the scales and -136 sum(q) for K (one more product
//    for all groups), and of a constant -136 and the same rounded P for V, block by
//    block, so that no large sums cancel later;
//  * a group's scale is a factor of its own accumulator for K, in fp32, and of
//    P for V, before P is rounded to bf16 (the operand type of the product; 2^-8
//    of a weight at most, as the bf16 cache's decode rounds it).
// Masked keys get P = 0 and scale 0: a page's unused places may hold anything.
#include <cuda_bf16.h>
#include <math.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "q4.cuh"

namespace ira {

constexpr int kDq4ItemSlots = 3;
constexpr int kDq4MinRun = 16;        // blocks of a run at least: fewer are not worth a cut
constexpr int kDq4SmemPerSm = 222 * 1024;
constexpr float kDq4Slack = 5.5f;     // scores may exceed the exponent base by e^5.5 before it moves

// Variants: one n-tile (up to 8 rows) or two.
template <int NT>
struct Dq4Shape {
  static constexpr int W = NT == 1 ? 7 : 3;     // consumer warps
  static constexpr int kCtas = 2;               // thread blocks per SM
  static constexpr int kThreads = 32 * (W + 1);
};

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
  int4* cut;        // [grid]: a cut item's first packed row, tokens, parts; parts 0: none
  int32_t* dev_err;
  int B, pt_stride, H_q, H_kv, G, P, num_pages, R, window;
  int QL, TG, NG, NR;  // query tokens per sequence, per item, items per (sequence, KV head), rows
  int slots;           // ring slots
  int bias_prefetch;   // rel_logits rows are 16-byte aligned
  float scale;
};

// Part of an item: blocks blk0 .. blk0 + nblk - 1 of the item's sequence.
struct Dq4Item {
  int row0;  // packed row (token * H_q + head) of its first token and head
  int tn, pos0;
  int blk0, nblk;
  int part;  // -1: the whole item; else its part number of this thread block
};

// Shared memory (byte offsets from a 128-byte aligned base).
struct Dq4Smem {
  int slot_bytes, item_bytes, item_off, comb_off, bar_off, total;
  __host__ __device__ Dq4Smem(int D, int NT, int NR, int W, int slots) {
    slot_bytes = 2 * q4_block_bytes(D);
    item_bytes = 64 + 8 * NT * D * 2;
    item_off = (slots * slot_bytes + 127) & ~127;
    comb_off = item_off + kDq4ItemSlots * item_bytes;
    bar_off = comb_off + (W * NR * (D + 4) + 2 * W * 8 * NT) * 4;
    total = bar_off + (2 * slots + 2 * kDq4ItemSlots) * 8 + 16;
  }
};

// Nibble n (0..3) of both halves of w as the bf16 pair 128 + u: (w >> 4n & mask) | 128, one lop3.
template <int n>
__device__ __forceinline__ uint32_t q4_expand(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w >> (4 * n)), "r"(0x000f000fu), "r"(0x43004300u));
  return r;
}
constexpr uint32_t kMinus136 = 0xc308c308u;

// mma_16816 into a new accumulator.
__device__ __forceinline__ void mma_16816_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Positions and blocks of token group `grp` of a sequence of length L >= QL.
struct Dq4Range {
  int tn, pos0, blk0, nblk;
};
__device__ __forceinline__ Dq4Range group_range(const DecodeQ4Params& p, int L, int grp) {
  Dq4Range r;
  const int first = grp * p.TG;
  r.tn = min(p.TG, p.QL - first);
  r.pos0 = L - p.QL + first;
  const int lo = p.window > 0 ? max(0, r.pos0 - p.window + 1) : 0;
  r.blk0 = lo >> 4;
  r.nblk = ((r.pos0 + r.tn - 1) >> 4) - r.blk0 + 1;
  return r;
}
__device__ __forceinline__ int clamped_len(const DecodeQ4Params& p, int b) {
  return min(max(__ldg(p.seq_lens + b), 0), p.pt_stride * p.P);
}
// Blocks of one KV head of sequence b (all its token groups); 0 when it has fewer keys than new tokens.
__device__ __forceinline__ int head_blocks(const DecodeQ4Params& p, int b) {
  const int L = clamped_len(p, b);
  if (L < p.QL) return 0;
  int n = 0;
  for (int g = 0; g < p.NG; ++g) n += group_range(p, L, g).nblk;
  return n;
}

template <int D, int NT>
__global__ void __launch_bounds__(Dq4Shape<NT>::kThreads, Dq4Shape<NT>::kCtas)
    decode_q4_kernel(const __grid_constant__ DecodeQ4Params p) {
  constexpr int W = Dq4Shape<NT>::W;
  constexpr int N = D / kQ4Group;  // groups of a row
  constexpr int HP = 8 * NT;
  constexpr int OP = D + 4;
  constexpr int BLK = q4_block_bytes(D);
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.G, NR = p.NR, slots = p.slots;
  const Dq4Smem S(D, NT, NR, W, slots);
  float* comb = reinterpret_cast<float*>(smem + S.comb_off);  // [W][NR][D + 4]
  float* comb_m = comb + W * NR * OP;                          // [W][HP]
  float* comb_l = comb_m + W * HP;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S.bar_off);
  uint64_t* empty = full + slots;
  uint64_t* rfull = empty + slots;
  uint64_t* rempty = rfull + kDq4ItemSlots;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(rempty + kDq4ItemSlots);
  auto item_rec = [&](int s) { return reinterpret_cast<Dq4Item*>(smem + S.item_off + s * S.item_bytes); };
  auto item_q = [&](int s) { return smem + S.item_off + s * S.item_bytes + 64; };

  for (int i = tid; i < slots; i += Dq4Shape<NT>::kThreads) {
    mbar_init(smem_u32(full + i), 1);
    mbar_init(smem_u32(empty + i), 1);
  }
  if (tid == 0) {
    for (int i = 0; i < kDq4ItemSlots; ++i) {
      mbar_init(smem_u32(rfull + i), 1);
      mbar_init(smem_u32(rempty + i), W);
    }
    *abort_flag = 0;
  }
  fence_mbar_init();
  __syncthreads();
  // launched with programmatic stream serialization: nothing of the previous
  // kernel's is read or overwritten before it has completed
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // =================================================================== producer
  if (warp == W) {
    // ---- this thread block's run [x, x1) of the batch's blocks
    int64_t total = 0;
    for (int b = lane; b < p.B; b += 32) {
      total += (int64_t)p.H_kv * head_blocks(p, b);
      if (blockIdx.x == 0) {
        const int Lr = __ldg(p.seq_lens + b);
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
    int b = 0, hkv = 0, grp = 0, nb = 0, off = 0, L = 0;  // nb: blocks per head of sequence b
    if (x < x1) {
      int64_t carry = 0;
      for (int b0 = 0;; b0 += 32) {
        const int bb = b0 + lane;
        const int mine = bb < p.B ? head_blocks(p, bb) : 0;
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
      while (off >= group_range(p, L, grp).nblk) off -= group_range(p, L, grp++).nblk;
    }

    int ki = 0, kb = 0;  // items and blocks published
    uint32_t sent = 0;   // on a time-out: the copies of the batch at kb that went out
    const int blocks_per_page = p.P / 16;
    const int batch = min(32, slots);
    int4 cut = make_int4(0, 0, 0, 0);
    bool ok = true;
    auto publish = [&](const Dq4Item& it, bool last) -> bool {
      const int s = ki % kDq4ItemSlots;
      bool good = true;
      if (ki >= kDq4ItemSlots && lane == 0)
        good = mbar_wait(smem_u32(rempty + s), ((ki / kDq4ItemSlots) - 1) & 1, abort_flag);
      good = __shfl_sync(0xffffffffu, good, 0);
      if (!good) return false;
      if (lane == 0) {
        *item_rec(s) = it;
        const uint32_t fb = smem_u32(rfull + s);
        if (last) {
          mbar_arrive(fb);
        } else {
          const uint32_t bytes = G * D * 2;  // a token's heads are contiguous
          mbar_arrive_expect_tx(fb, it.tn * bytes);
          for (int i = 0; i < it.tn; ++i)
            bulk_load(smem_u32(item_q(s)) + i * bytes, p.q + ((size_t)it.row0 + (size_t)i * p.H_q) * D, bytes, fb);
        }
      }
      ++ki;
      return true;
    };
    while (x < x1 && ok) {
      const Dq4Range r = group_range(p, L, grp);
      Dq4Item it;
      it.row0 = (b * p.QL + grp * p.TG) * p.H_q + hkv * G;
      it.tn = r.tn;
      it.pos0 = r.pos0;
      it.blk0 = r.blk0 + off;
      it.nblk = (int)min((int64_t)(r.nblk - off), x1 - x);
      it.part = -1;
      if (it.nblk < r.nblk) {
        it.part = off > 0 ? 0 : 1;
        if (off == 0) {  // the thread block with an item's first part has the record of its cut
          const int64_t e = x + r.nblk - 1;
          const int last = (int)(((e + 1) * runs - 1) / total);
          cut = make_int4(it.row0, it.tn, last - (int)blockIdx.x + 1, 0);
        }
      }
      if (p.bias_prefetch && lane < it.tn * G) {  // this row's bias for the part's keys
        const int i = lane / G, pr = it.pos0 + i;
        const int far = pr - 16 * it.blk0, near = pr - (16 * (it.blk0 + it.nblk) - 1);
        const int dlo = min(max(near, 0), p.R - 1) & ~3;
        const int dhi = min(min(max(far, 0), p.R - 1) + 4, p.R) & ~3;
        const float* row = p.rel + ((size_t)it.row0 + (size_t)i * p.H_q + (lane - i * G)) * p.R;
        if (dhi > dlo) bulk_prefetch_l2(row + dlo, (uint32_t)(dhi - dlo) * 4);
      }
      ok = publish(it, false);
      if (!ok) break;
      // ---- its blocks: a lane each, a batch of at most 32 (and of the ring's slots: no
      // two lanes share one) at a time.  A lane's copy goes out as soon as its slot is
      // free; page ids are read a batch ahead.
      const int32_t* pt_row = p.page_table + (size_t)b * p.pt_stride;
      auto page_of = [&](int i) -> int {
        return lane < batch && i < it.nblk ? __ldg(pt_row + (it.blk0 + i) / blocks_per_page) : 0;
      };
      int page = page_of(lane);
      for (int i0 = 0; i0 < it.nblk; i0 += batch) {
        const int i = i0 + lane;
        const int next_page = page_of(i + batch);
        bool todo = lane < batch && i < it.nblk;
        const uint32_t all = __ballot_sync(0xffffffffu, todo);
        const uint32_t n = (uint32_t)(kb + lane), turn = n / (uint32_t)slots;
        const uint32_t sl = n - turn * (uint32_t)slots;
        uint8_t* dst = smem + sl * S.slot_bytes;
        const uint32_t fb = smem_u32(full + sl), eb = smem_u32(empty + sl);
        const bool fine = page >= 0 && page < p.num_pages;
        const size_t at =
            (((size_t)page * p.H_kv + hkv) * blocks_per_page + (it.blk0 + i) % blocks_per_page) * BLK;
        unsigned long long t0 = 0;
        for (uint32_t tries = 1;; ++tries) {
          if (todo && (turn == 0 || mbar_try_wait(eb, (turn - 1) & 1))) {
            todo = false;
            if (fine) {
              mbar_arrive_expect_tx(fb, 2 * BLK);
              bulk_load(smem_u32(dst), p.k_cache + at, BLK, fb);
              bulk_load(smem_u32(dst) + BLK, p.v_cache + at, BLK, fb);
            } else {  // reads as zeros: scale 0 (16 * N bf16 of K and of V)
#pragma unroll 1
              for (int w = 0; w < 8 * N; ++w) {
                reinterpret_cast<uint32_t*>(dst + q4_scale_off(D))[w] = 0u;
                reinterpret_cast<uint32_t*>(dst + BLK + q4_scale_off(D))[w] = 0u;
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
              mbar_arrive(fb);
            }
          }
          if (__all_sync(0xffffffffu, !todo)) break;
          __nanosleep(100);  // about the time of two blocks at full bandwidth; the ring holds tens
          if ((tries & 31u) == 0) {  // bounded, as mbar_wait
            if (t0 == 0) t0 = globaltimer();
            if (__any_sync(0xffffffffu, *abort_flag || globaltimer() - t0 > kWaitTimeoutNs)) {
              *abort_flag = 1;
              ok = false;
              break;
            }
          }
        }
        if (!ok) {
          sent = all & ~__ballot_sync(0xffffffffu, todo);
          break;
        }
        kb += min(batch, it.nblk - i0);
        page = next_page;
      }
      if (!ok) break;
      // ---- the next item
      x += it.nblk;
      off = 0;
      if (++grp == p.NG) {
        grp = 0;
        if (++hkv == p.H_kv) {
          hkv = 0;
          do {
            ++b;
          } while (b < p.B && clamped_len(p, b) < p.QL);
          if (b < p.B) L = clamped_len(p, b);
        }
      }
    }
    if (ok) {
      Dq4Item end;
      memset(&end, 0, sizeof(end));
      ok = publish(end, true);  // nblk = 0: no more items
    }
    if (lane == 0) p.cut[blockIdx.x] = cut;
    if (!ok) {  // drain: each slot's last copy in flight, which nobody reads
      for (int j = lane; j < slots; j += 32) {
        int n = kb - kb % slots + j;  // the slot's block in [kb, kb + slots), or before
        if (n < kb) n += slots;
        if (n - kb >= 32 || !((sent >> (n - kb)) & 1u)) n -= slots;
        if (n >= 0) mbar_wait_drain(smem_u32(full + j), (n / slots) & 1);
      }
    }
    if (!ok && lane == 0) {
      report(p.dev_err, INKLING_DEVERR_TIMEOUT);
      for (int j = max(0, ki - kDq4ItemSlots); j < ki; ++j)
        mbar_wait_drain(smem_u32(rfull + j % kDq4ItemSlots), (j / kDq4ItemSlots) & 1);
    }
    return;
  }

  // =================================================================== consumers
  // ---- sequences with nothing to attend to
  for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
    if (clamped_len(p, b) >= p.QL) continue;
    const int rows = p.QL * p.H_q;
    const size_t r0 = (size_t)b * rows;
    for (int i = tid; i < rows * (D / 8); i += 32 * W)
      reinterpret_cast<uint4*>(p.out + r0 * D)[i] = make_uint4(0, 0, 0, 0);
    if (p.lse_out)
      for (int i = tid; i < rows; i += 32 * W) p.lse_out[r0 + i] = -INFINITY;
  }

  const int g = lane >> 2, t = lane & 3;
  // Key of a block that MMA row g (and g + 8: 8 more) stands for: rows 2t, 2t + 1
  // are keys t, 4 + (t ^ 1), so that the 64-byte rows read together lie in both halves
  // of the shared-memory banks, for K (rows 2t, 2t + 1 at once) and V (t = 0..3 at once).
  const int key_g = (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1;
  const int key_t0 = t, key_t1 = 4 + (t ^ 1);

  int kb_w = 0;         // blocks of the items before this one, modulo W
  int s_slot = warp;    // this warp's next slot (it owns warp, warp + W, ...) and its phase
  uint32_t s_phase = 0;
  bool ok = true;
  for (int ki = 0;; ++ki) {
    const int is = ki % kDq4ItemSlots;
    if (!mbar_wait_warp(smem_u32(rfull + is), (ki / kDq4ItemSlots) & 1, abort_flag)) {
      ok = false;
      break;
    }
    const Dq4Item it = *item_rec(is);
    if (it.nblk == 0) break;
    const int rows = it.tn * G;
    // ---- q fragments (channel order of the K rows), and -136 sum(q) of every group
    // as an operand of one more product, with the block's scales: sum_j s_j (-136 sum_j(q))
    uint32_t qf[N][2][NT][2];
    uint32_t qs[NT][2];  // B fragment of -136 sum(q): k = N * part + group, three bf16 parts
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = nt * 8 + g;
      const uint8_t* qr = item_q(is) + r * D * 2;
      float sum[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        uint4 w = make_uint4(0, 0, 0, 0);  // channels 32j + 8t + 0..7
        if (r < rows) w = *reinterpret_cast<const uint4*>(qr + 64 * j + 16 * t);
        qf[j][0][nt][0] = __byte_perm(w.x, w.z, 0x5410);  // c, c + 4 for c = 0..3
        qf[j][0][nt][1] = __byte_perm(w.x, w.z, 0x7632);
        qf[j][1][nt][0] = __byte_perm(w.y, w.w, 0x5410);
        qf[j][1][nt][1] = __byte_perm(w.y, w.w, 0x7632);
        float c[4];
        mma_16816_new(c, kMinus136, kMinus136, kMinus136, kMinus136, qf[j][0][nt][0], qf[j][0][nt][1]);
        mma_16816(c, kMinus136, kMinus136, kMinus136, kMinus136, qf[j][1][nt][0], qf[j][1][nt][1]);
        // every row of c is the same; this lane takes column g
        const float even = __shfl_sync(0xffffffffu, c[0], g >> 1), odd = __shfl_sync(0xffffffffu, c[1], g >> 1);
        sum[j] = (g & 1) ? odd : even;
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
      qs[nt][0] = p0 < 3 ? pack_bf16(part(lo_, p0), part(hi_, p0)) : 0u;
      qs[nt][1] = N == 4 && t < 2 ? pack_bf16(part(lo_, 2), part(hi_, 2)) : 0u;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(rempty + is));

    // Bias of this lane's score columns: bias_at[nt][x] points at the distance of
    // key 0 of its MMA row g (keys further along lie below it).
    const int pos0 = it.pos0, pos1 = it.pos0 + it.tn - 1;
    const float* bias_at[NT][2];
    auto row_tok = [&](int nt, int x) { return min(nt * 8 + 2 * t + x, rows - 1) / G; };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = min(nt * 8 + 2 * t + x, rows - 1), i = r / G;
        bias_at[nt][x] = p.rel + ((size_t)it.row0 + (size_t)i * p.H_q + (r - i * G)) * p.R + (pos0 + i - key_g);
      }
    float far[NT][2];  // bias at and past the table's end
    const bool has_far = pos1 - it.blk0 * 16 >= p.R;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x)
        far[nt][x] = has_far ? __ldg(bias_at[nt][x] - (pos0 + row_tok(nt, x) - key_g) + p.R - 1) : 0.f;
    auto load_bias = [&](int key0, float (&bv)[NT][4]) {
      if (pos0 - (key0 + 15) >= p.R - 1) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) bv[nt][x] = far[nt][x & 1];
      } else if (key0 + 15 <= pos0 && pos1 - key0 < p.R) {  // every distance is inside the table
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) bv[nt][x] = __ldg(bias_at[nt][x & 1] - key0 - 8 * (x >> 1));
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int dist = pos0 + row_tok(nt, x & 1) - key_g - key0 - 8 * (x >> 1);
            const int at = min(max(dist, 0), p.R - 1) - dist;
            bv[nt][x] = __ldg(bias_at[nt][x & 1] - key0 - 8 * (x >> 1) + at);
          }
      }
    };

    float m_run[NT][2], l_run[NT][2], o[N][2][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[j][i][nt][x] = 0.f;
    }

    // One block; kInside: every row sees all of its 16 keys.
    auto block = [&](auto inside_c, int key0, const uint8_t* kp, uint32_t eb, const float (&bv)[NT][4]) {
      constexpr bool kInside = decltype(inside_c)::value;
      const uint8_t* vp = kp + BLK;
      uint32_t kw[2][N], vw[4][N / 2], ksc[2][N / 2], vsc[2][N / 2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint8_t* kr = kp + (key_g + 8 * x) * (D / 2) + 4 * N * t;
        const uint8_t* vr = vp + (key_t0 + 8 * x) * (D / 2) + 2 * N * g;
        const uint8_t* vr1 = vp + (key_t1 + 8 * x) * (D / 2) + 2 * N * g;
        const uint8_t* kc = kp + q4_scale_off(D) + (key_g + 8 * x) * (2 * N);
        const uint8_t* vc = vp + q4_scale_off(D) + (key_g + 8 * x) * (2 * N);
        if constexpr (N == 4) {
          const uint4 a = *reinterpret_cast<const uint4*>(kr);
          kw[x][0] = a.x;
          kw[x][1] = a.y;
          kw[x][2] = a.z;
          kw[x][3] = a.w;
          const uint2 v0 = *reinterpret_cast<const uint2*>(vr), v1 = *reinterpret_cast<const uint2*>(vr1);
          vw[2 * x][0] = v0.x;
          vw[2 * x][1] = v0.y;
          vw[2 * x + 1][0] = v1.x;
          vw[2 * x + 1][1] = v1.y;
          const uint2 s0 = *reinterpret_cast<const uint2*>(kc), s1 = *reinterpret_cast<const uint2*>(vc);
          ksc[x][0] = s0.x;
          ksc[x][1] = s0.y;
          vsc[x][0] = s1.x;
          vsc[x][1] = s1.y;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(kr);
          kw[x][0] = a.x;
          kw[x][1] = a.y;
          vw[2 * x][0] = *reinterpret_cast<const uint32_t*>(vr);
          vw[2 * x + 1][0] = *reinterpret_cast<const uint32_t*>(vr1);
          ksc[x][0] = *reinterpret_cast<const uint32_t*>(kc);
          vsc[x][0] = *reinterpret_cast<const uint32_t*>(vc);
        }
      }
      auto scale_of = [&](const uint32_t (&sc)[2][N / 2], int x, int j) {
        return __uint_as_float((j & 1) ? sc[x][j >> 1] & 0xffff0000u : sc[x][j >> 1] << 16);
      };

      // ---- scores of 16 keys x rows, from sum_j s_j (-136 sum_j(q)) on
      float sc[NT][4];
      {
        const int w = N == 4 ? t & 1 : 0;  // scales of groups 2w, 2w + 1 against k = 2t, 2t + 1 (and + 8)
        const uint32_t a0 = w ? ksc[0][N / 2 - 1] : ksc[0][0], a1 = w ? ksc[1][N / 2 - 1] : ksc[1][0];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816_new(sc[nt], a0, a1, a0, a1, qs[nt][0], qs[nt][1]);
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t a0 = q4_expand<0>(kw[0][j]), a1 = q4_expand<0>(kw[1][j]), a2 = q4_expand<1>(kw[0][j]),
                       a3 = q4_expand<1>(kw[1][j]);
        const uint32_t b0 = q4_expand<2>(kw[0][j]), b1 = q4_expand<2>(kw[1][j]), b2 = q4_expand<3>(kw[0][j]),
                       b3 = q4_expand<3>(kw[1][j]);
        const float s0 = scale_of(ksc, 0, j), s8 = scale_of(ksc, 1, j);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float c[4];
          mma_16816_new(c, a0, a1, a2, a3, qf[j][0][nt][0], qf[j][0][nt][1]);
          mma_16816(c, b0, b1, b2, b3, qf[j][1][nt][0], qf[j][1][nt][1]);
          sc[nt][0] = fmaf(c[0], s0, sc[nt][0]);
          sc[nt][1] = fmaf(c[1], s0, sc[nt][1]);
          sc[nt][2] = fmaf(c[2], s8, sc[nt][2]);
          sc[nt][3] = fmaf(c[3], s8, sc[nt][3]);
        }
      }
      bool see[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          sc[nt][x] = fmaf(sc[nt][x], p.scale, bv[nt][x]);
          if constexpr (!kInside) {
            const int dist = pos0 + row_tok(nt, x & 1) - (key0 + key_g + 8 * (x >> 1));
            see[nt][x] = dist >= 0 && (p.window <= 0 || dist < p.window);
            sc[nt][x] = see[nt][x] ? sc[nt][x] : -INFINITY;
          }
        }
      // ---- running maximum and sum.  The maximum, the exponents' base, is
      // taken anew over the warp only when a score passes it by kDq4Slack;
      // until then a weight is at most e^kDq4Slack and nothing is rescaled.
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mx[2] = {fmaxf(sc[nt][0], sc[nt][2]), fmaxf(sc[nt][1], sc[nt][3])};
        if (__any_sync(0xffffffffu, mx[0] > m_run[nt][0] + kDq4Slack || mx[1] > m_run[nt][1] + kDq4Slack)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1)
              mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], off));
            const float mn = fmaxf(m_run[nt][x], mx[x]);
            const float al = mn == -INFINITY ? 1.f : ex2((m_run[nt][x] - mn) * kLog2e);
            l_run[nt][x] *= al;
            m_run[nt][x] = mn;
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                o[j][h][nt][x] *= al;
                o[j][h][nt][x + 2] *= al;
              }
          }
        }
      }
      uint32_t pb[N][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float pr[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // the difference first: s * log2 e alone would lose it under a bias like -1e30
          const float base = m_run[nt][x & 1] == -INFINITY ? 0.f : m_run[nt][x & 1];
          pr[x] = ex2((sc[nt][x] - base) * kLog2e);
        }
        l_run[nt][0] += pr[0] + pr[2];
        l_run[nt][1] += pr[1] + pr[3];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            w[x] = pr[x] * scale_of(vsc, x >> 1, j);
            if constexpr (!kInside) w[x] = see[nt][x] ? w[x] : 0.f;  // a hidden place's scale may be NaN
          }
          pb[j][nt][0] = movmatrix_t(pack_bf16(w[0], w[1]));
          pb[j][nt][1] = movmatrix_t(pack_bf16(w[2], w[3]));
        }
      }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t sel = (j & 1) ? 0x7632 : 0x5410;
        const uint32_t w0 = __byte_perm(vw[0][j >> 1], vw[1][j >> 1], sel);
        const uint32_t w8 = __byte_perm(vw[2][j >> 1], vw[3][j >> 1], sel);
        const uint32_t a0 = q4_expand<0>(w0), a1 = q4_expand<1>(w0), a2 = q4_expand<0>(w8), a3 = q4_expand<1>(w8);
        const uint32_t b0 = q4_expand<2>(w0), b1 = q4_expand<3>(w0), b2 = q4_expand<2>(w8), b3 = q4_expand<3>(w8);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(o[j][0][nt], kMinus136, kMinus136, kMinus136, kMinus136, pb[j][nt][0], pb[j][nt][1]);
          mma_16816(o[j][1][nt], kMinus136, kMinus136, kMinus136, kMinus136, pb[j][nt][0], pb[j][nt][1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(o[j][0][nt], a0, a1, a2, a3, pb[j][nt][0], pb[j][nt][1]);
          mma_16816(o[j][1][nt], b0, b1, b2, b3, pb[j][nt][0], pb[j][nt][1]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(eb);
    };

    // ---- this warp's blocks of the item, their bias loaded one block ahead
    int i = warp - kb_w;
    if (i < 0) i += W;
    kb_w = (kb_w + it.nblk) % W;
    float bv[NT][4];
    if (i < it.nblk) load_bias((it.blk0 + i) * 16, bv);
    for (; i < it.nblk; i += W) {
      const int key0 = (it.blk0 + i) * 16;
      float bn[NT][4];
      if (i + W < it.nblk) load_bias(key0 + 16 * W, bn);
      if (!mbar_wait_warp(smem_u32(full + s_slot), s_phase, abort_flag)) {
        ok = false;
        break;
      }
      const uint8_t* kp = smem + s_slot * S.slot_bytes;
      const uint32_t eb = smem_u32(empty + s_slot);
      if (key0 + 15 <= pos0 && (p.window <= 0 || pos1 - key0 < p.window)) block(std::true_type{}, key0, kp, eb, bv);
      else block(std::false_type{}, key0, kp, eb, bv);
      s_slot += W;
      if (s_slot >= slots) {
        s_slot = warp;
        s_phase ^= 1;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) bv[nt][x] = bn[nt][x];
    }
    if (!ok) break;

    // ---- the warps' parts, joined through shared memory
    named_bar_sync(1, 32 * W);  // the previous item's readers are done
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float l = l_run[nt][x];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        const int r = nt * 8 + 2 * t + x;
        if (g == 0) {
          comb_m[warp * HP + r] = m_run[nt][x];
          comb_l[warp * HP + r] = l;
        }
        if (r < rows) {
#pragma unroll
          for (int j = 0; j < N; ++j)  // channels 32j + 4g + 0..3
            *reinterpret_cast<float4*>(comb + (warp * NR + r) * OP + 32 * j + 4 * g) =
                make_float4(o[j][0][nt][x], o[j][0][nt][x + 2], o[j][1][nt][x], o[j][1][nt][x + 2]);
        }
      }
    named_bar_sync(1, 32 * W);
    for (int u = tid; u < rows * (D / 4); u += 32 * W) {
      const int r = u / (D / 4), d = 4 * (u - r * (D / 4));
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < W; ++w) M = fmaxf(M, comb_m[w * HP + r]);
      const float base = M == -INFINITY ? 0.f : M;
      float l = 0.f;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = ex2((comb_m[w * HP + r] - base) * kLog2e);
        const float4 v = *reinterpret_cast<const float4*>(comb + (w * NR + r) * OP + d);
        l = fmaf(f, comb_l[w * HP + r], l);
        a.x = fmaf(f, v.x, a.x);
        a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z);
        a.w = fmaf(f, v.w, a.w);
      }
      if (it.part < 0) {
        const int i = r / G;
        const size_t row = (size_t)it.row0 + (size_t)i * p.H_q + (r - i * G);
        const float inv = l == 0.f ? 0.f : 1.f / l;  // every score -inf: an empty row
        *reinterpret_cast<uint2*>(p.out + row * D + d) =
            make_uint2(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv));
        if (d == 0 && p.lse_out) p.lse_out[row] = M + logf(l);
      } else {
        const size_t row = ((size_t)blockIdx.x * 2 + it.part) * NR + r;
        *reinterpret_cast<float4*>(p.part_o + row * D + d) = a;
        if (d == 0) p.part_ml[row] = make_float2(M, l);
      }
    }
  }
  if (!ok && lane == 0) report(p.dev_err, INKLING_DEVERR_TIMEOUT);
}

// ---------------------------------------------------------------------------
// Joins the parts of cut items: block (c, r) has row r of the item that thread
// block c's run cuts first.  Its parts are c's second and the first of c + 1 .. ;
// 8 warps take them in turn, D / 32 channels per lane.
template <int D>
__global__ void __launch_bounds__(256) merge_q4_kernel(const __grid_constant__ DecodeQ4Params p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int C = D / 32;
  const int4 cut = p.cut[blockIdx.x];
  const int r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (cut.z == 0 || r >= cut.y * p.G) return;
  __shared__ float s_o[8][D];
  __shared__ float2 s_ml[8];
  auto part_row = [&](int k) {
    return ((size_t)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * p.NR + r;
  };
  float M = -INFINITY, l = 0.f, acc[C];
#pragma unroll
  for (int c = 0; c < C; ++c) acc[c] = 0.f;
#pragma unroll 4
  for (int k = warp; k < cut.z; k += 8) {
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
  for (int w = 0; w < 8; ++w) M = fmaxf(M, s_ml[w].x);
  const float base = M == -INFINITY ? 0.f : M;
  float o = 0.f;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const float f = ex2((s_ml[w].x - base) * kLog2e);
    l = fmaf(s_ml[w].y, f, l);
    o = fmaf(s_o[w][d], f, o);
  }
  const int i = r / p.G;
  const size_t row = (size_t)cut.x + (size_t)i * p.H_q + (r - i * p.G);
  p.out[row * D + d] = __float2bfloat16(l == 0.f ? 0.f : o / l);
  if (d == 0 && p.lse_out) p.lse_out[row] = M + logf(l);
}

// ---------------------------------------------------------------------------
// Host side

struct Dq4Plan {
  int G, TG, NG, NR, NT, grid;
  size_t ml, cut, total;  // workspace offsets: parts first
  Dq4Plan(int32_t QL, int32_t H_q, int32_t H_kv, int32_t D, int32_t sms) {
    G = H_q / H_kv;
    TG = decode_token_group(QL, G);
    NG = (QL + TG - 1) / TG;
    NR = TG * G;
    NT = NR <= 8 ? 1 : 2;
    grid = sms * (NT == 1 ? Dq4Shape<1>::kCtas : Dq4Shape<2>::kCtas);
    ml = align256((size_t)grid * 2 * NR * D * sizeof(float));
    cut = ml + align256((size_t)grid * 2 * NR * sizeof(float2));
    total = cut + align256((size_t)grid * sizeof(int4));
  }
};

size_t decode_q4_workspace_bytes(int32_t, int32_t QL, int32_t H_q, int32_t H_kv, int32_t D, int32_t sms) {
  return Dq4Plan(QL, H_q, H_kv, D, sms).total;
}

template <typename K>
static bool launch_dependent(K kern, dim3 grid, int threads, int smem, const DecodeQ4Params& prm,
                             cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, prm) == cudaSuccess && cudaGetLastError() == cudaSuccess;
}

template <int D, int NT>
static int launch_decode_q4_t(const DecodeQ4Call& c, DecodeQ4Params prm, const Dq4Plan& plan) {
  using Sh = Dq4Shape<NT>;
  const int budget = kDq4SmemPerSm / Sh::kCtas - 1024;
  // a multiple of W: a slot always belongs to the same warp, which so waits for every phase of its barrier
  int slots = 9 * Sh::W;
  while (slots > Sh::W && Dq4Smem(D, NT, plan.NR, Sh::W, slots).total > budget) slots -= Sh::W;
  prm.slots = slots;
  const int smem = Dq4Smem(D, NT, plan.NR, Sh::W, slots).total;
  auto kern = decode_q4_kernel<D, NT>;
  static std::atomic<int> limit_set[kMaxDevices];
  if (!smem_limit_on_device(reinterpret_cast<const void*>(kern), budget, limit_set)) return INKLING_ERR_CUDA;
  if (!launch_dependent(kern, dim3(plan.grid), Sh::kThreads, smem, prm, c.stream)) return INKLING_ERR_CUDA;
  if (!launch_dependent(merge_q4_kernel<D>, dim3(plan.grid, plan.NR), 256, 0, prm, c.stream))
    return INKLING_ERR_CUDA;
  return INKLING_OK;
}

int launch_decode_q4(const DecodeQ4Call& c) {
  const Dq4Plan plan(c.QL, c.H_q, c.H_kv, c.D, c.sms);
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
  p.NG = plan.NG;
  p.NR = plan.NR;
  p.bias_prefetch = c.R % 4 == 0 && (reinterpret_cast<uintptr_t>(c.rel) & 15) == 0;
  p.scale = c.scale;
  if (c.D == 128) return plan.NT == 1 ? launch_decode_q4_t<128, 1>(c, p, plan) : launch_decode_q4_t<128, 2>(c, p, plan);
  return plan.NT == 1 ? launch_decode_q4_t<64, 1>(c, p, plan) : launch_decode_q4_t<64, 2>(c, p, plan);
}

}  // namespace ira

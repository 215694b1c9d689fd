// Decode attention with the relative-position bias over the 8-bit cache: the format's
// part of decode_blocks.cuh, which has the division of the work.
//
// Operation: inkling_rel_attn_decode_q8 in include/inkling_rel_attn.h.
//
// Per block a warp forms S^T = K Q^T (16 keys x rows) and O^T += V^T P^T with
// mma.sync on fp16 operands:
//  * an e4m3 number is an fp16 one, so K and V become operands by one conversion for
//    two values, exactly;
//  * q (bf16) becomes fp16 times a power of two of its row, 2^-eq, with which its largest
//    magnitude lies in [2^14, 2^15): what is lost lies below 2^-39 of that (fp16's
//    subnormals).  2^eq, the scale and the block's 2^e come back as one factor in fp32;
//  * a block's scale of V is a factor of P, taken relative to the largest one so far
//    (the O it belongs to is rescaled when that grows, as with the running maximum), so
//    P is an fp16 number of at most e^5.5 2^7, with 2^-11 of a weight as its rounding and
//    2^-32 of the largest weight times the largest scale below its range.
// Hidden keys get the bias -inf, so P = 0, and their rows of K and V are zeroed in shared
// memory: a page's unused places may hold anything.
// A row with a NaN is stored as zeros and a mark.  A row of q that sees it, by position and
// window, gets NaN, as its sum for K and as a weight for V, whatever bias or weight the key
// has: that must not depend on the order in which keys are taken.
#include <cuda_fp16.h>

#include "decode_blocks.cuh"
#include "launch.h"
#include "q8.cuh"

namespace ira {

constexpr int kPDown = 7;             // P carries 2^7, to use more of fp16's range
constexpr float kMostFactor = 0x1p96f;  // of a score: times the products (below 2^31) it stays finite

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

struct Q8Format {
  static constexpr bool kJoiner = true;
  static constexpr int kGroup = 1;  // a ring of 8 tiles (32 sequences to 32768 keys: 190.2 us; in fours 193.8)
  __host__ __device__ static constexpr int block_bytes(int D) { return q8_block_bytes(D); }
  __device__ static int key_of(int g) { return g; }

  template <int D>
  __device__ static __forceinline__ void empty_tail(uint8_t* blk) {  // the smallest scale, no NaN row
    *reinterpret_cast<uint2*>(blk + q8_tail_off(D)) = make_uint2(q8_scale_bits(kQ8MinExp), 0u);
  }
  template <int D>
  __device__ static __forceinline__ void zero_block(uint8_t* k, uint8_t* v) {
#pragma unroll 1
    for (int i = 0; i < D; ++i) {
      reinterpret_cast<uint4*>(k)[i] = make_uint4(0, 0, 0, 0);
      reinterpret_cast<uint4*>(v)[i] = make_uint4(0, 0, 0, 0);
    }
    empty_tail<D>(k);
    empty_tail<D>(v);
  }

  // q as fp16 times 2^-eq, and |scale| 2^eq of the rows 2t, 2t + 1 (a negative scale turns q round).
  template <int D>
  __device__ static __forceinline__ void prepare(const DecodeBlocksParams& p, const uint4* row, bool have, uint4* frag,
                                                 RunPrep& pr) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31, t = lane & 3;
    uint4 w[N];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      // unit c = 4x + t of 16 channels (x = j / 2), its first or second half
      w[j] = row[2 * (4 * (j >> 1) + t) + (j & 1)];
      if (!have) w[j] = make_uint4(0, 0, 0, 0);
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(w[j].x & 0x7fff7fffu, w[j].y & 0x7fff7fffu),
                               __vmaxu2(w[j].z & 0x7fff7fffu, w[j].w & 0x7fff7fffu)));
    }
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // (a row below 2^-60 keeps fewer bits; one with an infinity or a NaN has scores that are none)
    const int eq = max((int)(max(m & 0xffffu, m >> 16) >> 7) - 127 - 14, -74);
    const float f = copysignf(__uint_as_float((uint32_t)(127 - eq) << 23), p.scale);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint4 v = w[j];
      auto half2 = [&](uint32_t x) {
        return pack_f16(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xffff0000u) * f);
      };
      frag[32 * j] = make_uint4(half2(v.x), half2(v.y), half2(v.z), half2(v.w));
    }
    const float back = fabsf(p.scale) * __uint_as_float((uint32_t)(127 + eq) << 23);
    pr.extra[0] = __float_as_uint(__shfl_sync(0xffffffffu, back, 4 * (2 * t)));
    pr.extra[1] = __float_as_uint(__shfl_sync(0xffffffffu, back, 4 * (2 * t + 1)));
    pr.extra[2] = pr.extra[3] = 0u;
  }

  template <int D, bool MULTI>
  struct Consumer {
    static constexpr int U = kRunU, N = D / 16, BLK = q8_block_bytes(D), TAIL = q8_tail_off(D);
    int g, t, lane;
    int row_k, row_v[4];  // this lane's part of K row g, of V rows 2t, 2t + 1, 2t + 8, 2t + 9
    uint4 qf[D / 32];
    float back[2];       // |scale| 2^eq of the rows 2t, 2t + 1
    float o[N][4];       // channel D / 8 g + 2j (x = 0, 1) and the next (x = 2, 3) of rows 2t, 2t + 1, over 2^(ev - 7)
    int ev;              // largest exponent of V so far
    float kf[U][2];      // factor of a block's products
    uint32_t marks;      // not 0: the tile has rows with a NaN
    uint32_t vs[U];      // scales of the tile's V blocks

    __device__ __forceinline__ Consumer(int g_, int t_, int lane_) : g(g_), t(t_), lane(lane_) {
      row_k = q8_unit_at<D, false>(g, 2 * t);
#pragma unroll
      for (int x = 0; x < 4; ++x) row_v[x] = q8_unit_at<D, true>(2 * t + (x & 1) + 8 * (x >> 1), D == 128 ? 2 * g : g);
    }
    __device__ __forceinline__ void load_q(const uint4* frag) {
#pragma unroll
      for (int j = 0; j < D / 32; ++j) qf[j] = frag[32 * j];
    }
    __device__ __forceinline__ void begin(const RunPrep& pr) {
      back[0] = __uint_as_float(pr.extra[0]);
      back[1] = __uint_as_float(pr.extra[1]);
      ev = kQ8MinExp;
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[j][x] = 0.f;
    }
    __device__ __forceinline__ void settle() {}
    // Rows of keys before ``first`` and after ``last`` are zeroed, in K and V; a block without
    // another key gets a tail that is one.
    __device__ __forceinline__ void hide(uint8_t* slot, int key0, int first, int last) const {
      constexpr int L = D / 16;  // lanes per row
#pragma unroll 1
      for (int r = lane / L; r < kRunTile; r += 32 / L) {
        const int key = key0 + r;
        if (key <= last && key >= first) continue;
        // (the rows' units are exchanged within rows of 128 channels, and within pairs of rows of 64)
        uint8_t* k = slot + (r >> 4) * BLK;
        const int a = q8_unit_at<D, false>(r & 15, 2 * (lane % L));
        *reinterpret_cast<uint4*>(k + a) = make_uint4(0, 0, 0, 0);
        uint8_t* v = k + U * BLK;
        *reinterpret_cast<uint2*>(v + q8_unit_at<D, true>(r & 15, 2 * (lane % L))) = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(v + q8_unit_at<D, true>(r & 15, 2 * (lane % L) + 1)) = make_uint2(0, 0);
      }
      if (lane < U) {
        const int a = key0 + 16 * lane;
        if (a > last || a + 15 < first) {
          empty_tail<D>(slot + lane * BLK);
          empty_tail<D>(slot + (U + lane) * BLK);
        }
      }
    }
    __device__ __forceinline__ void scores(const DecodeBlocksParams&, const uint8_t* slot, float (&sc)[U][4]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint8_t* kp = slot + u * BLK;
        const uint2 tail = *reinterpret_cast<const uint2*>(kp + TAIL);
        const float s = __uint_as_float(tail.x);
        kf[u][0] = fminf(back[0] * s, kMostFactor);
        kf[u][1] = fminf(back[1] * s, kMostFactor);
        marks = u == 0 ? tail.y : marks | tail.y;
        float odd[4];  // two chains of products (one: 32 sequences to 32768 keys 190.0 us instead of 187.6)
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[u][x] = odd[x] = 0.f;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          // unit 4x + t of row g; in odd rows of 128 channels the halves x are exchanged
          const int at = D == 128 ? row_k ^ (64 * x) : row_k;
          const uint4 lo = *reinterpret_cast<const uint4*>(kp + at);
          const uint4 hi = *reinterpret_cast<const uint4*>(kp + at + 8 * D);
          const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16(wl[i], a0, a2);
            e4m3x4_to_f16(wh[i], a1, a3);
            const uint4 q = qf[2 * x + (i >> 1)];
            if (i & 1) mma_f16(odd, a0, a1, a2, a3, q.z, q.w);
            else mma_f16(sc[u], a0, a1, a2, a3, q.x, q.y);
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) sc[u][x] += odd[x];
      }
    }
    __device__ __forceinline__ float score(const DecodeBlocksParams&, int u, int x, float raw, float bias, bool) const {
      return fmaf(raw, kf[u][x & 1], bias);
    }
    // (The tails are read again: with their marks kept, 64 sequences of 4 drafts take 0.1 us more; with a branch for K
    // before the maximum and one for V after it 2; in all it is 0.7 us on 57.2, and nothing on one token.)
    template <class Sees>
    __device__ __forceinline__ void mark(const uint8_t* slot, float (&sc)[U][4], float (&sum)[2], const Sees& sees) const {
      if (marks == 0u) return;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t k = *reinterpret_cast<const uint32_t*>(slot + u * BLK + TAIL + 4);
        const uint32_t v = *reinterpret_cast<const uint32_t*>(slot + (U + u) * BLK + TAIL + 4);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (!sees(u, x)) continue;
          const int r = g + 8 * (x >> 1);
          if ((k >> r) & 1u) sum[x & 1] = __int_as_float(0x7fffffff);
          if ((v >> r) & 1u) sc[u][x] = __int_as_float(0x7fffffff);
        }
      }
    }
    __device__ __forceinline__ static int exp_of(uint32_t scale) { return (int)(scale >> 23) - 127; }
    __device__ __forceinline__ bool v_scales(const uint8_t* slot) {
      bool up = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint2 tail = *reinterpret_cast<const uint2*>(slot + (U + u) * BLK + TAIL);
        vs[u] = tail.x;
        marks |= tail.y;
        up = up || exp_of(vs[u]) > ev;
      }
      return up;
    }
    __device__ __forceinline__ float v_rebase() {
      const int was = ev;
#pragma unroll
      for (int u = 0; u < U; ++u) ev = max(ev, exp_of(vs[u]));
      return __uint_as_float((uint32_t)max(127 + was - ev, 0) << 23);
    }
    __device__ __forceinline__ void rescale(int x, float al) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        o[j][x] *= al;
        o[j][x + 2] *= al;
      }
    }
    __device__ __forceinline__ void values(const uint8_t* slot, uint32_t slot_bar, const float (&sc)[U][4], uint32_t) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint8_t* vp = slot + (U + u) * BLK;
        uint32_t vw[4][D / 32];  // channels D / 8 g + 4i .. + 3 of the four rows
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(vp + row_v[x]);
            vw[x][0] = v.x;
            vw[x][1] = v.y;
            vw[x][D / 32 - 2] = v.z;
            vw[x][D / 32 - 1] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(vp + row_v[x]);
            vw[x][0] = v.x;
            vw[x][1] = v.y;
          }
        }
        if (u == U - 1) {
          __syncwarp();
          if (lane == 0) mbar_arrive(slot_bar);  // the tile is in registers
        }
        const float f = __uint_as_float((uint32_t)max(127 + kPDown + exp_of(vs[u]) - ev, 0) << 23);
        const float w[4] = {sc[u][0] * f, sc[u][1] * f, sc[u][2] * f, sc[u][3] * f};
        uint32_t pb[2];
        pb[0] = movmatrix_t(pack_f16(w[0], w[1]));
        pb[1] = movmatrix_t(pack_f16(w[2], w[3]));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // channels 4i + 2h and + 1: MMA rows g and g + 8
            const uint32_t sel = h ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16(__byte_perm(vw[0][i], vw[1][i], sel), a0, a1);
            e4m3x4_to_f16(__byte_perm(vw[2][i], vw[3][i], sel), a2, a3);
            mma_f16(o[2 * i + h], a0, a1, a2, a3, pb[0], pb[1]);
          }
        }
      }
    }
    __device__ __forceinline__ void store(int x, float* row) const {
      const float f = __uint_as_float((uint32_t)(127 + ev - kPDown) << 23);
#pragma unroll
      for (int j = 0; j < N; j += 2)
        *reinterpret_cast<float4*>(row + (D / 8) * g + 2 * j) =
            make_float4(o[j][x] * f, o[j][x + 2] * f, o[j + 1][x] * f, o[j + 1][x + 2] * f);
    }
  };
};

struct Q8Launch {
  template <int D, bool MULTI>
  static bool launch(const DecodeBlocksCall& c, const DecodeBlocksParams& p, const RunPlan& plan, int smem) {
    auto kern = decode_blocks_kernel<Q8Format, D, MULTI>;
    static std::atomic<int> limit_set[kMaxDevices];
    return smem_limit_on_device(reinterpret_cast<const void*>(kern), kRunSmemBudget, limit_set) &&
           launch_dependent(kern, dim3(plan.grid), run_threads<Q8Format, MULTI>(), smem, p, c.stream) &&
           launch_dependent(merge_blocks_kernel<D>, dim3(plan.grid, plan.NR), 32 * kRunMergeWarps, 0, p, c.stream);
  }
};

int launch_decode_q8(const DecodeBlocksCall& c) { return launch_blocks<Q8Format, Q8Launch>(c, c.scale); }

}  // namespace ira

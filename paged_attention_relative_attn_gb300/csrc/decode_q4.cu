// Decode attention with the relative-position bias over the 4-bit cache: the format's
// part of decode_blocks.cuh, which has the division of the work.
//
// Operation: inkling_rel_attn_decode_q4 in include/inkling_rel_attn.h.
//
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
#include "decode_blocks.cuh"
#include "launch.h"
#include "q4.cuh"

namespace ira {

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

struct Q4Format {
  static constexpr bool kJoiner = false;
  static constexpr int kGroup = 4;
  __host__ __device__ static constexpr int block_bytes(int D) { return q4_block_bytes(D); }
  // Rows 2t, 2t + 1 are keys t, 4 + (t ^ 1), so that the 64-byte rows read together lie in both halves
  // of the shared-memory banks, for K (rows 2t, 2t + 1 at once) and V (t = 0..3 at once).
  __device__ static int key_of(int g) { return (g & 1) ? 4 + ((g >> 1) ^ 1) : g >> 1; }

  template <int D>
  __device__ static __forceinline__ void zero_block(uint8_t* k, uint8_t* v) {  // scale 0 (16 * N bf16 of K and of V)
#pragma unroll 1
    for (int w = 0; w < 8 * (D / kQ4Group); ++w) {
      reinterpret_cast<uint32_t*>(k + q4_scale_off(D))[w] = 0u;
      reinterpret_cast<uint32_t*>(v + q4_scale_off(D))[w] = 0u;
    }
  }

  // q in the channel order of the K rows, and -8 sum(q) of every group as an operand of
  // one more product, with the block's scales: sum_j s_j (-8 sum_j(q)).
  template <int D>
  __device__ static __forceinline__ void prepare(const DecodeBlocksParams&, const uint4* row, bool have, uint4* frag,
                                                 RunPrep& pr) {
    constexpr int N = D / kQ4Group;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float sum[N];
    uint4 qw[N];
#pragma unroll
    for (int j = 0; j < N; ++j) qw[j] = row[t + 4 * j];  // channels 32j + 8t + 0..7
#pragma unroll
    for (int j = 0; j < N; ++j) {
      uint4 w = qw[j];
      if (!have) w = make_uint4(0, 0, 0, 0);
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
    // k = 2t, 2t + 1 and 2t + 8, 2t + 9 of column g: k = N * part + group, three bf16 parts
    auto part = [&](float v, int i) {  // part i of v's three bf16 parts
      float h = __bfloat162float(__float2bfloat16(v));
      if (i == 0) return h;
      v -= h;
      h = __bfloat162float(__float2bfloat16(v));
      return i == 1 ? h : v - h;
    };
    const float lo_ = N == 2 || !(t & 1) ? sum[0] : sum[N - 2], hi_ = N == 2 || !(t & 1) ? sum[1] : sum[N - 1];
    const int p0 = N == 2 ? t : t >> 1;  // of k = 2t; k = 2t + 8 is two further on
    pr.extra[2] = pr.extra[3] = 0u;
    pr.extra[0] = p0 < 3 ? pack_bf16(part(lo_, p0), part(hi_, p0)) : 0u;
    pr.extra[1] = N == 4 && t < 2 ? pack_bf16(part(lo_, 2), part(hi_, 2)) : 0u;
  }

  template <int D, bool MULTI>
  struct Consumer {
    static constexpr int U = kRunU, N = D / kQ4Group, BLK = q4_block_bytes(D);
    int t, lane;
    // Constant operands of V's offset: rows g (m8[0]) or rows g + 8 (m8[1]) of the
    // product take -8 sum(P) of a group; kept in registers.
    uint32_t m8[2][4];
    int row_k, row_v0, row_v1, row_s;  // this lane's part of a K row, of V rows, of the scales
    uint4 qf[N];
    uint32_t qs[2];
    // O and, for groups 2i (x = 0, 1) and 2i + 1 (x = 2, 3), -8 sum(P s): O holds u, not
    // u - 8, until the two are put together
    float o[N][2][4], co[N / 2][4];

    __device__ __forceinline__ Consumer(int g, int t_, int lane_) : t(t_), lane(lane_) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        asm volatile("mov.b32 %0, %1;" : "=r"(m8[0][i]) : "r"((i & 1) ? 0u : kMinus8));
        asm volatile("mov.b32 %0, %1;" : "=r"(m8[1][i]) : "r"((i & 1) ? kMinus8 : 0u));
      }
      const int key_g = key_of(g);
      row_k = key_g * (D / 2) + 4 * N * t;
      row_v0 = t * (D / 2) + 2 * N * g;
      row_v1 = (4 + (t ^ 1)) * (D / 2) + 2 * N * g;
      row_s = q4_scale_off(D) + key_g * (2 * N);
    }
    __device__ __forceinline__ void load_q(const uint4* frag) {
#pragma unroll
      for (int j = 0; j < N; ++j) qf[j] = frag[32 * j];
    }
    __device__ __forceinline__ void begin(const RunPrep& pr) {
      qs[0] = pr.extra[0];
      qs[1] = pr.extra[1];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
#pragma unroll
        for (int j = 0; j < N; ++j) o[j][0][x] = o[j][1][x] = 0.f;
#pragma unroll
        for (int j = 0; j < N / 2; ++j) co[j][x] = 0.f;
      }
    }
    // Put O and its offset together: at the end, and often enough that the offset's
    // rounding does not add up (rows of odd nibbles hold 16 times their value).
    __device__ __forceinline__ void settle() {
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
    }
    // Keys before ``first`` and after ``last`` get scales of 0: their places may hold NaN.
    __device__ __forceinline__ void hide(uint8_t* slot, int key0, int first, int last) const {
      const int key = key0 + lane;
      if (lane < kRunTile && (key > last || key < first)) {
        uint8_t* sk = slot + (lane >> 4) * BLK + q4_scale_off(D) + (lane & 15) * (2 * N);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          reinterpret_cast<uint32_t*>(sk)[j] = 0u;
          reinterpret_cast<uint32_t*>(sk + U * BLK)[j] = 0u;
        }
      }
    }
    // scales of rows g (x = 0) and g + 8, two groups to a word
    __device__ __forceinline__ void load_scales(const uint8_t* blk, uint32_t (&sc)[2][N / 2]) const {
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
    }
    __device__ __forceinline__ static float scale_of(const uint32_t (&sc)[2][N / 2], int x, int j) {
      return __uint_as_float((j & 1) ? sc[x][j >> 1] & 0xffff0000u : sc[x][j >> 1] << 16);
    }
    // Products with q, from sum_j s_j (-8 sum_j(q)) on; 1 / kDown of <q, k>.
    __device__ __forceinline__ void scores(const DecodeBlocksParams&, const uint8_t* slot, float (&sc)[U][4]) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint8_t* kp = slot + u * BLK;
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
        mma_16816_new(sc[u], z0, z1, z0, z1, qs[0], qs[1]);
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
    }
    __device__ __forceinline__ float score(const DecodeBlocksParams& p, int, int, float raw, float bias,
                                           bool hidden) const {
      const float s = fmaf(raw, p.scale, bias);
      return MULTI && hidden ? -INFINITY : s;  // (of a key that other rows see: its scale may be NaN)
    }
    template <class Sees>
    __device__ __forceinline__ void mark(const uint8_t*, float (&)[U][4], float (&)[2], const Sees&) const {
    }  // a NaN is in its group's scale
    __device__ __forceinline__ bool v_scales(const uint8_t*) { return false; }  // V has no base
    __device__ __forceinline__ float v_rebase() { return 1.f; }
    __device__ __forceinline__ void rescale(int x, float al) {
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
    __device__ __forceinline__ void values(const uint8_t* slot, uint32_t slot_bar, const float (&sc)[U][4],
                                           uint32_t hidden) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint8_t* vp = slot + (U + u) * BLK;
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
          if (lane == 0) mbar_arrive(slot_bar);  // the tile is in registers
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
            for (int x = 0; x < 4; ++x) w[x] = hidden >> (4 * u + x) & 1u ? 0.f : w[x];
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
    __device__ __forceinline__ void store(int x, float* row) const {  // channels 32j + 4g + 0..3
      const int g = lane >> 2;
#pragma unroll
      for (int j = 0; j < N; ++j)
        *reinterpret_cast<float4*>(row + 32 * j + 4 * g) =
            make_float4(o[j][0][x] * kDown, o[j][0][x + 2] * (kDown / 16), o[j][1][x] * kDown,
                        o[j][1][x + 2] * (kDown / 16));
    }
  };
};

size_t decode_q4_workspace_bytes(int32_t, int32_t QL, int32_t H_q, int32_t H_kv, int32_t D, int32_t sms) {
  return RunPlan(QL, H_q, H_kv, D, sms).total;
}

struct Q4Launch {
  template <int D, bool MULTI>
  static bool launch(const DecodeBlocksCall& c, const DecodeBlocksParams& p, const RunPlan& plan, int smem) {
    auto kern = decode_blocks_kernel<Q4Format, D, MULTI>;
    static std::atomic<int> limit_set[kMaxDevices];
    return smem_limit_on_device(reinterpret_cast<const void*>(kern), kRunSmemBudget, limit_set) &&
           launch_dependent(kern, dim3(plan.grid), run_threads<Q4Format, MULTI>(), smem, p, c.stream) &&
           launch_dependent(merge_blocks_kernel<D>, dim3(plan.grid, plan.NR), 32 * kRunMergeWarps, 0, p, c.stream);
  }
};

int launch_decode_q4(const DecodeBlocksCall& c) { return launch_blocks<Q4Format, Q4Launch>(c, c.scale * kDown); }

}  // namespace ira

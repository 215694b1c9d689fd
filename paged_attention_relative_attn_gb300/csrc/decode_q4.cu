// Decode attention with the relative-position bias over the 4-bit cache.
//
// Operation: inkling_rel_attn_decode_q4 in include/inkling_rel_attn.h.
//
// One block per (sequence, KV head, token group); its rows are the group's
// (token, query head) pairs, at most 16.  Its warps take the 16-token blocks of
// the visible range in turn.  Per block a warp forms S^T = K Q^T (16 keys x rows)
// and O^T += V^T P^T with mma.sync m16n8k16 in bf16:
//  * a nibble u becomes the bf16 number 128 + u by or-ing it into the mantissa
//    of 128 -- one instruction for two values; the excess 136 over x = u - 8 is
//    taken out by products with a constant matrix of -136: once per item for K
//    (the accumulators of a group start at -136 sum(q)), and with the same
//    rounded P for V, so nothing but P's own rounding is left;
//  * a group's scale is a factor of its own accumulator for K, in fp32, and of
//    P for V, before P is rounded to bf16 (the operand type of the product; 2^-9
//    relative, as the bf16 cache's decode rounds it).
// Masked keys get P = 0 and scale 0: a page's unused rows may hold anything.
#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "plan.cuh"
#include "ptx.cuh"
#include "q4.cuh"

namespace ira {

constexpr int kDq4Warps = 8;
constexpr int kDq4Threads = 32 * kDq4Warps;

struct DecodeQ4Params {
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const float* rel;
  __nv_bfloat16* out;
  float* lse_out;
  int32_t* dev_err;
  int B, pt_stride, H_q, H_kv, G, P, num_pages, R, window;
  int QL, TG, NG;  // query tokens per sequence, per item, items per (sequence, KV head)
  float scale;
};

// Nibble n (0..3) of both halves of w as the bf16 pair 128 + u.
template <int n>
__device__ __forceinline__ uint32_t q4_expand(uint32_t w) {
  return ((w >> (4 * n)) & 0x000f000fu) | 0x43004300u;
}
constexpr uint32_t kMinus136 = 0xc308c308u;

template <int D, int NT>
__global__ void __launch_bounds__(kDq4Threads) decode_q4_kernel(const __grid_constant__ DecodeQ4Params p) {
  constexpr int N = D / kQ4Group;  // groups of a row
  constexpr int HP = 8 * NT;
  constexpr int OP = D + 4;
  extern __shared__ float comb[];  // [warps][rows][D + 4], then m, l
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = p.G;
  const int b = blockIdx.x / (p.H_kv * p.NG);
  const int rest = blockIdx.x - b * p.H_kv * p.NG;
  const int hkv = rest / p.NG, grp = rest - hkv * p.NG;
  const int first = grp * p.TG, tn = min(p.TG, p.QL - first);
  const int NR = p.TG * G, rows = tn * G;
  float* comb_m = comb + kDq4Warps * NR * OP;
  float* comb_l = comb_m + kDq4Warps * HP;

  const int L_in = __ldg(p.seq_lens + b);
  const int L = min(max(L_in, 0), p.pt_stride * p.P);
  if (tid == 0 && hkv == 0 && grp == 0) {
    if (L_in > L) report(p.dev_err, INKLING_DEVERR_SEQ_TOO_LONG);
    if (p.QL > 1 && L < p.QL) report(p.dev_err, INKLING_DEVERR_BAD_CHUNK);
  }
  auto out_row = [&](int r) -> size_t {
    const int i = r / G;
    return ((size_t)b * p.QL + first + i) * p.H_q + hkv * G + (r - i * G);
  };
  if (L < p.QL) {  // nothing visible (or fewer keys than new tokens)
    for (int x = tid; x < rows * D; x += kDq4Threads) p.out[out_row(x / D) * D + x % D] = __float2bfloat16(0.f);
    if (p.lse_out && tid < rows) p.lse_out[out_row(tid)] = -INFINITY;
    return;
  }
  const int pos1 = L - p.QL + first + tn - 1;  // the group's last position
  const int pos0 = pos1 - tn + 1;
  const int lo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;

  // ---- q fragments (channel order of the K rows) and -136 sum(q) per group
  uint32_t qf[N][2][NT][2];
  float qsum[N][NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + g;
    const bool live = r < rows;
    const __nv_bfloat16* qr = p.q + (live ? out_row(r) : 0) * D;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      uint4 w = make_uint4(0, 0, 0, 0);  // channels 32j + 8t + 0..7
      if (live) w = __ldg(reinterpret_cast<const uint4*>(qr + 32 * j + 8 * t));
      qf[j][0][nt][0] = __byte_perm(w.x, w.z, 0x5410);  // c, c + 4 for c = 0..3
      qf[j][0][nt][1] = __byte_perm(w.x, w.z, 0x7632);
      qf[j][1][nt][0] = __byte_perm(w.y, w.w, 0x5410);
      qf[j][1][nt][1] = __byte_perm(w.y, w.w, 0x7632);
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i)
        mma_16816(c, kMinus136, kMinus136, kMinus136, kMinus136, qf[j][i][nt][0], qf[j][i][nt][1]);
      qsum[j][nt][0] = c[0];
      qsum[j][nt][1] = c[1];
    }
  }
  // position and bias row of this lane's score columns
  int row_pos[NT][2];
  const float* row_rel[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = min(nt * 8 + 2 * t + x, rows - 1);
      row_pos[nt][x] = pos0 + r / G;
      row_rel[nt][x] = p.rel + out_row(r) * p.R;
    }

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

  const int32_t* pt_row = p.page_table + (size_t)b * p.pt_stride;
  for (int blk = (lo >> 4) + warp; blk <= (pos1 >> 4); blk += kDq4Warps) {
    const int key0 = blk * 16;
    const int lp = key0 / p.P;
    const int page = __ldg(pt_row + lp);
    const bool ok = page >= 0 && page < p.num_pages;
    if (!ok && lane == 0) report(p.dev_err, INKLING_DEVERR_BAD_PAGE);
    uint32_t kw[2][N], vw[4][(N + 1) / 2], ksc[2][(N + 1) / 2], vsc[2][(N + 1) / 2];
    const size_t at = q4_block_at(ok ? page : 0, hkv, key0 - lp * p.P, p.H_kv, p.P, D);
    const uint8_t* kb = p.k_cache + at;
    const uint8_t* vb = p.v_cache + at;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < N; ++j)
        kw[x][j] = __ldg(reinterpret_cast<const uint32_t*>(kb + (g + 8 * x) * (D / 2)) + N * t + j);
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int j = 0; j < N / 2; ++j)
        vw[x][j] = __ldg(reinterpret_cast<const uint32_t*>(vb + (2 * t + (x & 1) + 8 * (x >> 1)) * (D / 2)) +
                         (N / 2) * g + j);
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < N / 2; ++j) {
        const int w = (g + 8 * x) * (N / 2) + j;
        ksc[x][j] = ok ? __ldg(reinterpret_cast<const uint32_t*>(kb + q4_scale_off(D)) + w) : 0u;
        vsc[x][j] = ok ? __ldg(reinterpret_cast<const uint32_t*>(vb + q4_scale_off(D)) + w) : 0u;
      }
    auto scale_of = [&](const uint32_t (&s)[2][(N + 1) / 2], int x, int j) {
      return __uint_as_float((j & 1) ? s[x][j >> 1] & 0xffff0000u : s[x][j >> 1] << 16);
    };

    uint32_t pb[N][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // ---- scores of 16 keys x 8 rows
      float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float c[4] = {qsum[j][nt][0], qsum[j][nt][1], qsum[j][nt][0], qsum[j][nt][1]};
        mma_16816(c, q4_expand<0>(kw[0][j]), q4_expand<0>(kw[1][j]), q4_expand<1>(kw[0][j]),
                  q4_expand<1>(kw[1][j]), qf[j][0][nt][0], qf[j][0][nt][1]);
        mma_16816(c, q4_expand<2>(kw[0][j]), q4_expand<2>(kw[1][j]), q4_expand<3>(kw[0][j]),
                  q4_expand<3>(kw[1][j]), qf[j][1][nt][0], qf[j][1][nt][1]);
#pragma unroll
        for (int x = 0; x < 4; ++x) s[x] = fmaf(c[x], scale_of(ksc, x >> 1, j), s[x]);
      }
      // ---- bias and mask
      bool see[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int dist = row_pos[nt][x & 1] - (key0 + g + 8 * (x >> 1));
        see[x] = dist >= 0 && (p.window <= 0 || dist < p.window);
        const float bias = __ldg(row_rel[nt][x & 1] + min(max(dist, 0), p.R - 1));
        s[x] = see[x] ? fmaf(s[x], p.scale, bias) : -INFINITY;
      }
      // ---- running maximum and sum
      float mx[2] = {fmaxf(s[0], s[2]), fmaxf(s[1], s[3])};
      float pr[4];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) mx[x] = fmaxf(mx[x], __shfl_xor_sync(0xffffffffu, mx[x], off));
        const float mn = fmaxf(m_run[nt][x], mx[x]);
        const float base = mn == -INFINITY ? 0.f : mn;
        // differences first: s * log2 e alone would lose them, or overflow, under a mask of fp32's lowest value
        const float al = ex2((m_run[nt][x] - base) * kLog2e);
        pr[x] = ex2((s[x] - base) * kLog2e);
        pr[x + 2] = ex2((s[x + 2] - base) * kLog2e);
        l_run[nt][x] = fmaf(l_run[nt][x], al, pr[x] + pr[x + 2]);
        m_run[nt][x] = mn;
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            o[j][i][nt][x] *= al;
            o[j][i][nt][x + 2] *= al;
          }
      }
#pragma unroll
      for (int j = 0; j < N; ++j) {
        float w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = see[x] ? pr[x] * scale_of(vsc, x >> 1, j) : 0.f;
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
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_16816(o[j][0][nt], kMinus136, kMinus136, kMinus136, kMinus136, pb[j][nt][0], pb[j][nt][1]);
        mma_16816(o[j][0][nt], q4_expand<0>(w0), q4_expand<1>(w0), q4_expand<0>(w8), q4_expand<1>(w8),
                  pb[j][nt][0], pb[j][nt][1]);
        mma_16816(o[j][1][nt], kMinus136, kMinus136, kMinus136, kMinus136, pb[j][nt][0], pb[j][nt][1]);
        mma_16816(o[j][1][nt], q4_expand<2>(w0), q4_expand<3>(w0), q4_expand<2>(w8), q4_expand<3>(w8),
                  pb[j][nt][0], pb[j][nt][1]);
      }
    }
  }

  // ---- the warps' parts
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
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float* dst = comb + (warp * NR + r) * OP + 32 * j + 4 * g + 2 * i;
            dst[0] = o[j][i][nt][x];
            dst[1] = o[j][i][nt][x + 2];
          }
      }
    }
  __syncthreads();
  for (int x = tid; x < rows * D; x += kDq4Threads) {
    const int r = x / D, d = x - r * D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kDq4Warps; ++w) M = fmaxf(M, comb_m[w * HP + r]);
    const float base = M == -INFINITY ? 0.f : M;
    float l = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kDq4Warps; ++w) {
      const float sc = ex2((comb_m[w * HP + r] - base) * kLog2e);
      l = fmaf(sc, comb_l[w * HP + r], l);
      acc = fmaf(sc, comb[(w * NR + r) * OP + d], acc);
    }
    // every score -inf: an empty row
    p.out[out_row(r) * D + d] = __float2bfloat16(l == 0.f ? 0.f : acc / l);
    if (d == 0 && p.lse_out) p.lse_out[out_row(r)] = M + logf(l);
  }
}

template <int D, int NT>
static int launch_decode_q4_t(const DecodeQ4Call& c, const DecodeQ4Params& prm) {
  auto kern = decode_q4_kernel<D, NT>;
  const int NR = prm.TG * prm.G;
  const int smem = kDq4Warps * (NR * (D + 4) + 2 * 8 * NT) * 4;
  static std::atomic<int> limit_set[kMaxDevices];
  if (!smem_limit_on_device(reinterpret_cast<const void*>(kern), kDq4Warps * (8 * NT * (D + 4) + 16 * NT) * 4,
                            limit_set))
    return INKLING_ERR_CUDA;
  const int64_t grid = (int64_t)c.B * c.H_kv * prm.NG;
  if (grid > INT32_MAX) return INKLING_ERR_ARG;
  kern<<<(unsigned)grid, kDq4Threads, smem, c.stream>>>(prm);
  return cudaGetLastError() == cudaSuccess ? INKLING_OK : INKLING_ERR_CUDA;
}

size_t decode_q4_workspace_bytes(int32_t, int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

int launch_decode_q4(const DecodeQ4Call& c) {
  DecodeQ4Params p;
  p.q = static_cast<const __nv_bfloat16*>(c.q);
  p.k_cache = static_cast<const uint8_t*>(c.k_cache);
  p.v_cache = static_cast<const uint8_t*>(c.v_cache);
  p.page_table = c.page_table;
  p.seq_lens = c.seq_lens;
  p.rel = c.rel;
  p.out = static_cast<__nv_bfloat16*>(c.out);
  p.lse_out = c.lse_out;
  p.dev_err = c.dev_err;
  p.B = c.B;
  p.pt_stride = c.pt_stride;
  p.H_q = c.H_q;
  p.H_kv = c.H_kv;
  p.G = c.H_q / c.H_kv;
  p.P = c.P;
  p.num_pages = c.num_pages;
  p.R = c.R;
  p.window = c.window;
  p.QL = c.QL;
  p.TG = decode_token_group(c.QL, p.G);
  p.NG = (c.QL + p.TG - 1) / p.TG;
  p.scale = c.scale;
  const int NT = p.TG * p.G <= 8 ? 1 : 2;
  if (c.D == 128) return NT == 1 ? launch_decode_q4_t<128, 1>(c, p) : launch_decode_q4_t<128, 2>(c, p);
  return NT == 1 ? launch_decode_q4_t<64, 1>(c, p) : launch_decode_q4_t<64, 2>(c, p);
}

}  // namespace ira

// What the entry points of the 4-bit and the 8-bit cache share: argument checks,
// workspace layout, and calls that differ in the launcher alone.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"

namespace ira {

inline bool cache_shape_ok(int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages) {
  if (H_kv <= 0 || (D != 64 && D != 128)) return false;
  return page_size > 0 && page_size % 16 == 0 && page_size <= 256 && num_pages > 0;
}

// Scratch pages (64 tokens) that hold what a chunk of max_q_len tokens sees.
inline int64_t expanded_pages(int32_t max_q_len, int32_t window, int32_t max_seq_len) {
  int64_t keys = std::max<int32_t>(max_seq_len, 1);
  // the first visible key is rounded down to a multiple of 64
  if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window - 1 + std::max<int32_t>(max_q_len, 0) + 63);
  return (keys + 63) / 64;
}

struct ExpandedLayout {
  int64_t pages;  // per sequence
  size_t table, lens, k, v, total;
  ExpandedLayout(int32_t B, int32_t max_q_len, int32_t H_kv, int32_t D, int32_t window, int32_t max_seq_len) {
    pages = expanded_pages(max_q_len, window, max_seq_len);
    const size_t pool = align256((size_t)B * pages * 64 * H_kv * D * 2);
    table = 0;
    lens = align256((size_t)B * pages * 4);
    k = lens + align256((size_t)B * 4);
    v = k + pool;
    total = v + pool;
  }
};

inline int rows_call(int (*launch)(const RowsCall&, bool), bool append, void* k_rows, void* v_rows,
                     const int64_t* slot_map, int32_t T, int32_t H_kv, int32_t D, int32_t page_size,
                     int32_t num_pages, void* k_cache, void* v_cache, int32_t* device_error, void* stream) {
  if (T < 0 || !cache_shape_ok(H_kv, D, page_size, num_pages)) return INKLING_ERR_ARG;
  if (H_kv > 65535) return INKLING_ERR_ARG;  // heads are a dimension of the grid
  if (T == 0) return INKLING_OK;
  if (!k_rows || !v_rows || !slot_map || !k_cache || !v_cache) return INKLING_ERR_ARG;
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_map, 8) || !aligned(device_error, 4))
    return INKLING_ERR_ALIGN;
  if (device_info().ok != 1) return INKLING_ERR_DEVICE;
  RowsCall c;
  c.k_rows = k_rows;
  c.v_rows = v_rows;
  c.k_cache = k_cache;
  c.v_cache = v_cache;
  c.slots = slot_map;
  c.T = T;
  c.H_kv = H_kv;
  c.D = D;
  c.P = page_size;
  c.num_pages = num_pages;
  c.dev_err = device_error;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch(c, append);
}

inline int decode_call(int (*launch)(const DecodeBlocksCall&), const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* page_table, int32_t page_table_stride, const int32_t* seq_lens,
                       const float* rel_logits, int32_t B, int32_t q_len, int32_t H_q, int32_t H_kv, int32_t D,
                       int32_t page_size, int32_t num_pages, int32_t R, int32_t window, float scale, void* out,
                       float* lse_out, void* workspace, size_t workspace_bytes, int32_t* device_error,
                       void* stream) {
  if (B < 0 || q_len < 1 || q_len > 64) return INKLING_ERR_ARG;
  if (!common_shape_ok(H_q, H_kv, D, page_size, num_pages, R, page_table_stride)) return INKLING_ERR_ARG;
  if ((int64_t)B * q_len * H_q > INT32_MAX / 4) return INKLING_ERR_ARG;
  if ((int64_t)num_pages * H_kv > INT32_MAX / (page_size / 16)) return INKLING_ERR_ARG;  // the pool's blocks
  if (!(scale >= -0x1p54f && scale <= 0x1p54f)) return INKLING_ERR_ARG;  // (4-bit: times 2^73 it stays finite)
  if (B == 0) return INKLING_OK;
  if (!q || !k_cache || !v_cache || !page_table || !seq_lens || !rel_logits || !out) return INKLING_ERR_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(workspace, 16) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(rel_logits, 4) ||
      !aligned(lse_out, 4) || !aligned(device_error, 4))
    return INKLING_ERR_ALIGN;
  const DevInfo di = device_info();
  if (di.ok != 1) return INKLING_ERR_DEVICE;
  const size_t need = decode_q4_workspace_bytes(B, q_len, H_q, H_kv, D, di.sms);
  if (need > 0 && (!workspace || workspace_bytes < need)) return INKLING_ERR_WORKSPACE;
  DecodeBlocksCall c;
  c.q = q;
  c.k_cache = k_cache;
  c.v_cache = v_cache;
  c.page_table = page_table;
  c.pt_stride = page_table_stride;
  c.seq_lens = seq_lens;
  c.rel = rel_logits;
  c.B = B;
  c.QL = q_len;
  c.H_q = H_q;
  c.H_kv = H_kv;
  c.D = D;
  c.P = page_size;
  c.num_pages = num_pages;
  c.R = R;
  c.window = window;
  c.scale = scale;
  c.out = out;
  c.lse_out = lse_out;
  c.workspace = workspace;
  c.sms = di.sms;
  c.dev_err = device_error;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch(c);
}

inline int prefill_call(int (*expand)(const ExpandCall&), const void* q, const int32_t* cu_seqlens_q,
                        const void* k_cache, const void* v_cache, const int32_t* page_table,
                        int32_t page_table_stride, const int32_t* seq_lens, const float* rel_logits, int32_t B,
                        int32_t T, int32_t max_q_len, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                        int32_t num_pages, int32_t R, int32_t window, float scale, int32_t max_seq_len, void* out,
                        float* lse_out, void* workspace, size_t workspace_bytes, int32_t* device_error,
                        void* stream) {
  if (B < 0 || T < 0 || max_q_len < 0 || max_seq_len < 0) return INKLING_ERR_ARG;
  if (!common_shape_ok(H_q, H_kv, D, page_size, num_pages, R, page_table_stride)) return INKLING_ERR_ARG;
  if (R % 4 != 0) return INKLING_ERR_ARG;
  if (!(scale == scale)) return INKLING_ERR_ARG;
  if (B == 0 || T == 0 || max_q_len == 0) return INKLING_OK;
  if (!q || !cu_seqlens_q || !k_cache || !v_cache || !page_table || !seq_lens || !rel_logits || !out)
    return INKLING_ERR_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16) ||
      !aligned(rel_logits, 16) || !aligned(workspace, 256) || !aligned(page_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(cu_seqlens_q, 4) || !aligned(lse_out, 4) || !aligned(device_error, 4))
    return INKLING_ERR_ALIGN;
  const ExpandedLayout lay(B, max_q_len, H_kv, D, window, max_seq_len);
  // grid limits of the expansion and of the attention; scratch page ids are int32
  if (lay.pages * 64 > INT32_MAX - 64 || B * lay.pages > INT32_MAX) return INKLING_ERR_ARG;
  if ((int64_t)B * ((max_q_len + 127LL) / 128) > 65535) return INKLING_ERR_ARG;
  if (device_info().ok != 1) return INKLING_ERR_DEVICE;
  if (!workspace || workspace_bytes < lay.total) return INKLING_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  ExpandCall e;
  e.k_cache = k_cache;
  e.v_cache = v_cache;
  e.page_table = page_table;
  e.pt_stride = page_table_stride;
  e.cu_seqlens_q = cu_seqlens_q;
  e.seq_lens = seq_lens;
  e.B = B;
  e.H_kv = H_kv;
  e.D = D;
  e.P = page_size;
  e.num_pages = num_pages;
  e.window = window;
  e.pages_per_seq = (int32_t)lay.pages;
  e.k_out = ws + lay.k;
  e.v_out = ws + lay.v;
  e.table_out = reinterpret_cast<int32_t*>(ws + lay.table);
  e.lens_out = reinterpret_cast<int32_t*>(ws + lay.lens);
  e.dev_err = device_error;
  e.stream = static_cast<cudaStream_t>(stream);
  const int rc = expand(e);
  if (rc != INKLING_OK) return rc;
  PrefillCall c;
  c.q = q;
  c.cu_seqlens_q = cu_seqlens_q;
  c.k_cache = e.k_out;
  c.v_cache = e.v_out;
  c.page_table = e.table_out;
  c.pt_stride = (int32_t)lay.pages;
  c.seq_lens = e.lens_out;
  c.rel = rel_logits;
  c.B = B;
  c.T = T;
  c.max_q_len = max_q_len;
  c.H_q = H_q;
  c.H_kv = H_kv;
  c.D = D;
  c.P = 64;
  c.num_pages = (int32_t)(B * lay.pages);
  c.R = R;
  c.window = window;
  c.scale = scale;
  c.max_seq_len = (int32_t)(lay.pages * 64);
  c.out = out;
  c.lse_out = lse_out;
  c.dev_err = device_error;
  c.stream = static_cast<cudaStream_t>(stream);
  c.after_expansion = true;
  return launch_prefill(c);
}

}  // namespace ira

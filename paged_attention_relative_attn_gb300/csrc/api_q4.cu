// C ABI of the 4-bit cache and the step tables: argument checks, workspace
// layout and launches.  See include/inkling_rel_attn.h for the contracts.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>

#include "internal.h"

using namespace ira;

namespace {

bool cache_shape_ok(int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages) {
  if (H_kv <= 0 || (D != 64 && D != 128)) return false;
  return page_size > 0 && page_size % 16 == 0 && page_size <= 256 && num_pages > 0;
}

// Scratch pages (64 tokens) that hold what a chunk of max_q_len tokens sees.
int64_t prefill_q4_pages(int32_t max_q_len, int32_t window, int32_t max_seq_len) {
  int64_t keys = std::max<int32_t>(max_seq_len, 1);
  // the first visible key is rounded down to a multiple of 64
  if (window > 0) keys = std::min<int64_t>(keys, (int64_t)window - 1 + std::max<int32_t>(max_q_len, 0) + 63);
  return (keys + 63) / 64;
}

struct PrefillQ4Layout {
  int64_t pages;  // per sequence
  size_t table, lens, k, v, total;
  PrefillQ4Layout(int32_t B, int32_t max_q_len, int32_t H_kv, int32_t D, int32_t window, int32_t max_seq_len) {
    pages = prefill_q4_pages(max_q_len, window, max_seq_len);
    const size_t pool = align256((size_t)B * pages * 64 * H_kv * D * 2);
    table = 0;
    lens = align256((size_t)B * pages * 4);
    k = lens + align256((size_t)B * 4);
    v = k + pool;
    total = v + pool;
  }
};

int rows_q4(bool append, void* k_rows, void* v_rows, const int64_t* slot_map, int32_t T, int32_t H_kv, int32_t D,
            int32_t page_size, int32_t num_pages, void* k_cache, void* v_cache, int32_t* device_error,
            void* stream) {
  if (T < 0 || !cache_shape_ok(H_kv, D, page_size, num_pages)) return INKLING_ERR_ARG;
  if (H_kv > 65535) return INKLING_ERR_ARG;  // heads are a dimension of the grid
  if (T == 0) return INKLING_OK;
  if (!k_rows || !v_rows || !slot_map || !k_cache || !v_cache) return INKLING_ERR_ARG;
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_map, 8) || !aligned(device_error, 4))
    return INKLING_ERR_ALIGN;
  if (device_info().ok != 1) return INKLING_ERR_DEVICE;
  Q4RowsCall c;
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
  return launch_q4_rows(c, append);
}

}  // namespace

extern "C" {

int inkling_rel_attn_build_tables(const int32_t* seq_lens, const int32_t* new_lens, int32_t* page_table,
                                  int32_t page_table_stride, int32_t* free_pages, const int32_t* free_count,
                                  int32_t B, int32_t page_size, int32_t num_pages, int32_t max_tokens,
                                  int32_t* kv_lens, int32_t* cu_seqlens_q, int64_t* slot_map,
                                  int32_t* free_left, int32_t* device_error, void* stream) {
  return inkling_rel_attn_build_tables_step(seq_lens, new_lens, page_table, page_table_stride, free_pages, free_count,
                                            B, page_size, num_pages, max_tokens, kv_lens, cu_seqlens_q, slot_map,
                                            free_left, nullptr, device_error, stream);
}

int inkling_rel_attn_build_tables_step(const int32_t* seq_lens, const int32_t* new_lens, int32_t* page_table,
                                       int32_t page_table_stride, int32_t* free_pages, const int32_t* free_count,
                                       int32_t B, int32_t page_size, int32_t num_pages, int32_t max_tokens,
                                       int32_t* kv_lens, int32_t* cu_seqlens_q, int64_t* slot_map,
                                       int32_t* free_left, int32_t* step_lens, int32_t* device_error, void* stream) {
  if (B < 0 || B > kTablesMaxBatch || max_tokens < 0 || max_tokens == INT32_MAX) return INKLING_ERR_ARG;
  if (page_size <= 0 || page_size % 16 != 0 || page_size > 256) return INKLING_ERR_ARG;
  if (num_pages <= 0 || num_pages == INT32_MAX || page_table_stride <= 0) return INKLING_ERR_ARG;
  if ((int64_t)page_table_stride * page_size > INT32_MAX) return INKLING_ERR_ARG;
  if (B == 0) return INKLING_OK;
  if (!seq_lens || !new_lens || !page_table || !free_pages || !free_count || !kv_lens || !cu_seqlens_q ||
      !free_left || (max_tokens > 0 && !slot_map))
    return INKLING_ERR_ARG;
  if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(page_table, 4) || !aligned(free_pages, 4) ||
      !aligned(free_count, 4) || !aligned(kv_lens, 4) || !aligned(cu_seqlens_q, 4) || !aligned(slot_map, 8) ||
      !aligned(free_left, 4) || !aligned(step_lens, 4) || !aligned(device_error, 4))
    return INKLING_ERR_ALIGN;
  if (device_info().ok != 1) return INKLING_ERR_DEVICE;
  TablesCall c;
  c.seq_lens = seq_lens;
  c.new_lens = new_lens;
  c.page_table = page_table;
  c.pt_stride = page_table_stride;
  c.free_pages = free_pages;
  c.free_count = free_count;
  c.B = B;
  c.P = page_size;
  c.num_pages = num_pages;
  c.max_tokens = max_tokens;
  c.kv_lens = kv_lens;
  c.cu_seqlens_q = cu_seqlens_q;
  c.slot_map = slot_map;
  c.free_left = free_left;
  c.step_lens = step_lens;
  c.dev_err = device_error;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_build_tables(c);
}

int inkling_rel_attn_kv_append_q4(const void* k_new, const void* v_new, const int64_t* slot_map, int32_t T,
                                  int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages, void* k_cache,
                                  void* v_cache, int32_t* device_error, void* stream) {
  return rows_q4(true, const_cast<void*>(k_new), const_cast<void*>(v_new), slot_map, T, H_kv, D, page_size,
                 num_pages, k_cache, v_cache, device_error, stream);
}

int inkling_rel_attn_kv_read_q4(const int64_t* slot_map, const void* k_cache, const void* v_cache, int32_t T,
                                int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages, void* k_rows,
                                void* v_rows, int32_t* device_error, void* stream) {
  return rows_q4(false, k_rows, v_rows, slot_map, T, H_kv, D, page_size, num_pages, const_cast<void*>(k_cache),
                 const_cast<void*>(v_cache), device_error, stream);
}

size_t inkling_rel_attn_decode_q4_workspace_size(int32_t B, int32_t q_len, int32_t H_q, int32_t H_kv, int32_t D,
                                                 int32_t num_sms) {
  if (B <= 0 || q_len < 1 || H_q <= 0 || H_kv <= 0 || H_q % H_kv != 0 || D <= 0) return 0;
  if (num_sms <= 0) {
    const DevInfo di = device_info();
    num_sms = di.ok >= 0 && di.sms > 0 ? di.sms : 152;
  }
  return decode_q4_workspace_bytes(B, q_len, H_q, H_kv, D, num_sms);
}

int inkling_rel_attn_decode_q4(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                               int32_t page_table_stride, const int32_t* seq_lens, const float* rel_logits,
                               int32_t B, int32_t q_len, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                               int32_t num_pages, int32_t R, int32_t window, float scale, void* out,
                               float* lse_out, void* workspace, size_t workspace_bytes, int32_t* device_error,
                               void* stream) {
  if (B < 0 || q_len < 1 || q_len > 64) return INKLING_ERR_ARG;
  if (!common_shape_ok(H_q, H_kv, D, page_size, num_pages, R, page_table_stride)) return INKLING_ERR_ARG;
  if ((int64_t)B * q_len * H_q > INT32_MAX / 4) return INKLING_ERR_ARG;
  if ((int64_t)num_pages * H_kv > INT32_MAX / (page_size / 16)) return INKLING_ERR_ARG;  // the pool's blocks
  if (!(scale >= -0x1p54f && scale <= 0x1p54f)) return INKLING_ERR_ARG;  // times 2^73 it stays finite
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
  DecodeQ4Call c;
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
  return launch_decode_q4(c);
}

size_t inkling_rel_attn_prefill_q4_workspace_size(int32_t B, int32_t max_q_len, int32_t H_kv, int32_t D,
                                                  int32_t window, int32_t max_seq_len) {
  if (B <= 0 || max_q_len <= 0 || H_kv <= 0 || D <= 0) return 0;
  return PrefillQ4Layout(B, max_q_len, H_kv, D, window, max_seq_len).total;
}

int inkling_rel_attn_prefill_q4(const void* q, const int32_t* cu_seqlens_q, const void* k_cache,
                                const void* v_cache, const int32_t* page_table, int32_t page_table_stride,
                                const int32_t* seq_lens, const float* rel_logits, int32_t B, int32_t T,
                                int32_t max_q_len, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                                int32_t num_pages, int32_t R, int32_t window, float scale, int32_t max_seq_len,
                                void* out, float* lse_out, void* workspace, size_t workspace_bytes,
                                int32_t* device_error, void* stream) {
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
  const PrefillQ4Layout lay(B, max_q_len, H_kv, D, window, max_seq_len);
  // grid limits of the expansion and of the attention; scratch page ids are int32
  if (lay.pages * 64 > INT32_MAX - 64 || B * lay.pages > INT32_MAX) return INKLING_ERR_ARG;
  if ((int64_t)B * ((max_q_len + 127LL) / 128) > 65535) return INKLING_ERR_ARG;
  if (device_info().ok != 1) return INKLING_ERR_DEVICE;
  if (!workspace || workspace_bytes < lay.total) return INKLING_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  Q4ExpandCall e;
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
  const int rc = launch_q4_expand(e);
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

int inkling_rel_attn_packed(int32_t call, const int64_t* a, int32_t count) {
  if (!a) return INKLING_ERR_ARG;
  int at = 0;
  bool fits = true;
  auto ptr = [&]() { return reinterpret_cast<void*>(a[at++]); };
  auto i32 = [&]() {
    const int64_t v = a[at++];
    fits = fits && v >= INT32_MIN && v <= INT32_MAX;
    return (int32_t)v;
  };
  auto real = [&]() {
    double v;
    std::memcpy(&v, a + at++, sizeof(v));
    return (float)v;
  };
  auto ci = [&]() { return static_cast<const int32_t*>(ptr()); };
  // (braces: arguments are taken in order)
  switch (call) {
    case INKLING_PACKED_BUILD_TABLES: {
      if (count != 16 && count != 17) return INKLING_ERR_ARG;
      const int32_t *seq_lens = ci(), *new_lens = ci();
      int32_t* table = static_cast<int32_t*>(ptr());
      const int32_t stride = i32();
      int32_t* free_pages = static_cast<int32_t*>(ptr());
      const int32_t* free_count = ci();
      const int32_t B = i32(), page_size = i32(), num_pages = i32(), max_tokens = i32();
      int32_t* kv_lens = static_cast<int32_t*>(ptr());
      int32_t* cu = static_cast<int32_t*>(ptr());
      int64_t* slots = static_cast<int64_t*>(ptr());
      int32_t* left = static_cast<int32_t*>(ptr());
      int32_t* step = count == 17 ? static_cast<int32_t*>(ptr()) : nullptr;
      int32_t* err = static_cast<int32_t*>(ptr());
      void* stream = ptr();
      if (!fits) return INKLING_ERR_ARG;
      return inkling_rel_attn_build_tables_step(seq_lens, new_lens, table, stride, free_pages, free_count, B, page_size,
                                                num_pages, max_tokens, kv_lens, cu, slots, left, step, err, stream);
    }
    case INKLING_PACKED_KV_APPEND_Q4:
    case INKLING_PACKED_KV_READ_Q4: {
      if (count != 12) return INKLING_ERR_ARG;
      void *x = ptr(), *y = ptr(), *z = ptr();
      const int32_t T = i32(), H_kv = i32(), D = i32(), page_size = i32(), num_pages = i32();
      void *u = ptr(), *w = ptr();
      int32_t* err = static_cast<int32_t*>(ptr());
      void* stream = ptr();
      if (!fits) return INKLING_ERR_ARG;
      if (call == INKLING_PACKED_KV_APPEND_Q4)
        return inkling_rel_attn_kv_append_q4(x, y, static_cast<const int64_t*>(z), T, H_kv, D, page_size, num_pages, u,
                                             w, err, stream);
      return inkling_rel_attn_kv_read_q4(static_cast<const int64_t*>(x), y, z, T, H_kv, D, page_size, num_pages, u, w,
                                         err, stream);
    }
    case INKLING_PACKED_DECODE_Q4: {
      if (count != 23) return INKLING_ERR_ARG;
      const void *q = ptr(), *k = ptr(), *v = ptr();
      const int32_t* table = ci();
      const int32_t stride = i32();
      const int32_t* seq_lens = ci();
      const float* rel = static_cast<const float*>(ptr());
      const int32_t B = i32(), q_len = i32(), H_q = i32(), H_kv = i32(), D = i32(), page_size = i32(),
                    num_pages = i32(), R = i32(), window = i32();
      const float scale = real();
      void* out = ptr();
      float* lse = static_cast<float*>(ptr());
      void* ws = ptr();
      const size_t ws_bytes = (size_t)a[at++];
      int32_t* err = static_cast<int32_t*>(ptr());
      if (!fits) return INKLING_ERR_ARG;
      return inkling_rel_attn_decode_q4(q, k, v, table, stride, seq_lens, rel, B, q_len, H_q, H_kv, D, page_size,
                                        num_pages, R, window, scale, out, lse, ws, ws_bytes, err, ptr());
    }
    case INKLING_PACKED_PREFILL_Q4: {
      if (count != 26) return INKLING_ERR_ARG;
      const void* q = ptr();
      const int32_t* cu = ci();
      const void *k = ptr(), *v = ptr();
      const int32_t* table = ci();
      const int32_t stride = i32();
      const int32_t* seq_lens = ci();
      const float* rel = static_cast<const float*>(ptr());
      const int32_t B = i32(), T = i32(), max_q_len = i32(), H_q = i32(), H_kv = i32(), D = i32(),
                    page_size = i32(), num_pages = i32(), R = i32(), window = i32();
      const float scale = real();
      const int32_t max_seq_len = i32();
      void* out = ptr();
      float* lse = static_cast<float*>(ptr());
      void* ws = ptr();
      const size_t ws_bytes = (size_t)a[at++];
      int32_t* err = static_cast<int32_t*>(ptr());
      if (!fits) return INKLING_ERR_ARG;
      return inkling_rel_attn_prefill_q4(q, cu, k, v, table, stride, seq_lens, rel, B, T, max_q_len, H_q, H_kv, D,
                                         page_size, num_pages, R, window, scale, max_seq_len, out, lse, ws, ws_bytes,
                                         err, ptr());
    }
  }
  return INKLING_ERR_ARG;
}

}  // extern "C"

// C ABI of the 4-bit cache and the step tables, and the calls packed into words.  See include/inkling_rel_attn.h for the contracts.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "api_blocks.h"

using namespace ira;

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
  return rows_call(launch_q4_rows, true, const_cast<void*>(k_new), const_cast<void*>(v_new), slot_map, T, H_kv, D, page_size,
                 num_pages, k_cache, v_cache, device_error, stream);
}

int inkling_rel_attn_kv_read_q4(const int64_t* slot_map, const void* k_cache, const void* v_cache, int32_t T,
                                int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages, void* k_rows,
                                void* v_rows, int32_t* device_error, void* stream) {
  return rows_call(launch_q4_rows, false, k_rows, v_rows, slot_map, T, H_kv, D, page_size, num_pages, const_cast<void*>(k_cache),
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
  return decode_call(launch_decode_q4, q, k_cache, v_cache, page_table, page_table_stride, seq_lens, rel_logits, B, q_len,
                     H_q, H_kv, D, page_size, num_pages, R, window, scale, out, lse_out, workspace, workspace_bytes,
                     device_error, stream);
}

size_t inkling_rel_attn_prefill_q4_workspace_size(int32_t B, int32_t max_q_len, int32_t H_kv, int32_t D,
                                                  int32_t window, int32_t max_seq_len) {
  if (B <= 0 || max_q_len <= 0 || H_kv <= 0 || D <= 0) return 0;
  return ExpandedLayout(B, max_q_len, H_kv, D, window, max_seq_len).total;
}

int inkling_rel_attn_prefill_q4(const void* q, const int32_t* cu_seqlens_q, const void* k_cache,
                                const void* v_cache, const int32_t* page_table, int32_t page_table_stride,
                                const int32_t* seq_lens, const float* rel_logits, int32_t B, int32_t T,
                                int32_t max_q_len, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                                int32_t num_pages, int32_t R, int32_t window, float scale, int32_t max_seq_len,
                                void* out, float* lse_out, void* workspace, size_t workspace_bytes,
                                int32_t* device_error, void* stream) {
  return prefill_call(launch_q4_expand, q, cu_seqlens_q, k_cache, v_cache, page_table, page_table_stride, seq_lens,
                      rel_logits, B, T, max_q_len, H_q, H_kv, D, page_size, num_pages, R, window, scale, max_seq_len, out,
                      lse_out, workspace, workspace_bytes, device_error, stream);
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
    case INKLING_PACKED_KV_READ_Q4:
    case INKLING_PACKED_KV_APPEND_Q8:
    case INKLING_PACKED_KV_READ_Q8: {
      if (count != 12) return INKLING_ERR_ARG;
      void *x = ptr(), *y = ptr(), *z = ptr();
      const int32_t T = i32(), H_kv = i32(), D = i32(), page_size = i32(), num_pages = i32();
      void *u = ptr(), *w = ptr();
      int32_t* err = static_cast<int32_t*>(ptr());
      void* stream = ptr();
      if (!fits) return INKLING_ERR_ARG;
      if (call == INKLING_PACKED_KV_APPEND_Q4 || call == INKLING_PACKED_KV_APPEND_Q8) {
        const auto append =
            call == INKLING_PACKED_KV_APPEND_Q4 ? inkling_rel_attn_kv_append_q4 : inkling_rel_attn_kv_append_q8;
        return append(x, y, static_cast<const int64_t*>(z), T, H_kv, D, page_size, num_pages, u, w, err, stream);
      }
      const auto read = call == INKLING_PACKED_KV_READ_Q4 ? inkling_rel_attn_kv_read_q4 : inkling_rel_attn_kv_read_q8;
      return read(static_cast<const int64_t*>(x), y, z, T, H_kv, D, page_size, num_pages, u, w, err, stream);
    }
    case INKLING_PACKED_DECODE_Q4:
    case INKLING_PACKED_DECODE_Q8: {
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
      const auto decode = call == INKLING_PACKED_DECODE_Q4 ? inkling_rel_attn_decode_q4 : inkling_rel_attn_decode_q8;
      return decode(q, k, v, table, stride, seq_lens, rel, B, q_len, H_q, H_kv, D, page_size, num_pages, R, window,
                    scale, out, lse, ws, ws_bytes, err, ptr());
    }
    case INKLING_PACKED_PREFILL_Q4:
    case INKLING_PACKED_PREFILL_Q8: {
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
      const auto prefill =
          call == INKLING_PACKED_PREFILL_Q4 ? inkling_rel_attn_prefill_q4 : inkling_rel_attn_prefill_q8;
      return prefill(q, cu, k, v, table, stride, seq_lens, rel, B, T, max_q_len, H_q, H_kv, D, page_size, num_pages, R,
                     window, scale, max_seq_len, out, lse, ws, ws_bytes, err, ptr());
    }
    case INKLING_PACKED_FORK_PAGES: {
      if (count != 16) return INKLING_ERR_ARG;
      const int32_t *source = ci(), *seq_lens = ci();
      int32_t* table = static_cast<int32_t*>(ptr());
      const int32_t stride = i32();
      int32_t* refs = static_cast<int32_t*>(ptr());
      const int32_t *free_pages = ci(), *free_count = ci();
      const int32_t B = i32(), page_size = i32(), num_pages = i32();
      int32_t* out[5];
      for (int32_t*& o : out) o = static_cast<int32_t*>(ptr());
      if (!fits) return INKLING_ERR_ARG;
      return inkling_rel_attn_fork_pages(source, seq_lens, table, stride, refs, free_pages, free_count, B, page_size,
                                         num_pages, out[0], out[1], out[2], out[3], out[4], ptr());
    }
    case INKLING_PACKED_RELEASE_PAGES: {
      if (count != 14) return INKLING_ERR_ARG;
      const int32_t *seq_lens = ci(), *new_lens = ci(), *table = ci();
      const int32_t stride = i32();
      int32_t *refs = static_cast<int32_t*>(ptr()), *free_pages = static_cast<int32_t*>(ptr());
      const int32_t* free_count = ci();
      const int32_t B = i32(), page_size = i32(), num_pages = i32();
      int32_t* out[3];
      for (int32_t*& o : out) o = static_cast<int32_t*>(ptr());
      if (!fits) return INKLING_ERR_ARG;
      return inkling_rel_attn_release_pages(seq_lens, new_lens, table, stride, refs, free_pages, free_count, B,
                                            page_size, num_pages, out[0], out[1], out[2], ptr());
    }
    case INKLING_PACKED_COMPACT_PAGES: {
      if (count != 14) return INKLING_ERR_ARG;
      const int32_t* seq_lens = ci();
      int32_t* table = static_cast<int32_t*>(ptr());
      const int32_t stride = i32();
      int32_t *refs = static_cast<int32_t*>(ptr()), *free_pages = static_cast<int32_t*>(ptr());
      const int32_t* free_count = ci();
      const int32_t B = i32(), page_size = i32(), num_pages = i32();
      int32_t* out[4];
      for (int32_t*& o : out) o = static_cast<int32_t*>(ptr());
      if (!fits) return INKLING_ERR_ARG;
      return inkling_rel_attn_compact_pages(seq_lens, table, stride, refs, free_pages, free_count, B, page_size,
                                            num_pages, out[0], out[1], out[2], out[3], ptr());
    }
    case INKLING_PACKED_COPY_PAGES: {
      if (count != 10) return INKLING_ERR_ARG;
      void* const* pools = static_cast<void* const*>(ptr());
      const int32_t n_pools = i32();
      const int64_t page_bytes = a[at++];
      const int32_t num_pages = i32();
      const int32_t *src = ci(), *dst = ci();
      const int32_t n = i32();
      const int32_t* moves = ci();
      int32_t* err = static_cast<int32_t*>(ptr());
      if (!fits) return INKLING_ERR_ARG;
      return inkling_rel_attn_copy_pages(pools, n_pools, page_bytes, num_pages, src, dst, n, moves, err, ptr());
    }
  }
  return INKLING_ERR_ARG;
}

}  // extern "C"

// C ABI of the 8-bit cache.  See include/inkling_rel_attn.h for the contracts.
#include <cuda_runtime.h>

#include <cstdint>

#include "api_blocks.h"

using namespace ira;

extern "C" {

int inkling_rel_attn_kv_append_q8(const void* k_new, const void* v_new, const int64_t* slot_map, int32_t T,
                                  int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages, void* k_cache,
                                  void* v_cache, int32_t* device_error, void* stream) {
  return rows_call(launch_q8_rows, true, const_cast<void*>(k_new), const_cast<void*>(v_new), slot_map, T, H_kv, D,
                   page_size, num_pages, k_cache, v_cache, device_error, stream);
}

int inkling_rel_attn_kv_read_q8(const int64_t* slot_map, const void* k_cache, const void* v_cache, int32_t T,
                                int32_t H_kv, int32_t D, int32_t page_size, int32_t num_pages, void* k_rows,
                                void* v_rows, int32_t* device_error, void* stream) {
  return rows_call(launch_q8_rows, false, k_rows, v_rows, slot_map, T, H_kv, D, page_size, num_pages,
                   const_cast<void*>(k_cache), const_cast<void*>(v_cache), device_error, stream);
}

size_t inkling_rel_attn_decode_q8_workspace_size(int32_t B, int32_t q_len, int32_t H_q, int32_t H_kv, int32_t D,
                                                 int32_t num_sms) {
  return inkling_rel_attn_decode_q4_workspace_size(B, q_len, H_q, H_kv, D, num_sms);  // the same division of the work
}

int inkling_rel_attn_decode_q8(const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                               int32_t page_table_stride, const int32_t* seq_lens, const float* rel_logits,
                               int32_t B, int32_t q_len, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                               int32_t num_pages, int32_t R, int32_t window, float scale, void* out,
                               float* lse_out, void* workspace, size_t workspace_bytes, int32_t* device_error,
                               void* stream) {
  return decode_call(launch_decode_q8, q, k_cache, v_cache, page_table, page_table_stride, seq_lens, rel_logits, B, q_len,
                     H_q, H_kv, D, page_size, num_pages, R, window, scale, out, lse_out, workspace, workspace_bytes,
                     device_error, stream);
}

size_t inkling_rel_attn_prefill_q8_workspace_size(int32_t B, int32_t max_q_len, int32_t H_kv, int32_t D,
                                                  int32_t window, int32_t max_seq_len) {
  return inkling_rel_attn_prefill_q4_workspace_size(B, max_q_len, H_kv, D, window, max_seq_len);  // bf16 pages alike
}

int inkling_rel_attn_prefill_q8(const void* q, const int32_t* cu_seqlens_q, const void* k_cache,
                                const void* v_cache, const int32_t* page_table, int32_t page_table_stride,
                                const int32_t* seq_lens, const float* rel_logits, int32_t B, int32_t T,
                                int32_t max_q_len, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                                int32_t num_pages, int32_t R, int32_t window, float scale, int32_t max_seq_len,
                                void* out, float* lse_out, void* workspace, size_t workspace_bytes,
                                int32_t* device_error, void* stream) {
  return prefill_call(launch_q8_expand, q, cu_seqlens_q, k_cache, v_cache, page_table, page_table_stride, seq_lens,
                      rel_logits, B, T, max_q_len, H_q, H_kv, D, page_size, num_pages, R, window, scale, max_seq_len, out,
                      lse_out, workspace, workspace_bytes, device_error, stream);
}

}  // extern "C"

// C ABI of shared pages: argument checks and launches.  See include/inkling_rel_attn.h for the contracts.
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

using namespace ira;

namespace {

int tables_shape(int32_t stride, int32_t B, int32_t page_size, int32_t num_pages) {
  if (B < 0 || B > kTablesMaxBatch) return INKLING_ERR_ARG;
  if (page_size <= 0 || page_size % 16 != 0 || page_size > 256) return INKLING_ERR_ARG;
  if (num_pages <= 0 || num_pages == INT32_MAX || stride <= 0) return INKLING_ERR_ARG;
  if ((int64_t)stride * page_size > INT32_MAX) return INKLING_ERR_ARG;
  return INKLING_OK;
}

}  // namespace

extern "C" {

int inkling_rel_attn_fork_pages(const int32_t* source, const int32_t* seq_lens, int32_t* page_table,
                                int32_t page_table_stride, int32_t* page_refs, const int32_t* free_pages,
                                const int32_t* free_count, int32_t B, int32_t page_size, int32_t num_pages,
                                int32_t* kv_lens, int32_t* copy_src, int32_t* copy_dst, int32_t* free_left,
                                int32_t* device_error, void* stream) {
  const int rc = tables_shape(page_table_stride, B, page_size, num_pages);
  if (rc != INKLING_OK) return rc;
  if (B == 0) return INKLING_OK;
  if (!source || !seq_lens || !page_table || !page_refs || !free_pages || !free_count || !kv_lens || !copy_src ||
      !copy_dst || !free_left)
    return INKLING_ERR_ARG;
  if (!aligned(source, 4) || !aligned(seq_lens, 4) || !aligned(page_table, 4) || !aligned(page_refs, 4) ||
      !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(kv_lens, 4) || !aligned(copy_src, 4) ||
      !aligned(copy_dst, 4) || !aligned(free_left, 4) || !aligned(device_error, 4))
    return INKLING_ERR_ALIGN;
  if (device_info().ok != 1) return INKLING_ERR_DEVICE;
  PagesCall c = {};
  c.source = source;
  c.seq_lens = seq_lens;
  c.page_table = page_table;
  c.pt_stride = page_table_stride;
  c.page_refs = page_refs;
  c.free_pages = const_cast<int32_t*>(free_pages);  // read only
  c.free_count = free_count;
  c.B = B;
  c.P = page_size;
  c.num_pages = num_pages;
  c.kv_lens = kv_lens;
  c.src = copy_src;
  c.dst = copy_dst;
  c.count = free_left;
  c.dev_err = device_error;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_fork_pages(c);
}

int inkling_rel_attn_release_pages(const int32_t* seq_lens, const int32_t* new_lens, const int32_t* page_table,
                                   int32_t page_table_stride, int32_t* page_refs, int32_t* free_pages,
                                   const int32_t* free_count, int32_t B, int32_t page_size, int32_t num_pages,
                                   int32_t* kv_lens, int32_t* free_left, int32_t* device_error, void* stream) {
  const int rc = tables_shape(page_table_stride, B, page_size, num_pages);
  if (rc != INKLING_OK) return rc;
  if ((int64_t)B * page_table_stride > kReleaseMaxEntries) return INKLING_ERR_ARG;
  if (B == 0) return INKLING_OK;
  if (!seq_lens || !new_lens || !page_table || !page_refs || !free_pages || !free_count || !kv_lens || !free_left)
    return INKLING_ERR_ARG;
  if (!aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(page_table, 4) || !aligned(page_refs, 4) ||
      !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(kv_lens, 4) || !aligned(free_left, 4) ||
      !aligned(device_error, 4))
    return INKLING_ERR_ALIGN;
  if (device_info().ok != 1) return INKLING_ERR_DEVICE;
  PagesCall c = {};
  c.seq_lens = seq_lens;
  c.new_lens = new_lens;
  c.page_table = const_cast<int32_t*>(page_table);  // read only
  c.pt_stride = page_table_stride;
  c.page_refs = page_refs;
  c.free_pages = free_pages;
  c.free_count = free_count;
  c.B = B;
  c.P = page_size;
  c.num_pages = num_pages;
  c.kv_lens = kv_lens;
  c.count = free_left;
  c.dev_err = device_error;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_release_pages(c);
}

int inkling_rel_attn_compact_pages(const int32_t* seq_lens, int32_t* page_table, int32_t page_table_stride,
                                   int32_t* page_refs, int32_t* free_pages, const int32_t* free_count, int32_t B,
                                   int32_t page_size, int32_t num_pages, int32_t* move_src, int32_t* move_dst,
                                   int32_t* moves, int32_t* device_error, void* stream) {
  const int rc = tables_shape(page_table_stride, B, page_size, num_pages);
  if (rc != INKLING_OK) return rc;
  if (num_pages > kCompactMaxPages) return INKLING_ERR_ARG;
  if (B > 0 && (!seq_lens || !page_table)) return INKLING_ERR_ARG;
  if (!free_pages || !free_count || !move_src || !move_dst || !moves) return INKLING_ERR_ARG;
  if (!aligned(seq_lens, 4) || !aligned(page_table, 4) || !aligned(page_refs, 4) || !aligned(free_pages, 4) ||
      !aligned(free_count, 4) || !aligned(move_src, 4) || !aligned(move_dst, 4) || !aligned(moves, 4) ||
      !aligned(device_error, 4))
    return INKLING_ERR_ALIGN;
  if (device_info().ok != 1) return INKLING_ERR_DEVICE;
  PagesCall c = {};
  c.seq_lens = seq_lens;
  c.page_table = page_table;
  c.pt_stride = page_table_stride;
  c.page_refs = page_refs;
  c.free_pages = free_pages;
  c.free_count = free_count;
  c.B = B;
  c.P = page_size;
  c.num_pages = num_pages;
  c.src = move_src;
  c.dst = move_dst;
  c.count = moves;
  c.dev_err = device_error;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_compact_pages(c);
}

int inkling_rel_attn_copy_pages(void* const* pools, int32_t n_pools, int64_t page_bytes, int32_t num_pages,
                                const int32_t* src, const int32_t* dst, int32_t n, const int32_t* count,
                                int32_t* device_error, void* stream) {
  if (n_pools < 0 || n < 0 || num_pages <= 0) return INKLING_ERR_ARG;
  if (page_bytes <= 0 || page_bytes % 16 != 0 || page_bytes > INT32_MAX) return INKLING_ERR_ARG;
  if (n_pools == 0 || n == 0) return INKLING_OK;
  if (!pools || !src || !dst) return INKLING_ERR_ARG;
  for (int32_t i = 0; i < n_pools; ++i)
    if (!pools[i]) return INKLING_ERR_ARG;
  for (int32_t i = 0; i < n_pools; ++i)
    if (!aligned(pools[i], 16)) return INKLING_ERR_ALIGN;
  if (!aligned(src, 4) || !aligned(dst, 4) || !aligned(count, 4) || !aligned(device_error, 4)) return INKLING_ERR_ALIGN;
  const DevInfo di = device_info();
  if (di.ok != 1) return INKLING_ERR_DEVICE;
  CopyPagesCall c = {};
  c.pools = pools;
  c.n_pools = n_pools;
  c.page_bytes = page_bytes;
  c.num_pages = num_pages;
  c.src = src;
  c.dst = dst;
  c.n = n;
  c.count = count;
  c.sms = di.sms;
  c.dev_err = device_error;
  c.stream = static_cast<cudaStream_t>(stream);
  return launch_copy_pages(c);
}

}  // extern "C"

// Launchers of the 8-bit cache's and the page pool's calls, and the host
// helper they share (not part of the ABI).
#pragma once

#include <cuda.h>

#include "jsv_internal.cuh"

namespace jsv {

// Tensor map over contiguous rows of 64 or 128 bytes, box {row, box_outer},
// swizzled by the row's width.
bool encode_tensor_map_u8_2d(CUtensorMap *map, const void *base, uint64_t inner, uint64_t outer, uint32_t box_outer);

jsv_kv8_plan attention_kv8_plan(const BatchArgs &a, const jsv_kv8 &c);
size_t attention_kv8_workspace_bytes(const BatchArgs &a, const jsv_kv8 &c);
cudaError_t launch_tree_attention_kv8(const BatchArgs &a, const jsv_kv8 &c, const uint16_t *q,
                                      const uint16_t *k_cache, const uint16_t *v_cache, float scale, uint16_t *out,
                                      void *ws, cudaStream_t st);
cudaError_t launch_kv8_quantize(const BatchArgs &a, const jsv_kv8 &c, const uint16_t *k_cache,
                                const uint16_t *v_cache, const int32_t *from_len, const int32_t *to_len,
                                cudaStream_t st);
size_t pages_workspace_bytes(int num_pages, int rows);
cudaError_t launch_pages_alloc(const jsv_page_pool &pool, int32_t *table, int B, int max_pages, const int32_t *begin,
                               const int32_t *end, bool full_only, void *ws, cudaStream_t st);
cudaError_t launch_pages_fork(const jsv_page_pool &pool, int32_t *table, int B, int max_pages, int n,
                              const int32_t *src, const int32_t *dst, const int32_t *len, bool full_only,
                              int32_t *copy_src, int32_t *copy_dst, void *ws, cudaStream_t st);
cudaError_t launch_pages_trim(const jsv_page_pool &pool, int32_t *table, int B, int max_pages,
                              const int32_t *keep_begin, const int32_t *keep_end, cudaStream_t st);
cudaError_t launch_pages_compact(const jsv_page_pool &pool, const int32_t *table, int B, int max_pages,
                                 int32_t *new_table, int32_t *new_refcount, int32_t *copy_src, int32_t *copy_dst,
                                 int max_copies, int32_t *num_copies, void *ws, cudaStream_t st);
cudaError_t launch_pages_copy(const jsv_page_pool &pool, void *const *buffers, const int64_t *page_bytes,
                              int n_buffers, const int32_t *copy_src, const int32_t *copy_dst, int n,
                              const int32_t *num_copies, cudaStream_t st);

}  // namespace jsv

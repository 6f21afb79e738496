// Internal declarations of the cache write and the eviction.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace onela {

struct CacheWriteParams {
  int B, n, Hkv;
  int row_bytes;  // of one (token, head) row
  int page, pages, row_pages;
  int64_t k_stride, v_stride;  // bytes between tokens
  const void *k, *v;
  void *k_pool, *v_pool;
  const int32_t *table, *start, *counts;
  int32_t *status;
};

struct CacheEvictParams {
  int R, Hkv;
  int row_bytes;
  int page, pages, row_pages, dst_pages, dst_row_pages;
  int keep, recent;
  const void *k_pool, *v_pool;
  void *dst_k, *dst_v;
  const int32_t *table, *lengths, *dst_table;
  int32_t *dst_lengths, *kept;
  const float *mass;
  float *dst_mass;
  int32_t *status;
};

cudaError_t launch_cache_write(const CacheWriteParams &p, cudaStream_t s);
cudaError_t launch_cache_evict(const CacheEvictParams &p, cudaStream_t s);

}  // namespace onela

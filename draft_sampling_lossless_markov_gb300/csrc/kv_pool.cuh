// A paged key/value cache as the kernels see it.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "dspark.h"

namespace dspark {

struct KvPool {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;  // null: bf16
  float* v_scale;
  const int32_t* table;
  int64_t table_ld;
  int32_t n_pages, heads, shift, n_req, max_pages;  // pages of 1 << shift tokens
};

inline KvPool kv_pool(const dspark_kv_cache& c) {
  KvPool p;
  p.k = static_cast<uint8_t*>(c.k);
  p.v = static_cast<uint8_t*>(c.v);
  p.k_scale = c.dtype == DSPARK_E4M3 ? c.k_scale : nullptr;
  p.v_scale = c.dtype == DSPARK_E4M3 ? c.v_scale : nullptr;
  p.table = c.table;
  p.table_ld = c.table_ld;
  p.n_pages = c.n_pages;
  p.heads = c.n_kv_heads;
  p.shift = __builtin_ctz((unsigned)c.page_size);
  p.n_req = c.n_req;
  p.max_pages = c.max_pages;
  return p;
}

// The pool's row of head 0 at position pos of request req (the other heads' follow
// 1 << shift rows apart); -1 for a request, a position or a page out of range.
// Rows of the pool are below 2^30.
__device__ __forceinline__ int32_t pool_row(const KvPool& p, int32_t req, int64_t pos) {
  if (req < 0 || req >= p.n_req || pos < 0 || (pos >> p.shift) >= p.max_pages) return -1;
  const int32_t page = p.table[req * p.table_ld + (pos >> p.shift)];
  if (page < 0 || page >= p.n_pages) return -1;
  return ((page * p.heads) << p.shift) + (int32_t)(pos & ((1 << p.shift) - 1));
}

}  // namespace dspark

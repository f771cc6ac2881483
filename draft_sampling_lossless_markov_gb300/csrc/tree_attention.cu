// Attention of every request's drafted rows over its cached context and the drafted
// rows they descend from, read from the paged cache.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "kv_pool.cuh"
#include "launch.h"
#include "tc_ptx.cuh"

namespace dspark {

namespace {

struct TreeArgs {
  KvPool pool;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const int32_t* offsets;
  const int32_t* base;
  const uint64_t* tree;
  int64_t ldq, ldo;
  int32_t N, q_heads, max_tree;
  float scale;
  WsHeader* hdr;
};

template <bool kCodes>
__device__ __forceinline__ float element(const uint8_t* pool, int64_t at) {
  if (kCodes) return __half2float(__half(__nv_cvt_fp8_to_halfraw(pool[at], __NV_E4M3)));
  return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(pool)[at]);
}

// One warp a row and query head, D / 32 elements of the head a lane, one token at
// a time under a running maximum.
template <int D, bool kCodes>
__global__ void __launch_bounds__(128) k_tree_attention(const TreeArgs a) {
  ptx::launch_dependents();
  ptx::grid_wait();
  constexpr int E = D / 32;
  const int r = blockIdx.x / a.q_heads, h = blockIdx.x % a.q_heads, kv = h / (a.q_heads / a.pool.heads);
  const int lane = threadIdx.x & 31;
  const int32_t lo = a.offsets[r], hi = a.offsets[r + 1], base = a.base[r];
  const int64_t held = (int64_t)base + hi - lo;
  if (lo < 0 || hi < lo || hi > a.N || hi - lo > a.max_tree || base < 0 ||
      held > (int64_t)a.pool.max_pages << a.pool.shift) {
    if (threadIdx.x == 0 && a.hdr) report_error(a.hdr, DSPARK_BAD_INPUT, r);
    return;
  }
  for (int j = threadIdx.x / 32; j < hi - lo; j += 4) {
    const int64_t row = lo + j;
    const uint64_t mask = a.tree ? a.tree[row] : ~0ull >> (63 - j);
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = ldf(a.q + row * a.ldq + h * D + lane + 32 * e), o[e] = 0.f;
    for (int64_t t = 0; t < held; ++t) {
      if (t >= base && !((mask >> (t - base)) & 1)) continue;
      const int32_t p = pool_row(a.pool, r, t);
      if (p < 0) {
        if (lane == 0 && a.hdr) report_error(a.hdr, DSPARK_BAD_INPUT, r);
        continue;
      }
      const int64_t at = (int64_t)p + ((int64_t)kv << a.pool.shift);
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], element<kCodes>(a.pool.k, at * D + lane + 32 * e), s);
      s = warp_sum(s) * a.scale * (kCodes ? a.pool.k_scale[at] : 1.f);
      const float w = kCodes ? a.pool.v_scale[at] : 1.f;
      if (s > m) {
        const float f = __expf(m - s);
        l *= f;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] *= f;
        m = s;
      }
      const float x = __expf(s - m);
      l += x;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(x * w, element<kCodes>(a.pool.v, at * D + lane + 32 * e), o[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) a.out[row * a.ldo + h * D + lane + 32 * e] = __float2bfloat16_rn(l == 0.f ? 0.f : o[e] / l);
  }
}

}  // namespace

size_t tree_attention_ws(int, int, int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_tree_attention(const dspark_tree_attention_args& a, uint8_t* ws, cudaStream_t s) {
  TreeArgs t;
  t.pool = kv_pool(a.cache);
  t.q = static_cast<const __nv_bfloat16*>(a.q);
  t.out = static_cast<__nv_bfloat16*>(a.out);
  t.offsets = a.offsets;
  t.base = a.base;
  t.tree = a.tree;
  t.ldq = a.ldq;
  t.ldo = a.ldo;
  t.N = a.N;
  t.q_heads = a.n_q_heads;
  t.max_tree = a.max_tree;
  t.scale = a.scale;
  t.hdr = reinterpret_cast<WsHeader*>(ws);
  const int64_t grid = (int64_t)a.cache.n_req * a.n_q_heads;
  if (grid > INT32_MAX) return cudaErrorNotSupported;
  const bool codes = a.cache.dtype == DSPARK_E4M3;
  const cudaError_t e =
      launch_overlapped(a.cache.head_dim == 64 ? (codes ? k_tree_attention<64, true> : k_tree_attention<64, false>)
                                               : (codes ? k_tree_attention<128, true> : k_tree_attention<128, false>),
                        (unsigned)grid, 128, 0, 1, s, t);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dspark

// out[m, n] = sum_b a_scale[m, b] w_scale[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
// for e4m3 codes a and w with one scale for each block of 128 columns (and, for
// w, of 128 rows).  64 x 64 tiles on the CUDA cores, fp32 sums per block.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int TB = 64;   // rows and columns of a tile
constexpr int TK = 32;   // columns staged at a time

__device__ __forceinline__ float e4m3(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
  return __half2float(__half(h));
}

template <typename TO>
__device__ __forceinline__ void store_out(TO* p, float v);
template <>
__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename TO>
__global__ void __launch_bounds__(256) k_matmul_simple(const dspark_matmul_fp8_args p, int kb) {
  __shared__ float sa[TK][TB + 1], sw[TK][TB + 1];
  const int M = p.n_rows ? min(p.M, *p.n_rows) : p.M;
  const int m0 = blockIdx.y * TB, n0 = blockIdx.x * TB;
  if (m0 >= M) return;
  const uint8_t* a = static_cast<const uint8_t*>(p.a);
  const uint8_t* w = static_cast<const uint8_t*>(p.w);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int b = 0; b < kb; ++b) {
    float part[4][4] = {};
    for (int k0 = b * DSPARK_FP8_BLOCK; k0 < min(p.K, (b + 1) * DSPARK_FP8_BLOCK); k0 += TK) {
      __syncthreads();
      for (int i = threadIdx.x; i < TB * TK; i += 256) {
        const int r = i / TK, c = i % TK;
        const bool k_in = k0 + c < p.K;
        sa[c][r] = k_in && m0 + r < M ? e4m3(a[(int64_t)(m0 + r) * p.lda + k0 + c]) : 0.f;
        sw[c][r] = k_in && n0 + r < p.N ? e4m3(w[(int64_t)(n0 + r) * p.ldw + k0 + c]) : 0.f;
      }
      __syncthreads();
#pragma unroll 4
      for (int c = 0; c < TK; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sa[c][ty * 4 + i], sw[c][tx * 4 + j], part[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = min(m0 + ty * 4 + i, M - 1);
      const float s = p.a_scale[(int64_t)m * kb + b] * p.w_scale[(int64_t)(n0 / DSPARK_FP8_BLOCK) * kb + b];
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(part[i][j], s, acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < M && n < p.N) store_out(static_cast<TO*>(p.out) + (int64_t)m * p.ldo + n, acc[i][j]);
    }
}

}  // namespace

size_t matmul_fp8_ws(int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_matmul_fp8(const dspark_matmul_fp8_args& a, uint8_t*, cudaStream_t s) {
  const int kb = (a.K + DSPARK_FP8_BLOCK - 1) / DSPARK_FP8_BLOCK;
  const dim3 grid((unsigned)((a.N + TB - 1) / TB), (unsigned)((a.M + TB - 1) / TB));
  if (a.out_dtype == DSPARK_BF16)
    k_matmul_simple<__nv_bfloat16><<<grid, 256, 0, s>>>(a, kb);
  else
    k_matmul_simple<float><<<grid, 256, 0, s>>>(a, kb);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace dspark

// Quantisation to e4m3 codes with one fp32 scale for each block of 128 columns
// (and of 1 or 128 rows):
//     amax = max(|x|, 2^-100), scale = amax / 448, code = e4m3(x * (448 / amax)).
// A block's values stay in registers between the maximum and the conversion,
// so x is read once.  Bounded by memory: 3 (bf16) or 5 (fp32) bytes an element.
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace dspark {

namespace {

constexpr int QT = 256;             // threads
constexpr int QL = 16;              // lanes that share a row's 128 columns, 8 each
constexpr float kAmaxMin = 7.888609052210118e-31f;  // 2^-100: keeps 448 / amax finite

// elements c0 .. c0 + 7 of a row, zero from column K on; vec: one aligned load
template <typename T>
__device__ __forceinline__ void load_cols(const T* row, int c0, int K, bool vec, float (&v)[8]) {
  if (vec && c0 + 8 <= K) {
    load8_stream(row + c0, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c0 + i < K ? to_f32(row[c0 + i]) : 0.f;
  }
}

__device__ __forceinline__ float finite_amax(const float (&v)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = fabsf(v[i]);
    a = fmaxf(a, t < INFINITY ? t : 0.f);
  }
  return a;
}

// the conversion saturates at 448, which only the rounding of amax * (448 / amax)
// can pass; non-finite values become the NaN code
__device__ __forceinline__ void store_codes(uint8_t* row, int c0, int K, bool vec, const float (&v)[8], float inv) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float2 f;
      f.x = v[4 * h + 2 * j] * inv;
      f.y = v[4 * h + 2 * j + 1] * inv;
      if (!(fabsf(f.x) < INFINITY)) f.x = NAN;
      if (!(fabsf(f.y) < INFINITY)) f.y = NAN;
      p |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * j);
    }
    w[h] = p;
  }
  if (vec && c0 + 8 <= K) {
    *reinterpret_cast<uint2*>(row + c0) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < K) row[c0 + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// one row of 128 columns per 16 lanes
template <typename T>
__global__ void __launch_bounds__(QT) k_quant_rows(const T* __restrict__ x, int64_t ldx, uint8_t* __restrict__ codes,
                                                   int64_t ldq, float* __restrict__ scale, int M, int K, int kb,
                                                   bool vec) {
  const int64_t units = (int64_t)M * kb;
  const int64_t u = (int64_t)blockIdx.x * (QT / QL) + threadIdx.x / QL;
  const int l = threadIdx.x % QL;
  const bool live = u < units;
  const int64_t row = live ? u / kb : 0;
  const int b = live ? (int)(u - row * kb) : 0;
  const int c0 = b * DSPARK_FP8_BLOCK + l * 8;
  float v[8];
  load_cols(x + row * ldx, c0, K, vec, v);
  float a = finite_amax(v);
#pragma unroll
  for (int o = QL / 2; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  a = fmaxf(a, kAmaxMin);
  if (!live) return;
  store_codes(codes + row * ldq, c0, K, vec, v, __fdiv_rn(448.f, a));
  if (l == 0) scale[u] = __fdiv_rn(a, 448.f);
}

// one 128 x 128 block per CTA: 16 lanes a row, 8 rows a thread
template <typename T>
__global__ void __launch_bounds__(QT) k_quant_blocks(const T* __restrict__ x, int64_t ldx,
                                                     uint8_t* __restrict__ codes, int64_t ldq,
                                                     float* __restrict__ scale, int M, int K, int kb, bool vec) {
  __shared__ float red[QT / 32];
  const int64_t rb = blockIdx.x / kb;
  const int b = (int)(blockIdx.x - rb * kb);
  const int c0 = b * DSPARK_FP8_BLOCK + (threadIdx.x % QL) * 8;
  const int64_t r0 = rb * DSPARK_FP8_BLOCK + threadIdx.x / QL;
  float v[8][8];
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + i * (QT / QL);
    load_cols(x + r * ldx, c0, r < M ? K : 0, vec, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, finite_amax(v[i]));
  a = warp_max(a);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  a = kAmaxMin;
#pragma unroll
  for (int i = 0; i < QT / 32; ++i) a = fmaxf(a, red[i]);
  const float inv = __fdiv_rn(448.f, a);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + i * (QT / QL);
    if (r < M) store_codes(codes + r * ldq, c0, K, vec, v[i], inv);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = __fdiv_rn(a, 448.f);
}

template <typename T>
void launch_t(const dspark_quant_fp8_args& a, cudaStream_t s) {
  const int kb = (a.K + DSPARK_FP8_BLOCK - 1) / DSPARK_FP8_BLOCK;
  const T* x = static_cast<const T*>(a.x);
  uint8_t* q = static_cast<uint8_t*>(a.codes);
  // 16-byte loads and 8-byte stores when every row allows them
  const bool vec = ((uintptr_t)x % 16) == 0 && (a.ldx * sizeof(T)) % 16 == 0 && ((uintptr_t)q % 8) == 0 &&
                   (a.ldq % 8) == 0;
  if (a.block_rows == 1) {
    const int64_t grid = ((int64_t)a.M * kb + QT / QL - 1) / (QT / QL);
    k_quant_rows<T><<<(unsigned)grid, QT, 0, s>>>(x, a.ldx, q, a.ldq, a.scale, a.M, a.K, kb, vec);
  } else {
    const int64_t grid = (int64_t)((a.M + DSPARK_FP8_BLOCK - 1) / DSPARK_FP8_BLOCK) * kb;
    k_quant_blocks<T><<<(unsigned)grid, QT, 0, s>>>(x, a.ldx, q, a.ldq, a.scale, a.M, a.K, kb, vec);
  }
}

}  // namespace

cudaError_t launch_quant_fp8(const dspark_quant_fp8_args& a, cudaStream_t s) {
  if (a.dtype == DSPARK_BF16)
    launch_t<__nv_bfloat16>(a, s);
  else
    launch_t<float>(a, s);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace dspark

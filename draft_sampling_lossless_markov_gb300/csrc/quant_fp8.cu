// Quantisation to e4m3 codes with one fp32 scale for each block of 128 columns
// (and of 1 or 128 rows):
//     amax = max(|x|, 2^-100), scale = amax / 448, code = e4m3(x * 448 / amax),
// the code that of the exact quotient (quant_codes.cuh).
// A block's elements stay in registers between the maximum and the conversion,
// so x is read once: 3 (bf16) or 5 (fp32) bytes an element, bounded by memory
// as long as the arithmetic stays below some 15 (25) instructions an element.
// 151936 x 2560 in 128 x 128 blocks: 172 us from bf16 and 295 us from fp32 (1.0 and
// 0.97 of the measured copy rate); in rows 240 us (0.72) and 309 us (0.93).
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "quant_codes.cuh"
#include "tc_ptx.cuh"
#include "vec8.cuh"

namespace dspark {

namespace {

constexpr int QT = 256;             // threads
constexpr int QL = 16;              // lanes that share a row's 128 columns, 8 each

// N words from place `shift` (below 4) of w on
template <int N>
__device__ __forceinline__ void shift_words(uint32_t* w, int shift) {
#pragma unroll
  for (int i = 0; i < N + 1; ++i) w[i] = (shift & 2) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = (shift & 1) ? w[i + 1] : w[i];
}
// A matrix and how its rows are read: by vectors where every row begins on 16
// bytes, else by the vectors around the eight elements wherever those lie inside
// the matrix (2048 x 2050 in 128 x 128 blocks: bf16 8.1 us, fp32 6.6; element by
// element 17.5 and 12.1).
template <typename T, bool kVec>
struct Source {
  const T* x;
  const T* end;
};
// elements c0 .. c0 + 7 of a row, zero from column K on
template <typename T, bool kVec>
__device__ __forceinline__ void load_cols(Vec8<T>& v, const Source<T, kVec>& src, const T* row, int c0, int K) {
  constexpr int kVecs = sizeof(T) == 2 ? 2 : 3, kWords = 2 * (int)sizeof(T);  // of the eight elements
  const T* p = row + c0;
  if (c0 + 8 <= K) {
    if (kVec) {
      v.load(p);
      return;
    }
    const uintptr_t a = (uintptr_t)p & ~(uintptr_t)15;
    const uint32_t off = (uint32_t)((uintptr_t)p - a);
    if (a >= (uintptr_t)src.x && a + 16 * kVecs <= (uintptr_t)src.end) {
      uint32_t w[4 * kVecs + 2];
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const uint4 q = load16_once(reinterpret_cast<const void*>(a + 16 * i));
        w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
      }
      w[4 * kVecs] = w[4 * kVecs + 1] = 0;
      if constexpr (sizeof(T) == 2) {
        shift_words<kWords + 1>(w, (int)(off >> 2));
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (off & 2) * 8);
      } else {
        shift_words<kWords>(w, (int)(off >> 2));
      }
      v.set(w);
      return;
    }
  }
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) {
    if constexpr (sizeof(T) == 2) {
      const uint16_t* e = reinterpret_cast<const uint16_t*>(p) + 2 * i;
      const uint32_t lo = c0 + 2 * i < K ? e[0] : 0, hi = c0 + 2 * i + 1 < K ? e[1] : 0;
      w[i] = lo | (hi << 16);
    } else {
      w[i] = c0 + i < K ? reinterpret_cast<const uint32_t*>(p)[i] : 0;
    }
  }
  v.set(w);
}

// the eight codes at columns c0 .. c0 + 7 of a row, those before column K
template <typename T>
__device__ __forceinline__ void store_codes(uint8_t* row, int c0, int K, bool vec, const Vec8<T>& v, float a, float inv,
                                            float rest, bool finite) {
  const uint2 q = codes8(v, a, inv, rest, finite);
  if (vec && c0 + 8 <= K) {
    *reinterpret_cast<uint2*>(row + c0) = q;
  } else {
    const uint32_t w[2] = {q.x, q.y};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c0 + i < K) row[c0 + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// (No __restrict__ in these kernels: their loads must stay behind the wait.)
//
// One block of 128 columns of one row per 16 lanes.  A CTA takes 16 QU blocks
// that follow each other in the scales' order (row by row).  The divisions of a
// group's QU blocks are made by QU of its lanes at once.
template <int QU, typename T, bool kVec>
__global__ void __launch_bounds__(QT, 4) k_quant_rows(const Source<T, kVec> src, int64_t ldx, uint8_t* codes, int64_t ldq,
                                                      float* scale, int64_t blocks, int K, uint32_t kb, bool vec) {
  ptx::launch_dependents();
  ptx::grid_wait();
  constexpr int G = QT / QL;
  const int l = threadIdx.x % QL;
  const int64_t first = (int64_t)blockIdx.x * (G * QU) + threadIdx.x / QL;
  int64_t row = blocks <= UINT32_MAX ? (uint32_t)first / kb : first / kb;
  uint32_t b = (uint32_t)(first - row * kb);
  Vec8<T> v[QU];
  int64_t rows[QU];
  int c0[QU];
#pragma unroll
  for (int u = 0; u < QU; ++u) {
    rows[u] = row;
    c0[u] = (int)b * DSPARK_FP8_BLOCK + l * 8;
    load_cols(v[u], src, src.x + row * ldx, c0[u], first + u * G < blocks ? K : 0);
    b += G;
    if (b >= kb) {
      const uint32_t n = b / kb;
      row += n;
      b -= n * kb;
    }
  }
  // lane u of a group divides for block u
  uint32_t mine = 0, non_finite = 0;
#pragma unroll
  for (int u = 0; u < QU; ++u) {
    uint32_t m = amax_bits(v[u]);
#pragma unroll
    for (int o = QL / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (__any_sync(0xffffffffu, m >= kInfBits)) {
      if (m >= kInfBits) non_finite |= 1u << u;
      m = finite_amax_bits(v[u]);
#pragma unroll
      for (int o = QL / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    if (l == u) mine = m;
  }
  const float a = fmaxf(__uint_as_float(mine), kAmaxMin);
  const float inv = inv_of<T>(a), rest = inv_rest(a, inv);
  if (l < QU && first + l * G < blocks) scale[first + l * G] = __fdiv_rn(a, 448.f);
#pragma unroll
  for (int u = 0; u < QU; ++u) {
    const float au = __shfl_sync(0xffffffffu, a, u, QL), iu = __shfl_sync(0xffffffffu, inv, u, QL);
    const float ru = std::is_same<T, float>::value ? 0.f : __shfl_sync(0xffffffffu, rest, u, QL);
    if (first + u * G < blocks)
      store_codes(codes + rows[u] * ldq, c0[u], K, vec, v[u], au, iu, ru, !((non_finite >> u) & 1u));
  }
}

// One 128 x 128 block per CTA: 16 lanes a row, BR rows a thread, four (fp32) or
// eight: 64 KB are on their way to an SM either way (151936 x 2560 fp32: 290 us,
// with eight 313; bf16: 169 us, with four 213).
template <typename T>
constexpr int block_threads() {
  return std::is_same<T, float>::value ? 512 : 256;
}
template <typename T, bool kVec>
__global__ void __launch_bounds__(block_threads<T>(), 1024 / block_threads<T>())
    k_quant_blocks(const Source<T, kVec> src, int64_t ldx, uint8_t* codes, int64_t ldq, float* scale, int M, int K, int kb, bool vec) {
  constexpr int BT = block_threads<T>(), BR = DSPARK_FP8_BLOCK * QL / BT;
  __shared__ uint32_t red[BT / 32], fin[BT / 32];
  ptx::launch_dependents();
  ptx::grid_wait();
  const int rb = blockIdx.x / kb, b = blockIdx.x - rb * kb;
  const int c0 = b * DSPARK_FP8_BLOCK + (threadIdx.x % QL) * 8;
  const int64_t r0 = (int64_t)rb * DSPARK_FP8_BLOCK + threadIdx.x / QL;
  Vec8<T> v[BR];
#pragma unroll
  for (int i = 0; i < BR; ++i) {
    const int64_t r = r0 + i * (BT / QL);
    load_cols(v[i], src, src.x + r * ldx, c0, r < M ? K : 0);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < BR; ++i) m = max(m, amax_bits(v[i]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  m = red[0];
#pragma unroll
  for (int i = 1; i < BT / 32; ++i) m = max(m, red[i]);
  const bool finite = m < kInfBits;
  if (!finite) {  // the whole CTA
    m = 0;
#pragma unroll
    for (int i = 0; i < BR; ++i) m = max(m, finite_amax_bits(v[i]));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) fin[threadIdx.x >> 5] = m;
    __syncthreads();
    m = fin[0];
#pragma unroll
    for (int i = 1; i < BT / 32; ++i) m = max(m, fin[i]);
  }
  const float a = fmaxf(__uint_as_float(m), kAmaxMin), inv = inv_of<T>(a), rest = inv_rest(a, inv);
#pragma unroll
  for (int i = 0; i < BR; ++i) {
    const int64_t r = r0 + i * (BT / QL);
    if (r < M) store_codes(codes + r * ldq, c0, K, vec, v[i], a, inv, rest, finite);
  }
  if (threadIdx.x == 0) scale[blockIdx.x] = __fdiv_rn(a, 448.f);
}

template <typename T, bool kVec>
cudaError_t launch_t(const dspark_quant_fp8_args& a, cudaStream_t s) {
  const int64_t kb = ((int64_t)a.K + DSPARK_FP8_BLOCK - 1) / DSPARK_FP8_BLOCK;
  const T* x = static_cast<const T*>(a.x);
  uint8_t* q = static_cast<uint8_t*>(a.codes);
  const Source<T, kVec> src{x, x + ((int64_t)a.M - 1) * a.ldx + a.K};
  // 8-byte stores when every row allows them
  const bool vec = ((uintptr_t)q % 8) == 0 && (a.M == 1 || a.ldq % 8 == 0);
  if (a.block_rows == 1) {
    // two blocks of a group at a time where CTAs are few (2048 x 4096 bf16: 7.2
    // against 7.6 us, 64 x 4096 1.9 against 2.5), four where they are many
    // (151936 x 2560 fp32: 303 against 320 us)
    const int64_t blocks = a.M * kb;
    const bool many = blocks >= 1 << 18;
    const int64_t each = QT / QL * (many ? 4 : 2), grid = (blocks + each - 1) / each;
    if (grid > INT32_MAX) return cudaErrorNotSupported;
    return launch_overlapped(many ? k_quant_rows<4, T, kVec> : k_quant_rows<2, T, kVec>, (unsigned)grid, QT, 0, 1, s, src,
                             a.ldx, q, a.ldq, a.scale, blocks, a.K, (uint32_t)kb, vec);
  }
  const int64_t grid = (((int64_t)a.M + DSPARK_FP8_BLOCK - 1) / DSPARK_FP8_BLOCK) * kb;
  if (grid > INT32_MAX) return cudaErrorNotSupported;
  return launch_overlapped(k_quant_blocks<T, kVec>, (unsigned)grid, block_threads<T>(), 0, 1, s, src, a.ldx, q, a.ldq,
                           a.scale, a.M, a.K, (int)kb, vec);
}
template <typename T>
cudaError_t launch_t(const dspark_quant_fp8_args& a, cudaStream_t s) {
  const bool vec = ((uintptr_t)a.x % 16) == 0 && (a.M == 1 || (a.ldx * (int64_t)sizeof(T)) % 16 == 0);
  return vec ? launch_t<T, true>(a, s) : launch_t<T, false>(a, s);
}

}  // namespace

cudaError_t launch_quant_fp8(const dspark_quant_fp8_args& a, cudaStream_t s) {
  const cudaError_t e = a.dtype == DSPARK_BF16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace dspark

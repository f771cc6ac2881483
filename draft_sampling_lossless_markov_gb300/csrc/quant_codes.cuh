// e4m3 codes of eight elements under one block's scale:
//     amax = max(|x|, 2^-100), code = e4m3(x * 448 / amax),
// the code that of the exact quotient (inv_rest, code_between).
//
// The maximum is taken on the bits of |x| (as whole numbers they order like the
// values, with infinities and NaN above all), so a block is known to be finite
// from its maximum alone; only others look at each element.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "tc_ptx.cuh"
#include "vec8.cuh"

namespace dspark {

constexpr float kAmaxMin = 7.888609052210118e-31f;  // 2^-100: keeps 448 / amax finite
constexpr uint32_t kInfBits = 0x7F800000u;

// the bits of the largest |x|, as a float's
__device__ __forceinline__ uint32_t amax_bits(const Vec8<__nv_bfloat16>& v) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t x = __vmaxu2(__vmaxu2(v.a.x & m, v.a.y & m), __vmaxu2(v.a.z & m, v.a.w & m));
  return max(x << 16, x & 0xFFFF0000u);
}
__device__ __forceinline__ uint32_t amax_bits(const Vec8<float>& v) {
  const auto b = [](float f) { return __float_as_uint(f) & 0x7FFFFFFFu; };
  return max(max(max(b(v.a.x), b(v.a.y)), max(b(v.a.z), b(v.a.w))), max(max(b(v.b.x), b(v.b.y)), max(b(v.b.z), b(v.b.w))));
}
template <typename T>
__device__ __forceinline__ uint32_t finite_amax_bits(const Vec8<T>& v) {
  float x[8];
  v.get(x);
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    if (b < kInfBits) a = max(a, b);
  }
  return a;
}

// four quotients to codes; the conversion saturates at 448, which only the
// rounding of amax * (448 / amax) can pass
__device__ __forceinline__ uint32_t codes4(uint64_t q01, uint64_t q23) {
  const float2 a = ptx::unpack2(q01), b = ptx::unpack2(q23);
  return (uint32_t)__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
         ((uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16);
}

// fp32(448 / a); from bf16 the float below it, so that what is left (below) is positive
template <typename T>
__device__ __forceinline__ float inv_of(float a) {
  const float inv = __fdiv_rn(448.f, a);
  return std::is_same<T, float>::value ? inv : __uint_as_float(__float_as_uint(inv) - 1u);
}
// What 448 / a leaves past inv, good to 2^-31 of inv: inv + rest gives a bf16 x its
// quotient in one more FMA (and, of one sign, keeps that of a zero).  x 448 and (middle
// of two codes) a are whole numbers below 2^13 on a common scale, so x 448 / a is such a
// middle or at least 2^-13 of it away: the sum x rest + x inv, rounded once, is the
// middle itself where the quotient is, and on the quotient's side of it elsewhere.
// fp32(448 / a) x alone misses a middle for one code in some thousands; the rest costs
// 2048 x 4096 in rows 6.5 against 6.25 us, 151936 x 2560 240 against 233.
__device__ __forceinline__ float inv_rest(float a, float inv) { return fmaf(-a, inv, 448.f) * (1.f / 448.f) * inv; }

// Which of two neighbouring codes (down the one nearer 0) x * 448 / a rounds to:
// the sign of |x| 448 - middle a, both products as exact sums of two floats.
__device__ __forceinline__ uint32_t code_between(float x, float a, uint32_t down, uint32_t up) {
  const auto value = [](uint32_t c) { return __half2float(__half(__nv_cvt_fp8_to_halfraw((uint8_t)(c & 0x7Fu), __NV_E4M3))); };
  const float middle = 0.5f * (value(down) + value(up));
  const float unit = a > 1.f ? 5.421010862427522e-20f : 18446744073709551616.f;  // 2^-64 or 2^64: nothing over- or underflows
  const float xs = fabsf(x) * unit, as = a * unit;
  const float p = xs * 448.f, q = middle * as;
  const float d = (p - q) + (fmaf(xs, 448.f, -p) - fmaf(middle, as, -q));
  return d > 0.f || (d == 0.f && !(up & 1u)) ? up : down;
}

// a: the block's amax, inv: 448 / a, rest: inv_rest (bf16).  Non-finite elements become the NaN code.
template <typename T>
__device__ __forceinline__ uint2 codes8(const Vec8<T>& v, float a, float inv, float rest, bool finite) {
  float x[8];
  v.get(x);
  if (!finite) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((__float_as_uint(x[i]) & 0x7FFFFFFFu) >= kInfBits) x[i] = NAN;
  }
  uint32_t w[2];
  if constexpr (std::is_same<T, float>::value) {
    // the two roundings move a product by less than 2^-23 of it: where both
    // ends of +-2^-22 give one code, that is the exact quotient's
    const float up = inv * (1.f + 2.384185791015625e-07f), down = inv * (1.f - 2.384185791015625e-07f);
    const uint64_t up2 = ptx::pack2(up, up), down2 = ptx::pack2(down, down);
    uint32_t other[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t x01 = ptx::pack2(x[4 * h], x[4 * h + 1]), x23 = ptx::pack2(x[4 * h + 2], x[4 * h + 3]);
      w[h] = codes4(ptx::mul2(x01, up2), ptx::mul2(x23, up2));
      other[h] = codes4(ptx::mul2(x01, down2), ptx::mul2(x23, down2));
    }
    if ((w[0] ^ other[0]) | (w[1] ^ other[1])) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int sh = 8 * (i & 3);
        const uint32_t cu = (w[i >> 2] >> sh) & 255u, cd = (other[i >> 2] >> sh) & 255u;
        if (cu != cd) w[i >> 2] = (w[i >> 2] & ~(255u << sh)) | (code_between(x[i], a, cd, cu) << sh);
      }
    }
  } else {
    const uint64_t inv2 = ptx::pack2(inv, inv), rest2 = ptx::pack2(rest, rest);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint64_t x01 = ptx::pack2(x[4 * h], x[4 * h + 1]), x23 = ptx::pack2(x[4 * h + 2], x[4 * h + 3]);
      w[h] = codes4(ptx::fma2(x01, inv2, ptx::mul2(x01, rest2)), ptx::fma2(x23, inv2, ptx::mul2(x23, rest2)));
    }
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace dspark

// Eight consecutive elements of a row as a thread holds them (bf16 or fp32), and
// the bf16-pair operations the row kernels use.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "tc_ptx.cuh"

namespace dspark {

constexpr float kLowest = -3.402823466e+38f;

// 16 bytes that are read once.  Volatile: the load stays behind a wait in front of it.
__device__ __forceinline__ uint4 load16_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// bf16 pairs
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 0xFFFF in each half where a > b
__device__ __forceinline__ uint32_t gt_bf16x2(uint32_t a, uint32_t b) {
  return __hgt2_mask(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// the largest value of the type below x (finite or +inf)
__device__ __forceinline__ uint32_t bits_below(uint32_t b, uint32_t ulp) {
  return (b & 0x80000000u) ? b + ulp : b == 0 ? 0x80000000u + ulp : b - ulp;
}
template <typename T>
__device__ __forceinline__ float value_below(float x) {
  return __uint_as_float(bits_below(__float_as_uint(x + 0.f), std::is_same<T, float>::value ? 1u : 0x10000u));
}

// the lowest value of the type
template <typename T>
__device__ __forceinline__ float lowest() {
  return std::is_same<T, float>::value ? kLowest : __uint_as_float(0xFF7F0000u);
}

// eight elements as loaded
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 a;
  static constexpr int kAlign = 16;  // bytes, for load_aligned and store
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = load16_once(p); }
  __device__ __forceinline__ void load_aligned(const __nv_bfloat16* p) { load(p); }
  __device__ __forceinline__ void set(const uint32_t* w) { a = make_uint4(w[0], w[1], w[2], w[3]); }
  __device__ __forceinline__ void load_shared(const uint8_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void fill_neg_inf() { a = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u); }
  // -inf where the bit is clear
  __device__ __forceinline__ void mask(uint32_t bits) {
    const uint32_t r = bits | (bits << 15);  // bit 2 i, and bit 2 i + 1 sixteen places above it
    uint32_t* w[4] = {&a.x, &a.y, &a.z, &a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // the two bits at the top of bytes 0 and 2, each spread over two bytes
      uint32_t keep;
      asm("prmt.b32 %0, %1, 0, 0xAA88;" : "=r"(keep) : "r"(r << (7 - 2 * i)));
      *w[i] = (*w[i] & keep) | (0xFF80FF80u & ~keep);
    }
  }
  // element e as a bit place of reach(): word e / 2 in bits 0-3, half e % 2 in bit 4
  static __device__ __forceinline__ int element(int place) { return 2 * (place & 3) + (place >> 4); }
  __device__ __forceinline__ float at(int place) const {
    const uint32_t lo = (place & 1) ? a.y : a.x, hi = (place & 1) ? a.w : a.z, w = (place & 2) ? hi : lo;
    return (place & 16) ? bf_hi(w) : bf_lo(w);
  }
  // a bit for each element at or above x, a bf16 value above -inf
  __device__ __forceinline__ uint32_t reach(float x) const {
    const uint32_t below2 = (bits_below(__float_as_uint(x + 0.f), 0x10000u) >> 16) * 0x10001u;
    return (gt_bf16x2(a.x, below2) & 0x00010001u) | (gt_bf16x2(a.y, below2) & 0x00020002u) |
           (gt_bf16x2(a.z, below2) & 0x00040004u) | (gt_bf16x2(a.w, below2) & 0x00080008u);
  }
  // the largest element (NaN is passed over), of each half and of both
  __device__ __forceinline__ uint32_t max2() const { return max_bf16x2(max_bf16x2(a.x, a.y), max_bf16x2(a.z, a.w)); }
  __device__ __forceinline__ float max() const {
    const uint32_t x = max2();
    return fmaxf(bf_lo(x), bf_hi(x));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&d)[8], bool vec) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(d[2 * i], d[2 * i + 1]);
    if (vec) {
      __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(h));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[2 * i] = h[i].x;
        p[2 * i + 1] = h[i].y;
      }
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  static constexpr int kAlign = 32;
  __device__ __forceinline__ void set(const uint32_t* w) {
    a = make_float4(__uint_as_float(w[0]), __uint_as_float(w[1]), __uint_as_float(w[2]), __uint_as_float(w[3]));
    b = make_float4(__uint_as_float(w[4]), __uint_as_float(w[5]), __uint_as_float(w[6]), __uint_as_float(w[7]));
  }
  __device__ __forceinline__ void load_aligned(const float* p) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(a.x), "=f"(a.y), "=f"(a.z), "=f"(a.w), "=f"(b.x), "=f"(b.y), "=f"(b.z), "=f"(b.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void load(const float* p) {
    const uint4 u = load16_once(p), w = load16_once(p + 4);
    a = make_float4(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w));
    b = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
  }
  __device__ __forceinline__ void load_shared(const uint8_t* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 16);
  }
  __device__ __forceinline__ void fill_neg_inf() { a = b = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ void mask(uint32_t bits) {
    float* x[8] = {&a.x, &a.y, &a.z, &a.w, &b.x, &b.y, &b.z, &b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!((bits >> e) & 1u)) *x[e] = -INFINITY;
  }
  static __device__ __forceinline__ int element(int place) { return place; }
  __device__ __forceinline__ float at(int place) const {
    const float4 q = (place & 4) ? b : a;
    const float lo = (place & 1) ? q.y : q.x, hi = (place & 1) ? q.w : q.z;
    return (place & 2) ? hi : lo;
  }
  // a bit for each element at or above x
  __device__ __forceinline__ uint32_t reach(float x) const {
    return (a.x >= x) | (a.y >= x) << 1 | (a.z >= x) << 2 | (a.w >= x) << 3 | (b.x >= x) << 4 | (b.y >= x) << 5 |
           (b.z >= x) << 6 | (b.w >= x) << 7;
  }
  __device__ __forceinline__ float max() const {
    return fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&d)[8], bool vec) {
    if (vec) {
      asm volatile("st.global.v8.f32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"f"(d[0]), "f"(d[1]), "f"(d[2]),
                   "f"(d[3]), "f"(d[4]), "f"(d[5]), "f"(d[6]), "f"(d[7]), "l"(p)
                   : "memory");
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = d[i];
    }
  }
};

}  // namespace dspark

// The paged key/value cache: rows written to it as e4m3 codes with one fp32 scale
// for each row and head (or bf16), read back, and moved within it.
//
// All three are bounded by memory: a bf16 row and head of 128 is 256 bytes read and
// 132 written.  A row and head is the unit, D / 16 lanes with two vectors of 8 elements
// each (16 bytes of bf16; one vector a lane and divisions to find its place took a write
// 119 us for what now takes 70), so its maximum is two or three shuffles and a warp's accesses
// run over neighbouring heads of one row.  The places of a CTA's rows are looked up once,
// while the first elements are on their way.
//     65536 rows x 8 heads x 128, k and v, bf16 to e4m3   70 us, 0.86 of the measured copy rate
//     the same read back                                  64 us, 0.94
//     2000 requests' paths of up to 16 rows, bf16         30 us, 0.69
// Of the write's issue slots 67 % are taken; a move waits for its chain of look-ups (count and
// path, table, row), which eight CTAs an SM hide in part.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv_pool.cuh"
#include "launch.h"
#include "quant_codes.cuh"
#include "tc_ptx.cuh"
#include "vec8.cuh"

namespace dspark {

namespace {

constexpr int KT = 256;  // threads
constexpr int kSms = 152;
// Units a group of lanes has on their way at a time, and such passes a CTA makes at most.  65536 rows
// written with 1, 2 and 4 units: 70, 75 and 72 us (registers cost CTAs); read: 73, 64 and 63 us, and the
// smallest reads 4.1, 4.6 and 5.2 us.
constexpr int kWriteUnits = 1, kWritePasses = 4;
constexpr int kReadUnits = 2, kReadPasses = 2;

struct CacheRows {
  KvPool pool;
  const int32_t* mark_req;
  const int32_t* mark_pos;
  const int32_t* base;
  const int32_t* n_rows;
  int32_t N, per;     // rows, rows a CTA
  uint64_t row_inv;   // u / (2 heads) is u row_inv >> 32 for a unit u of a CTA (below 2^16, or of its only row)
  int64_t ldk, ldv;
  WsHeader* hdr;
};

__device__ __forceinline__ int32_t count_rows(const CacheRows& c) {
  return c.n_rows ? max(0, min(c.N, *c.n_rows)) : c.N;
}

// the pool's row of row i, -1 to skip it
__device__ __forceinline__ int32_t place_of(const CacheRows& c, int32_t i) {
  const int32_t req = c.mark_req[i];
  if (req == -1) return -1;
  int32_t row = -1;
  if (req >= 0 && req < c.pool.n_req) row = pool_row(c.pool, req, (int64_t)(c.base ? c.base[req] : 0) + c.mark_pos[i]);
  if (row < 0 && c.hdr) report_error(c.hdr, DSPARK_BAD_INPUT, i);
  return row;
}

// Units of a CTA's rows: row, then k or v, then head.
struct Unit {
  int32_t row, head;  // row within the CTA
  bool v;
};
__device__ __forceinline__ Unit unit_at(const CacheRows& c, int u) {
  Unit x;
  x.row = (int)((uint32_t)u * c.row_inv >> 32);
  const int rest = u - x.row * 2 * c.pool.heads;
  x.v = rest >= c.pool.heads;
  x.head = x.v ? rest - c.pool.heads : rest;
  return x;
}

template <int D, typename T, bool kCodes>
__global__ void __launch_bounds__(KT) k_cache_write(const CacheRows c, const T* k, const T* v) {
  ptx::launch_dependents();
  ptx::grid_wait();
  constexpr int LV = D / 16, G = KT / LV, KU = kWriteUnits;  // lanes of a unit, groups of them
  __shared__ int32_t place[KT];
  const int32_t n = count_rows(c), row0 = blockIdx.x * c.per;
  if (row0 >= n) return;
  const int rows = min(c.per, n - row0), units = rows * 2 * c.pool.heads;
  if (threadIdx.x < rows) place[threadIdx.x] = place_of(c, row0 + threadIdx.x);
  const int g = threadIdx.x / LV, l = threadIdx.x % LV;
#pragma unroll 1
  for (int u0 = 0; u0 < units; u0 += G * KU) {
    Vec8<T> x[KU][2];
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      const int u = u0 + i * G + g;
      const Unit at = unit_at(c, min(u, units - 1));
      const T* src = (at.v ? v + (row0 + at.row) * c.ldv : k + (row0 + at.row) * c.ldk) + (int64_t)at.head * D + l * 8;
      x[i][0].load(src);
      x[i][1].load(src + D / 2);
    }
    if (u0 == 0) __syncthreads();  // the places
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      const int u = u0 + i * G + g;
      const Unit at = unit_at(c, min(u, units - 1));
      const int32_t p = place[at.row];
      const bool live = u < units && p >= 0;
      const int64_t row = (int64_t)p + ((int64_t)at.head << c.pool.shift);
      if constexpr (kCodes) {
        uint32_t m = max(amax_bits(x[i][0]), amax_bits(x[i][1]));
#pragma unroll
        for (int o = LV / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const bool finite = m < kInfBits;
        if (__any_sync(0xffffffffu, !finite)) {
          uint32_t f = max(finite_amax_bits(x[i][0]), finite_amax_bits(x[i][1]));
#pragma unroll
          for (int o = LV / 2; o > 0; o >>= 1) f = max(f, __shfl_xor_sync(0xffffffffu, f, o));
          if (!finite) m = f;
        }
        const float a = fmaxf(__uint_as_float(m), kAmaxMin), inv = inv_of<T>(a), rest = inv_rest(a, inv);
        const uint2 q0 = codes8(x[i][0], a, inv, rest, finite), q1 = codes8(x[i][1], a, inv, rest, finite);
        if (live) {
          uint8_t* dst = (at.v ? c.pool.v : c.pool.k) + row * D + l * 8;
          *reinterpret_cast<uint2*>(dst) = q0;
          *reinterpret_cast<uint2*>(dst + D / 2) = q1;
          if (l == 0) (at.v ? c.pool.v_scale : c.pool.k_scale)[row] = __fdiv_rn(a, 448.f);
        }
      } else if (live) {
        __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(at.v ? c.pool.v : c.pool.k) + row * D + l * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(dst + h * (D / 2)) = x[i][h].a;
          } else {
            float f[8];
            x[i][h].get(f);
            Vec8<__nv_bfloat16>::store(dst + h * (D / 2), f, true);
          }
        }
      }
    }
  }
}

template <int D, typename T, bool kCodes>
__global__ void __launch_bounds__(KT) k_cache_read(const CacheRows c, T* k, T* v) {
  ptx::launch_dependents();
  ptx::grid_wait();
  constexpr int LV = D / 16, G = KT / LV, KU = kReadUnits;
  __shared__ int32_t place[KT];
  const int32_t n = count_rows(c), row0 = blockIdx.x * c.per;
  if (row0 >= n) return;
  const int rows = min(c.per, n - row0), units = rows * 2 * c.pool.heads;
  if (threadIdx.x < rows) place[threadIdx.x] = place_of(c, row0 + threadIdx.x);
  __syncthreads();
  const int g = threadIdx.x / LV, l = threadIdx.x % LV;
#pragma unroll 1
  for (int u0 = 0; u0 < units; u0 += G * KU) {
    uint4 x[KU][2];
    float scale[KU];
    T* dst[KU];
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      const int u = u0 + i * G + g;
      const Unit at = unit_at(c, min(u, units - 1));
      const int32_t p = place[at.row];
      dst[i] = nullptr;
      if (u >= units || p < 0) continue;
      dst[i] = (at.v ? v + (row0 + at.row) * c.ldv : k + (row0 + at.row) * c.ldk) + (int64_t)at.head * D + l * 8;
      const int64_t row = (int64_t)p + ((int64_t)at.head << c.pool.shift);
      const uint8_t* pool = at.v ? c.pool.v : c.pool.k;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (kCodes) {
          const uint2 q = *reinterpret_cast<const uint2*>(pool + row * D + h * (D / 2) + l * 8);
          x[i][h].x = q.x, x[i][h].y = q.y;
        } else {
          x[i][h] = *reinterpret_cast<const uint4*>(pool + (row * D + h * (D / 2) + l * 8) * 2);
        }
      }
      if constexpr (kCodes) scale[i] = (at.v ? c.pool.v_scale : c.pool.k_scale)[row];
    }
#pragma unroll
    for (int i = 0; i < KU; ++i) {
      if (!dst[i]) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float f[8];
        if constexpr (kCodes) {
          const uint32_t w[2] = {x[i][h].x, x[i][h].y};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[j >> 1] >> (16 * (j & 1))), __NV_E4M3)));
            f[2 * j] = y.x * scale[i];
            f[2 * j + 1] = y.y * scale[i];
          }
        } else {
          Vec8<__nv_bfloat16> y;
          y.a = x[i][h];
          y.get(f);
        }
        T* to = dst[i] + h * (D / 2);
        if constexpr (sizeof(T) == 2) {
          Vec8<__nv_bfloat16>::store(to, f, true);
        } else {  // rows begin on 16 bytes, not on 32
          __stcs(reinterpret_cast<float4*>(to), make_float4(f[0], f[1], f[2], f[3]));
          __stcs(reinterpret_cast<float4*>(to) + 1, make_float4(f[4], f[5], f[6], f[7]));
        }
      }
    }
  }
}

// A CTA holds whole units (request, k or v of a head): all of a unit's rows are in
// registers before the first is written, so a path may read what it writes.
// 16-byte vectors a thread, at most (2000 requests with 2, 4 and 8: 43, 30 and 32 us)
constexpr int MV = 4;
struct MoveArgs {
  KvPool pool;
  const int32_t* base;
  const int32_t* path;
  int64_t path_ld;
  const int32_t* n_path;
  int32_t cols, units;  // path columns, units a CTA (at most KT)
  uint64_t cols_inv;    // i / cols is i cols_inv >> 32 for i below 2^16
  WsHeader* hdr;
};
struct MoveUnit {
  uint8_t* rows;  // of the unit's head
  float* scales;
  int32_t entry;  // of node 0 of its path
};

template <int kRowBytes>
__global__ void __launch_bounds__(KT, 8) k_cache_move(const MoveArgs m) {
  ptx::launch_dependents();
  ptx::grid_wait();
  constexpr int VR = kRowBytes / 16;  // vectors a row
  const KvPool& pool = m.pool;
  __shared__ int32_t from[KT], to[KT];  // of (request of the CTA, node of its path)
  __shared__ MoveUnit at_unit[KT];
  const int t = threadIdx.x, per_req = 2 * pool.heads;
  const int64_t all = (int64_t)pool.n_req * per_req, u0 = (int64_t)blockIdx.x * m.units;
  const int units = (int)min((int64_t)m.units, all - u0);
  const int32_t req0 = (int32_t)(u0 / per_req);
  const int first = (int)(u0 - (int64_t)req0 * per_req);  // of the CTA's units in request req0
  const int entries = ((first + units - 1) / per_req + 1) * m.cols;
  if (t < entries) {
    const int of = (int)((uint32_t)t * m.cols_inv >> 32), i = t - of * m.cols;
    const int32_t r = req0 + of;
    int32_t a = -1, b = -1;
    const int32_t n = m.n_path[r], base = m.base[r], node = m.path[r * m.path_ld + i];
    bool bad = n < 0 || n > m.cols || base < 0;
    if (!bad && i < n) {
      bad = node < 0 || node >= DSPARK_MAX_TREE;
      if (!bad) {
        a = pool_row(pool, r, (int64_t)base + node);
        b = pool_row(pool, r, (int64_t)base + i);
        bad = a < 0 || b < 0;
        if (bad) a = -1;
      }
    }
    if (bad && m.hdr) report_error(m.hdr, DSPARK_BAD_INPUT, r);
    from[t] = a == b ? -1 : a;  // a node that stays
    to[t] = b;
  }
  if (t < units) {
    const int of = (first + t) / per_req, rest = first + t - of * per_req;
    const int64_t head = (int64_t)(rest < pool.heads ? rest : rest - pool.heads) << pool.shift;
    at_unit[t].rows = (rest < pool.heads ? pool.k : pool.v) + head * kRowBytes;
    at_unit[t].scales = pool.k_scale ? (rest < pool.heads ? pool.k_scale : pool.v_scale) + head : nullptr;
    at_unit[t].entry = of * m.cols;
  }
  __syncthreads();
  const int rows = units * m.cols;  // (unit, node)
  uint4 x[MV];
  uint8_t* dst[MV];
#pragma unroll
  for (int i = 0; i < MV; ++i) {
    const int row = (t + i * KT) / VR;
    dst[i] = nullptr;
    if (row >= rows) continue;
    const int of = (int)((uint32_t)row * m.cols_inv >> 32);
    const MoveUnit& u = at_unit[of];
    const int e = u.entry + row - of * m.cols;
    const int32_t src = from[e];
    if (src < 0) continue;
    uint8_t* lane = u.rows + t % VR * 16;
    x[i] = *reinterpret_cast<const uint4*>(lane + (int64_t)src * kRowBytes);
    dst[i] = lane + (int64_t)to[e] * kRowBytes;
  }
  // the scales: one each a thread
  constexpr int SV = MV / VR > 0 ? MV / VR : 1;
  float scale[SV];
  float* scale_to[SV];
#pragma unroll
  for (int i = 0; i < SV; ++i) {
    const int row = t + i * KT;
    scale_to[i] = nullptr;
    if (!pool.k_scale || row >= rows) continue;
    const int of = (int)((uint32_t)row * m.cols_inv >> 32);
    const MoveUnit& u = at_unit[of];
    const int e = u.entry + row - of * m.cols;
    if (from[e] < 0) continue;
    scale[i] = u.scales[from[e]];
    scale_to[i] = u.scales + to[e];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MV; ++i)
    if (dst[i]) *reinterpret_cast<uint4*>(dst[i]) = x[i];
#pragma unroll
  for (int i = 0; i < SV; ++i)
    if (scale_to[i]) *scale_to[i] = scale[i];
}

// rows a CTA: as many as give every group of lanes KU units, up to `passes` times while
// each SM has eight CTAs; one at least
int rows_per_cta(int64_t N, int heads, int D, int KU, int passes) {
  const int pass = KT / (D / 16) * KU;
  const int64_t each = N * 2 * heads / ((int64_t)8 * kSms * pass);
  const int units = pass * (int)std::max<int64_t>(1, std::min<int64_t>(passes, each));
  return std::max(1, std::min(KT, units / (2 * heads)));
}

template <typename A>
CacheRows cache_rows(const A& a, int KU, int passes, WsHeader* hdr) {
  CacheRows c;
  c.pool = kv_pool(a.cache);
  c.mark_req = a.mark_req;
  c.mark_pos = a.mark_pos;
  c.base = a.base;
  c.n_rows = a.n_rows;
  c.N = a.N;
  c.per = rows_per_cta(a.N, c.pool.heads, a.cache.head_dim, KU, passes);
  c.row_inv = c.per == 1 ? 0 : ((1ull << 32) + 2 * c.pool.heads - 1) / (2 * c.pool.heads);
  c.ldk = a.ldk;
  c.ldv = a.ldv;
  c.hdr = hdr;
  return c;
}

template <int D, typename T>
cudaError_t write_t(const dspark_cache_write_args& a, WsHeader* hdr, cudaStream_t s) {
  const CacheRows c = cache_rows(a, kWriteUnits, kWritePasses, hdr);
  const unsigned grid = (unsigned)((a.N + c.per - 1) / c.per);
  const T *k = static_cast<const T*>(a.k), *v = static_cast<const T*>(a.v);
  return launch_overlapped(a.cache.dtype == DSPARK_E4M3 ? k_cache_write<D, T, true> : k_cache_write<D, T, false>, grid, KT, 0,
                           1, s, c, k, v);
}
template <int D, typename T>
cudaError_t read_t(const dspark_cache_read_args& a, WsHeader* hdr, cudaStream_t s) {
  const CacheRows c = cache_rows(a, kReadUnits, kReadPasses, hdr);
  const unsigned grid = (unsigned)((a.N + c.per - 1) / c.per);
  T *k = static_cast<T*>(a.k), *v = static_cast<T*>(a.v);
  return launch_overlapped(a.cache.dtype == DSPARK_E4M3 ? k_cache_read<D, T, true> : k_cache_read<D, T, false>, grid, KT, 0, 1,
                           s, c, k, v);
}

cudaError_t counted(cudaError_t e) {
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_cache_write(const dspark_cache_write_args& a, WsHeader* hdr, cudaStream_t s) {
  const bool bf = a.dtype == DSPARK_BF16;
  if (a.cache.head_dim == 64)
    return counted(bf ? write_t<64, __nv_bfloat16>(a, hdr, s) : write_t<64, float>(a, hdr, s));
  return counted(bf ? write_t<128, __nv_bfloat16>(a, hdr, s) : write_t<128, float>(a, hdr, s));
}

cudaError_t launch_cache_read(const dspark_cache_read_args& a, WsHeader* hdr, cudaStream_t s) {
  const bool bf = a.dtype == DSPARK_BF16;
  if (a.cache.head_dim == 64)
    return counted(bf ? read_t<64, __nv_bfloat16>(a, hdr, s) : read_t<64, float>(a, hdr, s));
  return counted(bf ? read_t<128, __nv_bfloat16>(a, hdr, s) : read_t<128, float>(a, hdr, s));
}

cudaError_t launch_cache_move(const dspark_cache_move_args& a, WsHeader* hdr, cudaStream_t s) {
  MoveArgs m;
  m.pool = kv_pool(a.cache);
  m.base = a.base;
  m.path = a.path;
  m.path_ld = a.path_ld;
  m.n_path = a.n_path;
  m.cols = a.path_cols;
  m.hdr = hdr;
  const int row = a.cache.head_dim * (a.cache.dtype == DSPARK_E4M3 ? 1 : 2);
  m.cols_inv = ((1ull << 32) + a.path_cols - 1) / a.path_cols;
  // units whose vectors fill the CTA's registers and whose requests' paths its threads, fewer
  // where that would leave an SM less than four CTAs
  const int64_t all = (int64_t)m.pool.n_req * 2 * m.pool.heads;
  m.units = std::min(KT, std::max(1, KT * MV / (a.path_cols * (row / 16))));
  m.units = (int)std::max<int64_t>(1, std::min<int64_t>(m.units, all / ((int64_t)4 * kSms)));
  while (m.units > 1 && ((m.units + 2 * m.pool.heads - 2) / (2 * m.pool.heads) + 1) * m.cols > KT) --m.units;
  const int64_t grid = (all + m.units - 1) / m.units;
  if (grid > INT32_MAX) return cudaErrorNotSupported;
  return counted(launch_overlapped(row == 64 ? k_cache_move<64> : row == 128 ? k_cache_move<128> : k_cache_move<256>,
                                   (unsigned)grid, KT, 0, 1, s, m));
}

}  // namespace dspark

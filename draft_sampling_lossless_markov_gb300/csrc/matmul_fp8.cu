// out[m, n] = sum_b a_scale[m, b] w_scale[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
// for e4m3 codes a [M, K] and w [N, K], one scale for each block of 128 columns
// (and, for w, of 128 rows).
//
// A block's sum comes from the fp8 tensor cores (tcgen05 kind::f8f6f4, fp32
// accumulators in TMEM, four instructions of 32 columns); it then has to be
// scaled before it is added to the next block's, so the accumulator is read
// out once per block: acc += part * (a_scale w_scale) in fp32 registers, while the
// tensor cores fill the next TMEM buffer.
//
// Two kernels, chosen by M:
//   k_fp8_wide    rows of a on the TMEM lanes.  A CTA pair (cta_group::2) makes a
//                 256 x BN tile: each CTA stages its 128 rows of a and half of the
//                 BN rows of w.  A lane's scale is one register and a tile column
//                 block's scale is uniform, so the promotion is one packed FMA for
//                 two elements.
//   k_fp8_narrow  rows of w on the lanes, up to 64 rows of a on the columns:
//                 a weight-bandwidth kernel.  A cluster of S CTAs splits the
//                 blocks of K and adds its parts through distributed shared memory
//                 in rank order (no atomics: equal calls give equal bits).
//
// Every wait is bounded; one that gives up reports DSPARK_TIMEOUT.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace dspark {

namespace {

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr int kKb = DSPARK_FP8_BLOCK;  // columns of a block: one 128-byte swizzled row of shared memory

struct MmParams {
  int M, N, kb;
  const float* a_scale;  // [M, kb]
  const float* w_scale;  // [ceil(N / 128), kb]
  void* out;
  int64_t ldo;
  const int32_t* n_rows;
  int tma_out;  // the output's rows are 16-byte aligned: stores by TMA
  WsHeader* hdr;
};

__device__ __forceinline__ int rows_of(const MmParams& p) {
  return p.n_rows ? max(0, min(p.M, *p.n_rows)) : p.M;
}

__device__ __forceinline__ void store_out(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// ---------------------------------------------------------------------------
// wide: 256 x BN tiles by CTA pairs
// ---------------------------------------------------------------------------
constexpr int kEpiWarps = 8;
constexpr int kWideThreads = 32 * (kEpiWarps + 2);

template <int BN>
struct Wide {
  static constexpr uint32_t kA = 128 * kKb;         // bytes of a per CTA and stage
  static constexpr uint32_t kB = BN / 2 * kKb;      // bytes of w per CTA and stage
  static constexpr uint32_t kStage = kA + kB;
  static constexpr uint32_t kStg = kEpiWarps * 8192;  // output staging: two 4 KB buffers a warp
  static constexpr int kStages = BN == 256 ? 5 : 6;
  static constexpr int kBufs = 512 / BN;            // TMEM accumulators
  static constexpr uint32_t kSmem = kStages * kStage + kStg + 1024;
};

template <int BN, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWideThreads, 1)
    k_fp8_wide(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmO, const MmParams p) {
  using W = Wide<BN>;
  constexpr int NS = W::kStages, NB = W::kBufs;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the same offset in both CTAs: the descriptors of a pair name one place for both
  uint8_t* sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[NS], empty[NS], tfull[NB], tempty[NB];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s, never_s;
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    ptx::fence_mbar_init();
    abort_s = never_s = 0;
    ptx::prefetch_map(&tmA);
    ptx::prefetch_map(&tmW);
    ptx::prefetch_map(&tmO);
  }
  if (warp == kEpiWarps + 1) {
    ptx::tmem_alloc_pair(&tmem_slot, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  auto fail = [&](int what) {
    if (p.hdr) report_error(p.hdr, DSPARK_TIMEOUT, what);
    *abort_flag = 1;
  };
  const int M = rows_of(p);
  const int mt = (M + 255) / 256;
  const int64_t tiles = (int64_t)mt * ((p.N + BN - 1) / BN);

  if (warp == kEpiWarps) {
    if (lane == 0) {
      // loads: this CTA's rows of a and its half of w's rows, signalled to the first CTA
      const uint64_t pol_a = ptx::policy_evict_last(), pol_w = ptx::policy_evict_normal();
      uint32_t bar0[NS];
      for (int i = 0; i < NS; ++i) bar0[i] = ptx::map_to_rank(&full[i], 0);
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = pair; t < tiles && ok; t += pairs) {
        const int m0 = (int)(t % mt) * 256 + (int)rank * 128, n0 = (int)(t / mt) * BN + (int)rank * (BN / 2);
        for (int b = 0; b < p.kb; ++b, ++it) {
          const uint32_t s = it % NS;
          if (!ptx::mbar_wait(&empty[s], ((it / NS) & 1) ^ 1, abort_flag, kWaitLimitNs)) {
            fail(1);
            ok = false;
            break;
          }
          uint8_t* dst = sm + s * W::kStage;
          if (rank == 0) ptx::mbar_expect_tx(&full[s], 2 * W::kStage);
          ptx::tma_load_2d_pair(dst, &tmA, bar0[s], b * kKb, m0, pol_a);
          ptx::tma_load_2d_pair(dst + W::kA, &tmW, bar0[s], b * kKb, n0, pol_w);
        }
      }
      // nothing of the pair may be in flight when the CTAs leave: the last
      // commits have arrived here, or (after a failure) at least the loads
      for (uint32_t j = it > NS ? it - NS : 0; j < it; ++j)
        if (ok || rank == 0)
          ptx::mbar_wait(ok ? &empty[j % NS] : &full[j % NS], (j / NS) & 1, &never_s, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(256, BN);
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = pair; t < tiles && ok; t += pairs) {
        for (int b = 0; b < p.kb; ++b, ++it) {
          const uint32_t s = it % NS, a = it % NB;
          if (!ptx::mbar_wait(&full[s], (it / NS) & 1, abort_flag, kWaitLimitNs) ||
              !ptx::mbar_wait(&tempty[a], ((it / NB) & 1) ^ 1, abort_flag, kWaitLimitNs)) {
            fail(2);
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sa = ptx::smem_u32(sm + s * W::kStage), sb = sa + W::kA;
#pragma unroll
          for (int k = 0; k < kKb / 32; ++k)
            // K-major, 128B swizzle: 8-row atoms 1024 bytes apart, 32 columns are 32 bytes
            ptx::tc_mma_fp8_pair(tmem + a * BN, ptx::smem_desc_sw128(sa + k * 32, 16, 1024),
                                 ptx::smem_desc_sw128(sb + k * 32, 16, 1024), idesc, k ? 1u : 0u);
          ptx::tc_commit_pair(&empty[s]);
          ptx::tc_commit_pair(&tfull[a]);
        }
      }
    }
    __syncwarp();
  } else {
    constexpr int NC = BN / 2;  // columns of this warp
    constexpr int CH = 128 / (int)sizeof(TO);  // columns of a 128-byte staging row
    const int half = warp >> 2, quarter = warp & 3;
    uint8_t* stg = sm + NS * W::kStage + warp * 8192;
    const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * NC);
    uint32_t te[NB];
    for (int i = 0; i < NB; ++i) te[i] = ptx::map_to_rank(&tempty[i], 0);
    const int nblk = (p.N + kKb - 1) / kKb;
    uint32_t it = 0, stores = 0;
    bool ok = true;
    for (int64_t t = pair; t < tiles && ok; t += pairs) {
      const int row0 = (int)(t % mt) * 256 + (int)rank * 128 + quarter * 32;
      const int col0 = (int)(t / mt) * BN + half * NC;
      const float* as = p.a_scale + (int64_t)min(row0 + lane, M - 1) * p.kb;
      const float* wsc = p.w_scale + (int64_t)min(col0 / kKb, nblk - 1) * p.kb;
      uint64_t acc[NC / 2];
#pragma unroll
      for (int i = 0; i < NC / 2; ++i) acc[i] = 0;
      float scale = as[0] * wsc[0];
      for (int b = 0; b < p.kb; ++b, ++it) {
        const uint32_t a = it % NB;
        const float next = b + 1 < p.kb ? as[b + 1] * wsc[b + 1] : 0.f;
        const bool got = ptx::mbar_wait(&tfull[a], (it / NB) & 1, abort_flag, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) fail(3);
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint64_t s2 = ptx::pack2(scale, scale);
        float v[2][16];
        ptx::tmem_ld16(taddr + a * BN, v[0]);
#pragma unroll
        for (int c = 0; c < NC / 16; ++c) {
          ptx::tmem_ld_wait16(v[c & 1]);
          if (c + 1 < NC / 16) {
            ptx::tmem_ld16(taddr + a * BN + (c + 1) * 16, v[(c + 1) & 1]);
          } else {
            ptx::tc_fence_before();
            if (lane == 0) ptx::mbar_arrive_remote(te[a]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[c * 8 + i] = ptx::fma2(ptx::pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), s2, acc[c * 8 + i]);
        }
        scale = next;
      }
      if (!ok) break;
      // 32 rows x 128 bytes at a time through this warp's swizzled staging buffers
#pragma unroll
      for (int c = 0; c < NC / CH; ++c) {
        uint8_t* buf = stg + (stores & 1) * 4096;
        const int col = col0 + c * CH;
        if (stores >= 2) {
          if (lane == 0) ptx::bulk_wait_read1();
          __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint4 q;
          if (sizeof(TO) == 2) {
            const uint64_t* x = acc + c * (CH / 2) + u * 4;
            const float2 f0 = ptx::unpack2(x[0]), f1 = ptx::unpack2(x[1]), f2 = ptx::unpack2(x[2]),
                         f3 = ptx::unpack2(x[3]);
            q = make_uint4(pack_bf16(f0.x, f0.y), pack_bf16(f1.x, f1.y), pack_bf16(f2.x, f2.y), pack_bf16(f3.x, f3.y));
          } else {
            const uint64_t* x = acc + c * (CH / 2) + u * 2;
            q = make_uint4((uint32_t)x[0], (uint32_t)(x[0] >> 32), (uint32_t)x[1], (uint32_t)(x[1] >> 32));
          }
          *reinterpret_cast<uint4*>(buf + lane * 128 + ((u ^ (lane & 7)) << 4)) = q;
        }
        if (col < p.N && row0 < M) {
          if (p.tma_out && (row0 + 32 <= M || M == p.M)) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::tma_store_2d(&tmO, buf, col, row0);
          } else {
            __syncwarp();
            TO* o = static_cast<TO*>(p.out) + col;
            for (int r = 0; r < min(32, M - row0); ++r) {
              const uint32_t w32 =
                  *reinterpret_cast<const uint32_t*>(buf + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
              TO* dst = o + (int64_t)(row0 + r) * p.ldo;
              if (sizeof(TO) == 4) {
                if (col + lane < p.N) reinterpret_cast<uint32_t*>(dst)[lane] = w32;
              } else {
                if (col + 2 * lane < p.N) reinterpret_cast<uint16_t*>(dst)[2 * lane] = (uint16_t)w32;
                if (col + 2 * lane + 1 < p.N) reinterpret_cast<uint16_t*>(dst)[2 * lane + 1] = (uint16_t)(w32 >> 16);
              }
            }
          }
        }
        if (lane == 0) ptx::bulk_commit();
        ++stores;
        __syncwarp();
      }
    }
    if (lane == 0) ptx::bulk_wait0();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == kEpiWarps + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// narrow: 128 rows of w on the lanes, NT rows of a on the columns, a cluster over K
// ---------------------------------------------------------------------------
constexpr int kNarrowThreads = 192;  // 4 epilogue warps, loads, MMA

template <int NT>
struct Narrow {
  static constexpr uint32_t kW = 128 * kKb;
  static constexpr uint32_t kA = NT * kKb;
  static constexpr uint32_t kStage = kW + kA;
  static constexpr int kBufs = 4;
  static constexpr uint32_t kCols = NT * kBufs < 32 ? 32 : NT * kBufs;
  static constexpr uint32_t kRed = NT * 128 * 4;  // a tile's sums, one float each
};

template <int NT, typename TO>
__global__ void __launch_bounds__(kNarrowThreads, 1)
    k_fp8_narrow(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, const MmParams p,
                 int split, int stages, int m_tiles) {
  using C = Narrow<NT>;
  constexpr int NB = C::kBufs;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  constexpr int kMaxStages = 12;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], tfull[NB], tempty[NB];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s, never_s;
  volatile int* abort_flag = &abort_s;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? (int)ptx::cluster_rank() : 0;
  const int cl = blockIdx.x / split, cls = gridDim.x / split;
  float* red = reinterpret_cast<float*>(sm + stages * C::kStage);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], 4);
    }
    ptx::fence_mbar_init();
    abort_s = never_s = 0;
    ptx::prefetch_map(&tmA);
    ptx::prefetch_map(&tmW);
  }
  if (warp == 5) {
    ptx::tmem_alloc(&tmem_slot, C::kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  auto fail = [&](int what) {
    if (p.hdr) report_error(p.hdr, DSPARK_TIMEOUT, what);
    *abort_flag = 1;
  };
  const int M = rows_of(p);
  const int mt = min(m_tiles, (M + NT - 1) / NT);
  const int64_t tiles = (int64_t)mt * ((p.N + 127) / 128);
  const int b0 = (int)((int64_t)p.kb * rank / split), b1 = (int)((int64_t)p.kb * (rank + 1) / split);

  if (warp == 4) {
    if (lane == 0) {
      const uint64_t pol_a = ptx::policy_evict_last(), pol_w = ptx::policy_evict_first();
      uint32_t s = 0, ph = 0, n = 0;
      bool ok = true;
      for (int64_t t = cl; t < tiles && ok; t += cls) {
        const int m0 = (int)(t % mt) * NT, n0 = (int)(t / mt) * 128;
        for (int b = b0; b < b1; ++b) {
          if (!ptx::mbar_wait(&empty[s], ph ^ 1, abort_flag, kWaitLimitNs)) {
            fail(4);
            ok = false;
            break;
          }
          uint8_t* dst = sm + s * C::kStage;
          ptx::mbar_expect_tx(&full[s], C::kStage);
          ptx::tma_load_2d(dst, &tmW, &full[s], b * kKb, n0, pol_w);
          ptx::tma_load_2d(dst + C::kW, &tmA, &full[s], b * kKb, m0, pol_a);
          ++n;
          if (++s == (uint32_t)stages) s = 0, ph ^= 1;
        }
      }
      // nothing may be in flight when the CTA leaves
      for (uint32_t j = n > (uint32_t)stages ? n - stages : 0; j < n; ++j)
        ptx::mbar_wait(&full[j % stages], (j / stages) & 1, &never_s, kWaitLimitNs);
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, NT);
      uint32_t s = 0, ph = 0, it = 0;
      bool ok = true;
      for (int64_t t = cl; t < tiles && ok; t += cls) {
        for (int b = b0; b < b1; ++b, ++it) {
          const uint32_t a = it % NB;
          if (!ptx::mbar_wait(&full[s], ph, abort_flag, kWaitLimitNs) ||
              !ptx::mbar_wait(&tempty[a], ((it / NB) & 1) ^ 1, abort_flag, kWaitLimitNs)) {
            fail(5);
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sw = ptx::smem_u32(sm + s * C::kStage), sa = sw + C::kW;
#pragma unroll
          for (int k = 0; k < kKb / 32; ++k)
            ptx::tc_mma_fp8(tmem + a * NT, ptx::smem_desc_sw128(sw + k * 32, 16, 1024),
                            ptx::smem_desc_sw128(sa + k * 32, 16, 1024), idesc, k ? 1u : 0u);
          ptx::tc_commit(&empty[s]);
          ptx::tc_commit(&tfull[a]);
          if (++s == (uint32_t)stages) s = 0, ph ^= 1;
        }
      }
    }
    __syncwarp();
  }
  uint32_t it = 0;
  bool ok = true;
  for (int64_t t = cl; t < tiles; t += cls) {
    const int m0 = (int)(t % mt) * NT, n0 = (int)(t / mt) * 128;
    const int nm = min(NT, M - m0);
    if (warp < 4) {
      const float* wsc = p.w_scale + (int64_t)(n0 / kKb) * p.kb;
      float acc[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = 0.f;
      for (int b = b0; b < b1 && ok; ++b, ++it) {
        const uint32_t a = it % NB;
        const float ws = wsc[b];
        // lane l holds the scales of columns l and l + 32
        float sc[(NT + 31) / 32];
#pragma unroll
        for (int j = 0; j < (NT + 31) / 32; ++j) {
          const int c = j * 32 + lane;
          sc[j] = c < nm ? ws * p.a_scale[(int64_t)(m0 + c) * p.kb + b] : 0.f;
        }
        const bool got = ptx::mbar_wait(&tfull[a], (it / NB) & 1, abort_flag, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) fail(6);
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t ta = tmem + ((uint32_t)(warp * 32) << 16) + a * NT;
#pragma unroll
        for (int c = 0; c < NT / 16; ++c) {
          float v[16];
          ptx::tmem_ld16(ta + c * 16, v);
          ptx::tmem_ld_wait16(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int col = c * 16 + i;
            acc[col] = fmaf(v[i], __shfl_sync(0xffffffffu, sc[col / 32], col & 31), acc[col]);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&tempty[a]);
      }
      if (split == 1) {
        const int n = n0 + warp * 32 + lane;
        if (ok && n < p.N) {
          TO* o = static_cast<TO*>(p.out) + (int64_t)m0 * p.ldo + n;
#pragma unroll
          for (int i = 0; i < NT; ++i)
            if (i < nm) store_out(o + (int64_t)i * p.ldo, acc[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (i < nm) red[i * 128 + warp * 32 + lane] = acc[i];
      }
    }
    if (split > 1) {
      // every CTA adds the parts of its share of the tile's rows in rank order
      __syncwarp();
      ptx::cluster_sync();
      for (int u = threadIdx.x; u < nm * 32; u += kNarrowThreads) {
        if ((u / 32) % split != rank) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < split; ++r) {
          const float4 v = ptx::ld_cluster_f4(ptx::map_to_rank(red + u * 4, r));
          s.x += v.x;
          s.y += v.y;
          s.z += v.z;
          s.w += v.w;
        }
        TO* o = static_cast<TO*>(p.out) + (int64_t)(m0 + u / 32) * p.ldo;
        const int n = n0 + (u % 32) * 4;
        if (n < p.N) store_out(o + n, s.x);
        if (n + 1 < p.N) store_out(o + n + 1, s.y);
        if (n + 2 < p.N) store_out(o + n + 2, s.z);
        if (n + 3 < p.N) store_out(o + n + 3, s.w);
      }
      __syncwarp();
      ptx::cluster_sync();
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kCols);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct Dev {
  int sms = 0;
  int pairs = 0;  // CTA pairs of the wide kernel that run at the same time
  bool sm103 = false;
};

// properties of the current device, looked up once each
cudaError_t device(Dev* out) {
  constexpr int kMaxDev = 64;
  static Dev cache[kMaxDev];
  static bool have[kMaxDev] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorNotSupported;
  std::lock_guard<std::mutex> lock(mu);
  if (!have[dev]) {
    int major = 0, minor = 0;
    Dev d;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    d.sm103 = major == 10 && minor == 3;
    if (d.sm103) {
      const void* f = (const void*)k_fp8_wide<256, __nv_bfloat16>;
      if ((e = ensure_smem_limit(f, (int)Wide<256>::kSmem)) != cudaSuccess) return e;
      cudaLaunchConfig_t c = {};
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 2;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      c.gridDim = dim3((unsigned)(d.sms / 2 * 2));
      c.blockDim = dim3(kWideThreads);
      c.dynamicSmemBytes = Wide<256>::kSmem;
      c.attrs = at;
      c.numAttrs = 1;
      if ((e = cudaOccupancyMaxActiveClusters(&d.pairs, f, &c)) != cudaSuccess) return e;
      d.pairs = std::max(1, std::min(d.pairs, d.sms / 2));
    }
    cache[dev] = d;
    have[dev] = true;
  }
  *out = cache[dev];
  return cudaSuccess;
}

template <int BN, typename TO>
cudaError_t run_wide(const dspark_matmul_fp8_args& a, const MmParams& p, const Dev& d, cudaStream_t s) {
  CUtensorMap tmA, tmW, tmO = {};
  if (!tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a, a.K, a.M, a.lda, kKb, 128) ||
      !tensor_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.K, a.N, a.ldw, kKb, BN / 2))
    return cudaErrorInvalidValue;
  if (p.tma_out &&
      !tensor_map_2d(&tmO, sizeof(TO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.out,
                     a.N, a.M, a.ldo * (int64_t)sizeof(TO), 128 / sizeof(TO), 32))
    return cudaErrorInvalidValue;
  const void* f = (const void*)k_fp8_wide<BN, TO>;
  if (const cudaError_t e = ensure_smem_limit(f, (int)Wide<BN>::kSmem); e != cudaSuccess) return e;
  const int64_t tiles = (((int64_t)a.M + 255) / 256) * (((int64_t)a.N + BN - 1) / BN);
  const unsigned grid = 2 * (unsigned)std::min<int64_t>(tiles, d.pairs);
  k_fp8_wide<BN, TO><<<grid, kWideThreads, Wide<BN>::kSmem, s>>>(tmA, tmW, tmO, p);
  count_launches(1);
  return cudaGetLastError();
}

template <int NT, typename TO>
cudaError_t run_narrow(const dspark_matmul_fp8_args& a, const MmParams& p, const Dev& d, cudaStream_t s) {
  using C = Narrow<NT>;
  CUtensorMap tmA, tmW;
  if (!tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a, a.K, a.M, a.lda, kKb, NT) ||
      !tensor_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.K, a.N, a.ldw, kKb, 128))
    return cudaErrorInvalidValue;
  const int mt = (a.M + NT - 1) / NT;
  const int64_t tiles = (int64_t)mt * (((int64_t)a.N + 127) / 128);
  int split = 1;
  while (split < 8 && tiles * split * 2 <= d.sms && p.kb >= split * 4) split *= 2;
  // a deep ring where one CTA has an SM to itself for many blocks
  const int stages = split > 1 ? 4 : NT <= 16 ? 11 : NT <= 32 ? 9 : 8;
  const uint32_t smem = stages * C::kStage + (split > 1 ? C::kRed : 0) + 1024;
  const void* f = (const void*)k_fp8_narrow<NT, TO>;
  if (const cudaError_t e = ensure_smem_limit(f, (int)smem); e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.gridDim = dim3((unsigned)(split > 1 ? tiles * split : std::min<int64_t>(tiles, d.sms)));
  c.blockDim = dim3(kNarrowThreads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = at;
  c.numAttrs = split > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&c, k_fp8_narrow<NT, TO>, tmA, tmW, p, split, stages, mt);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

template <typename TO>
cudaError_t run(const dspark_matmul_fp8_args& a, const MmParams& p, const Dev& d, cudaStream_t s) {
  if (a.M <= 16) return run_narrow<16, TO>(a, p, d, s);
  if (a.M <= 32) return run_narrow<32, TO>(a, p, d, s);
  if (a.M <= 64) return run_narrow<64, TO>(a, p, d, s);
  const int64_t mt = ((int64_t)a.M + 255) / 256;
  // the tile width that finishes first: waves of pairs times the width
  const auto cost = [&](int bn) { return (mt * ((a.N + bn - 1) / bn) + d.pairs - 1) / d.pairs * bn; };
  return cost(128) < cost(256) ? run_wide<128, TO>(a, p, d, s) : run_wide<256, TO>(a, p, d, s);
}

}  // namespace

size_t matmul_fp8_ws(int, int, int) { return sizeof(WsHeader); }

cudaError_t launch_matmul_fp8(const dspark_matmul_fp8_args& a, uint8_t* ws, cudaStream_t s) {
  Dev d;
  if (const cudaError_t e = device(&d); e != cudaSuccess) return e;
  if (!d.sm103) return cudaErrorNotSupported;
  const int esize = (int)elem_size(a.out_dtype);
  MmParams p = {};
  p.M = a.M;
  p.N = a.N;
  p.kb = (int)(((int64_t)a.K + kKb - 1) / kKb);
  p.a_scale = a.a_scale;
  p.w_scale = a.w_scale;
  p.out = a.out;
  p.ldo = a.ldo;
  p.n_rows = a.n_rows;
  p.tma_out = ((uintptr_t)a.out % 16) == 0 && (a.M == 1 || (a.ldo * esize) % 16 == 0);
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  return a.out_dtype == DSPARK_BF16 ? run<__nv_bfloat16>(a, p, d, s) : run<float>(a, p, d, s);
}

}  // namespace dspark

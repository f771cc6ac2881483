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
//                 BN rows of w.  A row's scale is one number a lane, so the
//                 promotion is one packed FMA for two elements.  2048 x 4096 x 151936
//                 to bf16: 0.86 ms, 2.97 PFLOP/s, for a call in 20 ms (2070 MHz); back to
//                 back 0.96 to 1.01 ms, where the power cap holds the clock at 1.55 GHz.
//                 Bounded by the round trip of a TMEM buffer (MMA, commit, read-out,
//                 release; the tensor pipe is busy 63 % of the time) and then by power.
//   k_fp8_narrow  rows of w on the lanes, up to 64 rows of a on the columns: bounded
//                 by reading w (1 row x 2560 x 151936: 62 to 64 us, 0.90 to 0.92 of
//                 measured HBM; 64 x 7168 x 129280 to fp32: 148 us, 0.96; its 1010 tiles
//                 are 6.6 waves).  A cluster of S CTAs
//                 splits the blocks of K and adds its parts through distributed
//                 shared memory in rank order (no atomics: equal calls give equal
//                 bits): 8 x 2560 x 2560 5.4 us.
//
// Every wait is bounded; one that gives up reports DSPARK_TIMEOUT.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "launch.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace dspark {

namespace {

constexpr long long kWaitLimit = 4000000000ll;  // cycles: about two seconds
constexpr int kKb = DSPARK_FP8_BLOCK;  // columns of a block: one 128-byte swizzled row of shared memory

struct MmParams {
  int M, N, kb;
  const float* a_scale;  // [M, kb]
  const float* w_scale;  // [ceil(N / 128), kb]
  void* out;
  int64_t ldo;
  const int32_t* n_rows;
  // stores by TMA: 0 none (the output's rows are not 16-byte aligned), 1 those that
  // end inside a row, 2 a row's last one too.  A tensor's store writes whole 16-byte
  // pieces, so it would pass a row end that is no multiple of 16 bytes.
  int tma_out;
  int a_vec;    // a_scale is 16-byte aligned
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
// wide: 256 x (128 NH) tiles by CTA pairs
// ---------------------------------------------------------------------------
// Warps of a CTA: 8 NH epilogue warps (a warpgroup reads EC = 64 columns of TMEM;
// 16 of 32 columns for one part to fp32 rows that TMA cannot store, whose stores are
// many: 333 x 2050 x 10007 22.9 against 25.5 us, but 512 x 4096 x 4096 12.9 against 12.3),
// then one each for loads and scales and NH for the MMAs.
//
// A tile's columns are made as NH parts of 128, each with its own TMEM buffers:
// a buffer goes MMA -> commit -> read out -> release, and the commit and the
// release cross the pair (some 350 cycles each), so four smaller buffers keep the
// tensor cores busier than two of 256 columns.  Part h takes rows 64 h .. 64 h + 63
// of each CTA's rows of w: its columns 0-63 are the first CTA's, 64-127 the
// second's, so a warpgroup's 64 columns lie in one scale block.
template <int NH, int EC>
struct Wide {
  static constexpr int BN = 128 * NH;
  static constexpr int kEpiWarps = 4 * BN / EC;
  static constexpr int kThreads = 32 * (kEpiWarps + 2 + NH);
  // registers of the epilogue warps and of the last warpgroup (NH = 2)
  static constexpr int kRegsHigh = 104, kRegsLow = 64;
  static constexpr uint32_t kA = 128 * kKb;       // bytes of a per CTA and stage
  static constexpr uint32_t kB = BN / 2 * kKb;    // bytes of w per CTA and stage
  static constexpr uint32_t kStage = kA + kB;
  static constexpr int kStages = NH == 2 ? 4 : 6;
  static constexpr int kBufs = 4 / NH;            // TMEM buffers of 128 columns per part
  static constexpr uint32_t kStg = kEpiWarps * 4096;  // output staging: 32 rows x 128 bytes a warp
  static constexpr int kSlots = 4;                // scale ring: slots of 4 blocks
  static constexpr uint32_t kSlot = 4 * 2 * 128 * 4;  // [4 blocks][2 column blocks][128 rows] fp32
  static constexpr uint32_t kSmem = kStages * kStage + kStg + kSlots * kSlot + 1024;
};

template <int NH, int EC, typename TO>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Wide<NH, EC>::kThreads, 1)
    k_fp8_wide(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW,
               const __grid_constant__ CUtensorMap tmO, const MmParams p) {
  using W = Wide<NH, EC>;
  constexpr int NS = W::kStages, NB = W::kBufs, BN = W::BN, EW = W::kEpiWarps;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  // the same offset in both CTAs: the descriptors of a pair name one place for both
  uint8_t* sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* stg_all = sm + NS * W::kStage;
  float* ring = reinterpret_cast<float*>(stg_all + W::kStg);
  __shared__ uint64_t full[NS], empty[NS], tfull[NH * NB], tempty[NH * NB], sfull[W::kSlots], sempty[W::kSlots];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s, never_s;
  volatile int* abort_flag = &abort_s;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp-uniform
  const uint32_t rank = ptx::cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], NH);
    }
    for (int i = 0; i < NH * NB; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], 2 * EW / NH);
    }
    for (int i = 0; i < W::kSlots; ++i) {
      ptx::mbar_init(&sfull[i], 32);
      ptx::mbar_init(&sempty[i], EW);
    }
    ptx::fence_mbar_init();
    abort_s = never_s = 0;
    ptx::prefetch_map(&tmA);
    ptx::prefetch_map(&tmW);
    ptx::prefetch_map(&tmO);
  }
  if (warp == EW + 2) {
    ptx::tmem_alloc_pair(&tmem_slot, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  ptx::launch_dependents();
  ptx::grid_wait();
  auto fail = [&](int what) {
    if (p.hdr) report_error(p.hdr, DSPARK_TIMEOUT, what);
    *abort_flag = 1;
  };
  const int M = rows_of(p);
  const int mt = (M + 255) / 256;
  const int tiles = mt * ((p.N + BN - 1) / BN);
  const int nblk = (p.N + kKb - 1) / kKb;

  // the epilogue warps' accumulators need more than an even share of the
  // registers: with 96 each they spill (2048 x 4096 x 151936 1.03 ms, when this was 0.89)
  if (NH == 2) {
    if (warp >= EW)
      ptx::reg_dec<W::kRegsLow>();
    else
      ptx::reg_inc<W::kRegsHigh>();
  }
  if (warp == EW) {
    // loads: this CTA's rows of a and its half of w's rows, signalled to the
    // first CTA.  The whole warp runs the loop and one elected lane issues, as
    // for the MMAs: from one thread of a divergent branch the loads alone took
    // longer than the tensor cores.
    const uint64_t pol_a = ptx::policy_evict_last(), pol_w = ptx::policy_evict_normal();
    const uint32_t bar0 = ptx::map_to_rank(&full[0], 0);
    uint32_t s = 0, ph = 1, n = 0;
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += pairs) {
      const int m0 = (t % mt) * 256 + (int)rank * 128, n0 = (t / mt) * BN + (int)rank * (BN / 2);
      for (int b = 0; b < p.kb; ++b) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_cycles(&empty[s], ph, abort_flag, kWaitLimit));
        if (!ok) {
          if (lane == 0) fail(1);
          break;
        }
        if (ptx::elect_one()) {
          uint8_t* dst = sm + s * W::kStage;
          if (rank == 0) ptx::mbar_expect_tx(&full[s], 2 * W::kStage);
          ptx::tma_load_2d_pair(dst, &tmA, bar0 + s * 8, b * kKb, m0, pol_a);
          ptx::tma_load_2d_pair(dst + W::kA, &tmW, bar0 + s * 8, b * kKb, n0, pol_w);
        }
        __syncwarp();
        ++n;
        if (++s == NS) s = 0, ph ^= 1;
      }
    }
    // nothing of the pair may be in flight when the CTAs leave: the last
    // commits have arrived here, or (after a failure) at least the loads
    for (uint32_t j = n > NS ? n - NS : 0; j < n; ++j)
      if (ok || rank == 0)
        ptx::mbar_wait_cycles(ok ? &empty[j % NS] : &full[j % NS], (j / NS) & 1, &never_s, kWaitLimit);
    __syncwarp();
  } else if (warp > EW + 1) {
    // one MMA warp per part: its waits (some 80 cycles each even when they
    // are over) run beside the other's
    if (rank == 0) {
      const int h = warp - (EW + 2);
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(256, 128);
      // K-major, 128B swizzle: 8-row atoms 1024 bytes apart, 32 columns are 32 bytes
      const uint64_t da0 = ptx::smem_desc_sw128(ptx::smem_u32(sm), 16, 1024);
      const uint64_t db0 = ptx::smem_desc_sw128(ptx::smem_u32(sm + W::kA + h * (64 * kKb)), 16, 1024);
      const uint32_t d0 = tmem + h * NB * 128;
      uint32_t s = 0, ph = 0, q = 0, tph = 1;
      for (int t = pair; t < tiles; t += pairs) {
        for (int b = 0; b < p.kb; ++b) {
          // after a wait that gave up the loop runs on (its results are void): every later wait ends at once
          if (!ptx::mbar_wait_cycles(&full[s], ph, abort_flag, kWaitLimit) ||
              !ptx::mbar_wait_cycles(&tempty[h * NB + q], tph, abort_flag, kWaitLimit))
            fail(2);
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint64_t da = da0 + s * (W::kStage >> 4), db = db0 + s * (W::kStage >> 4);
            const uint32_t d = d0 + q * 128;
            ptx::tc_mma_fp8_pair<0>(d, da, db, idesc);
            ptx::tc_mma_fp8_pair<1>(d, da + 2, db + 2, idesc);
            ptx::tc_mma_fp8_pair<1>(d, da + 4, db + 4, idesc);
            ptx::tc_mma_fp8_pair<1>(d, da + 6, db + 6, idesc);
            ptx::tc_commit_pair(&tfull[h * NB + q]);
            ptx::tc_commit_pair(&empty[s]);
          }
          __syncwarp();
          if (++s == NS) s = 0, ph ^= 1;
          if (++q == NB) q = 0, tph ^= 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == EW + 1) {
    // scales: a_scale[row, b] w_scale[column block, b] of four blocks b at a time, four rows a lane
    uint32_t slot = 0, ph = 1;
    bool ok = true;
    for (int t = pair; t < tiles && ok; t += pairs) {
      const int m0 = (t % mt) * 256 + (int)rank * 128, nb = (t / mt) * NH;
      const float* w0 = p.w_scale + (int64_t)min(nb, nblk - 1) * p.kb;
      const float* w1 = p.w_scale + (int64_t)min(nb + NH - 1, nblk - 1) * p.kb;
      for (int b = 0; b < p.kb; b += 4) {
        float sa[4][4], sw[2][4];
        const int nb4 = min(4, p.kb - b);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float* ap = p.a_scale + (int64_t)min(m0 + r * 32 + lane, M - 1) * p.kb + b;
          if (nb4 == 4 && (p.kb & 3) == 0 && p.a_vec) {
            const float4 f = *reinterpret_cast<const float4*>(ap);
            sa[r][0] = f.x, sa[r][1] = f.y, sa[r][2] = f.z, sa[r][3] = f.w;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) sa[r][j] = j < nb4 ? ap[j] : 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sw[0][j] = j < nb4 ? w0[b + j] : 0.f;
          sw[1][j] = j < nb4 ? w1[b + j] : 0.f;
        }
        const bool got = ptx::mbar_wait_cycles(&sempty[slot], ph, abort_flag, kWaitLimit);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) fail(7);
          ok = false;
          break;
        }
        float* d = ring + slot * (W::kSlot / 4) + lane;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int r = 0; r < 4; ++r) d[(j * 2 + c) * 128 + r * 32] = sa[r][j] * sw[c][j];
        ptx::mbar_arrive(&sfull[slot]);
        if (++slot == W::kSlots) slot = 0, ph ^= 1;
      }
    }
  } else {
    constexpr int CH = 128 / (int)sizeof(TO);  // columns of a 128-byte staging row
    constexpr int per_part = 128 / EC, per_side = 64 / EC;
    const int g = warp >> 2, quarter = warp & 3;
    const int part = g / per_part, side = g % per_part / per_side, sub = g % per_side * EC;
    uint8_t* stg = stg_all + warp * 4096;
    const uint32_t taddr = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(part * NB * 128 + side * 64 + sub);
    const uint32_t te = ptx::map_to_rank(&tempty[part * NB], 0);
    const float* sc = ring + side * 128 + quarter * 32 + lane;
    uint32_t q = 0, tph = 0, slot = 0, sph = 0;
    bool staged = false;
    for (int t = pair; t < tiles; t += pairs) {
      const int row0 = (t % mt) * 256 + (int)rank * 128 + quarter * 32;
      const int col0 = (t / mt) * BN + side * (BN / 2) + part * 64 + sub;
      uint64_t acc[EC / 2];
#pragma unroll
      for (int i = 0; i < EC / 2; ++i) acc[i] = 0;
      for (int b = 0; b < p.kb; ++b) {
        bool got = true;
        if ((b & 3) == 0) got = ptx::mbar_wait_cycles(&sfull[slot], sph, abort_flag, kWaitLimit);
        const float scale = sc[slot * (W::kSlot / 4) + (b & 3) * 256];
        const uint64_t s2 = ptx::pack2(scale, scale);
        got = ptx::mbar_wait_cycles(&tfull[part * NB + q], tph, abort_flag, kWaitLimit) && got;
        if (!got) fail(3);  // the loop runs on: every later wait ends at once
        __syncwarp();
        ptx::tc_fence_after();
        // 16 columns arrive while the 16 before them are added
        float v[2][16];
        ptx::tmem_ld16(taddr + q * 128, v[0]);
#pragma unroll
        for (int c = 0; c < EC / 16; ++c) {
          ptx::tmem_ld_wait16(v[c & 1]);
          if (c + 1 < EC / 16) {
            ptx::tmem_ld16(taddr + q * 128 + (c + 1) * 16, v[(c + 1) & 1]);
          } else {
            ptx::tc_fence_before();
            if (lane == 0) ptx::mbar_arrive_remote(te + q * 8);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            acc[c * 8 + i] = ptx::fma2(ptx::pack2(v[c & 1][2 * i], v[c & 1][2 * i + 1]), s2, acc[c * 8 + i]);
        }
        if (++q == NB) q = 0, tph ^= 1;
        if ((b & 3) == 3 || b + 1 == p.kb) {
          if (lane == 0) ptx::mbar_arrive(&sempty[slot]);
          if (++slot == W::kSlots) slot = 0, sph ^= 1;
        }
      }
      // 32 rows x 128 bytes at a time through this warp's swizzled staging buffer
#pragma unroll
      for (int c = 0; c < EC / CH; ++c) {
        const int col = col0 + c * CH;
        if (col >= p.N || row0 >= M) break;
        if (staged) {
          if (lane == 0) ptx::bulk_wait_read0();
          __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint4 v;
          if (sizeof(TO) == 2) {
            const uint64_t* x = acc + c * (CH / 2) + u * 4;
            const float2 f0 = ptx::unpack2(x[0]), f1 = ptx::unpack2(x[1]), f2 = ptx::unpack2(x[2]),
                         f3 = ptx::unpack2(x[3]);
            v = make_uint4(pack_bf16(f0.x, f0.y), pack_bf16(f1.x, f1.y), pack_bf16(f2.x, f2.y), pack_bf16(f3.x, f3.y));
          } else {
            const uint64_t* x = acc + c * (CH / 2) + u * 2;
            v = make_uint4((uint32_t)x[0], (uint32_t)(x[0] >> 32), (uint32_t)x[1], (uint32_t)(x[1] >> 32));
          }
          // 128B swizzle: 16-byte unit u of row r at u ^ (r % 8)
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((u ^ (lane & 7)) << 4)) = v;
        }
        if ((p.tma_out == 2 || (p.tma_out == 1 && col + CH <= p.N)) && (row0 + 32 <= M || M == p.M)) {
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::tma_store_2d(&tmO, stg, col, row0);
            ptx::bulk_commit();
          }
          staged = true;
        } else {
          __syncwarp();
          // a row at a time, four bytes a lane
          TO* dst = static_cast<TO*>(p.out) + (int64_t)row0 * p.ldo + col;
          const int rows = min(32, M - row0);
#pragma unroll 8
          for (int r = 0; r < 32; ++r) {
            const uint32_t w32 =
                *reinterpret_cast<const uint32_t*>(stg + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
            if (r < rows) {
              TO* o = dst + (int64_t)r * p.ldo;
              if (sizeof(TO) == 4) {
                if (col + lane < p.N) reinterpret_cast<uint32_t*>(o)[lane] = w32;
              } else {
                if (col + 2 * lane < p.N) reinterpret_cast<uint16_t*>(o)[2 * lane] = (uint16_t)w32;
                if (col + 2 * lane + 1 < p.N) reinterpret_cast<uint16_t*>(o)[2 * lane + 1] = (uint16_t)(w32 >> 16);
              }
            }
          }
          __syncwarp();
        }
      }
    }
    if (lane == 0) ptx::bulk_wait0();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == EW + 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// narrow: 128 rows of w on the lanes, NT rows of a on the columns, a cluster over K
// ---------------------------------------------------------------------------
template <int NT>
struct Narrow {
  static constexpr int kCols32 = NT < 32 ? NT : 32;     // columns of an epilogue warp
  static constexpr int kEpiWarps = 4 * (NT / kCols32);
  static constexpr int kThreads = 32 * (kEpiWarps + 3);  // and loads, two for the MMAs
  static constexpr uint32_t kW = 128 * kKb;
  static constexpr uint32_t kA = NT * kKb;
  static constexpr uint32_t kStage = kW + kA;
  static constexpr int kBufs = 8;
  static constexpr uint32_t kTmemCols = NT * kBufs;
  static constexpr uint32_t kRed = NT * 128 * 4;  // a tile's sums, one float each
  // Stages of the ring: a deep one where a CTA has an SM to itself for many
  // blocks, fewer in a cluster.  Even, like kBufs: the two MMA warps take every
  // other block, and a parity wait only holds for a warp that has seen the phase
  // before end.  With 9 stages a warp met every other phase of a stage and could
  // take a block that had not arrived.
  static constexpr int kDeepStages = NT <= 16 ? 12 : NT <= 32 ? 10 : 8, kSplitStages = NT <= 32 ? 4 : 6;
  static_assert(kDeepStages % 2 == 0 && kSplitStages % 2 == 0 && kBufs % 2 == 0,
                "a stage and a buffer belong to one MMA warp");
  static constexpr uint32_t smem(bool split) {
    return (split ? kSplitStages * kStage + kRed : kDeepStages * kStage) + 1024;
  }
};

// Two clusters on the same SMs (of two streams, say) must never want more TMEM than
// there is: each could hold it on one SM and wait for the other's on the next, for
// ever.  Up to 32 rows two CTAs want 256 or 512 columns of the 512 and three do not fit
// an SM's shared memory; a CTA of 64 rows wants all of them and leaves no shared
// memory for another CTA.
constexpr uint32_t kSmShared = 228 * 1024;
static_assert(2 * Narrow<32>::kTmemCols <= 512 && 3 * Narrow<16>::smem(true) > kSmShared &&
                  Narrow<64>::smem(true) + Narrow<16>::smem(true) > kSmShared &&
                  Narrow<16>::smem(true) <= Narrow<32>::smem(true),
              "TMEM of the clusters that share an SM");

template <int NT, typename TO>
__global__ void __launch_bounds__(Narrow<NT>::kThreads, 1)
    k_fp8_narrow(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmW, const MmParams p,
                 int split, int m_tiles) {
  using C = Narrow<NT>;
  constexpr int NB = C::kBufs, EW = C::kEpiWarps, NC = C::kCols32;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full[C::kDeepStages], empty[C::kDeepStages], tfull[NB], tempty[NB];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_s, never_s;
  volatile int* abort_flag = &abort_s;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // warp-uniform
  const int rank = split > 1 ? (int)ptx::cluster_rank() : 0;
  const int cl = blockIdx.x / split, cls = gridDim.x / split;
  const int stages = split > 1 ? C::kSplitStages : C::kDeepStages;
  float* red = reinterpret_cast<float*>(sm + stages * C::kStage);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      ptx::mbar_init(&tfull[i], 1);
      ptx::mbar_init(&tempty[i], EW);
    }
    ptx::fence_mbar_init();
    abort_s = never_s = 0;
    ptx::prefetch_map(&tmA);
    ptx::prefetch_map(&tmW);
  }
  if (warp == EW + 1) {
    ptx::tmem_alloc(&tmem_slot, C::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  ptx::launch_dependents();
  ptx::grid_wait();
  auto fail = [&](int what) {
    if (p.hdr) report_error(p.hdr, DSPARK_TIMEOUT, what);
    *abort_flag = 1;
  };
  const int M = rows_of(p);
  const int mt = min(m_tiles, (M + NT - 1) / NT);
  const int64_t tiles = (int64_t)mt * ((p.N + 127) / 128);
  const int b0 = (int)((int64_t)p.kb * rank / split), b1 = (int)((int64_t)p.kb * (rank + 1) / split);

  if (warp == EW) {
    const uint64_t pol_a = ptx::policy_evict_last(), pol_w = ptx::policy_evict_first();
    uint32_t s = 0, ph = 1, n = 0;
    bool ok = true;
    for (int64_t t = cl; t < tiles && ok; t += cls) {
      const int m0 = (int)(t % mt) * NT, n0 = (int)(t / mt) * 128;
      for (int b = b0; b < b1; ++b) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait_cycles(&empty[s], ph, abort_flag, kWaitLimit));
        if (!ok) {
          if (lane == 0) fail(4);
          break;
        }
        if (ptx::elect_one()) {
          uint8_t* dst = sm + s * C::kStage;
          ptx::mbar_expect_tx(&full[s], C::kStage);
          ptx::tma_load_2d(dst, &tmW, &full[s], b * kKb, n0, pol_w);
          ptx::tma_load_2d(dst + C::kW, &tmA, &full[s], b * kKb, m0, pol_a);
        }
        __syncwarp();
        ++n;
        if (++s == (uint32_t)stages) s = 0, ph ^= 1;
      }
    }
    // nothing may be in flight when the CTA leaves
    for (uint32_t j = n > (uint32_t)stages ? n - stages : 0; j < n; ++j)
      ptx::mbar_wait_cycles(&full[j % stages], (j / stages) & 1, &never_s, kWaitLimit);
    __syncwarp();
  } else if (warp > EW) {
    // every other block each: a wait costs some 80 cycles even when it is over, and
    // one warp's waits and issues for a block took longer than its load
    const uint32_t other = warp - (EW + 1);
    constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, NT);
    const uint64_t dw0 = ptx::smem_desc_sw128(ptx::smem_u32(sm), 16, 1024);
    uint32_t s = 0, ph = 0, q = 0, tph = 1;
    bool ok = true;
    for (int64_t t = cl; t < tiles && ok; t += cls) {
      for (int b = b0; b < b1; ++b) {
        if ((q & 1) == other) {
          ok = ptx::mbar_wait_cycles(&full[s], ph, abort_flag, kWaitLimit) &&
               ptx::mbar_wait_cycles(&tempty[q], tph, abort_flag, kWaitLimit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) {
            if (lane == 0) fail(5);
            break;
          }
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint64_t dw = dw0 + s * (C::kStage >> 4), da = dw + (C::kW >> 4);
            ptx::tc_mma_fp8<0>(tmem + q * NT, dw, da, idesc);
            ptx::tc_mma_fp8<1>(tmem + q * NT, dw + 2, da + 2, idesc);
            ptx::tc_mma_fp8<1>(tmem + q * NT, dw + 4, da + 4, idesc);
            ptx::tc_mma_fp8<1>(tmem + q * NT, dw + 6, da + 6, idesc);
            ptx::tc_commit(&empty[s]);
            ptx::tc_commit(&tfull[q]);
          }
          __syncwarp();
        }
        if (++s == (uint32_t)stages) s = 0, ph ^= 1;
        if (++q == NB) q = 0, tph ^= 1;
      }
    }
  }
  uint32_t q = 0, tph = 0;
  bool ok = true;
  const int quarter = warp & 3, c0 = (warp >> 2) * NC;  // lanes and columns of an epilogue warp
  for (int64_t t = cl; t < tiles; t += cls) {
    const int m0 = (int)(t % mt) * NT, n0 = (int)(t / mt) * 128;
    const int nm = min(NT, M - m0);
    if (warp < EW) {
      const float* wsc = p.w_scale + (int64_t)(n0 / kKb) * p.kb;
      // lane l holds the scales of column c0 + l, four blocks' at a time, the next four on their way
      const bool mine = lane < NC && c0 + lane < nm;
      const float* asc = p.a_scale + (int64_t)(m0 + (mine ? c0 + lane : 0)) * p.kb;
      float acc[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) acc[i] = 0.f;
      float sa[4], sw[4];
      const auto fetch = [&](int b) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sa[j] = mine && b + j < b1 ? asc[b + j] : 0.f;
          sw[j] = b + j < b1 ? wsc[b + j] : 0.f;
        }
      };
      fetch(b0);
      for (int b = b0; b < b1 && ok; b += 4) {
        float sc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = sa[j] * sw[j];
        fetch(b + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (b + j >= b1) break;
          const bool got = ptx::mbar_wait_cycles(&tfull[q], tph, abort_flag, kWaitLimit);
          if (!__all_sync(0xffffffffu, got)) {
            if (lane == 0) fail(6);
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + q * NT + c0;
#pragma unroll
          for (int c = 0; c < NC / 16; ++c) {
            float v[16];
            ptx::tmem_ld16(ta + c * 16, v);
            ptx::tmem_ld_wait16(v);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[c * 16 + i] = fmaf(v[i], __shfl_sync(0xffffffffu, sc[j], c * 16 + i), acc[c * 16 + i]);
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&tempty[q]);
          if (++q == NB) q = 0, tph ^= 1;
        }
      }
      if (split == 1) {
        const int n = n0 + quarter * 32 + lane;
        if (ok && n < p.N) {
          TO* o = static_cast<TO*>(p.out) + (int64_t)(m0 + c0) * p.ldo + n;
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (c0 + i < nm) store_out(o + (int64_t)i * p.ldo, acc[i]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (c0 + i < nm) red[(c0 + i) * 128 + quarter * 32 + lane] = acc[i];
      }
    }
    if (split > 1) {
      // every CTA adds the parts of its share of the tile's rows in rank order
      __syncwarp();
      ptx::cluster_sync();
      for (int u = threadIdx.x; u < nm * 32; u += C::kThreads) {
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
  if (warp == EW + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct Dev {
  int sms = 0;
  int pairs = 0;  // clusters of two CTAs of the wide kernel that run at the same time
  bool sm103 = false;
};

void cluster_config(cudaLaunchConfig_t* c, cudaLaunchAttribute* at, unsigned cluster, unsigned grid, unsigned threads,
                    unsigned smem, cudaStream_t s) {
  at->id = cudaLaunchAttributeClusterDimension;
  at->val.clusterDim.x = cluster;
  at->val.clusterDim.y = at->val.clusterDim.z = 1;
  c->gridDim = dim3(grid);
  c->blockDim = dim3(threads);
  c->dynamicSmemBytes = smem;
  c->stream = s;
  c->attrs = at;
  c->numAttrs = cluster > 1 ? 1 : 0;
}

// pairs of the wide kernel that fit the device at once
cudaError_t count_pairs(int sms, int* n) {
  using W = Wide<2, 64>;
  const void* f = (const void*)k_fp8_wide<2, 64, __nv_bfloat16>;
  if (const cudaError_t e = ensure_smem_limit(f, (int)W::kSmem); e != cudaSuccess) return e;
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at[1];
  cluster_config(&c, at, 2, (unsigned)(sms / 2 * 2), W::kThreads, W::kSmem, nullptr);
  const cudaError_t e = cudaOccupancyMaxActiveClusters(n, f, &c);
  *n = std::max(1, std::min(*n, sms / 2));
  return e;
}

// The wide kernel's warps trade registers among themselves: what the epilogue
// warps ask for has to be there, or they would wait for ever.
cudaError_t check_registers() {
  using W = Wide<2, 64>;  // the same for both types
  const void* kernels[] = {(const void*)k_fp8_wide<2, 64, __nv_bfloat16>, (const void*)k_fp8_wide<2, 64, float>};
  for (const void* f : kernels) {
    cudaFuncAttributes at;
    if (const cudaError_t e = cudaFuncGetAttributes(&at, f); e != cudaSuccess) return e;
    const int rest = W::kThreads / 32 - W::kEpiWarps;
    if (at.numRegs * W::kThreads < 32 * (W::kEpiWarps * W::kRegsHigh + rest * W::kRegsLow)) return cudaErrorNotSupported;
  }
  return cudaSuccess;
}

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
      if ((e = count_pairs(d.sms, &d.pairs)) != cudaSuccess) return e;
      if ((e = check_registers()) != cudaSuccess) return e;
    }
    cache[dev] = d;
    have[dev] = true;
  }
  *out = cache[dev];
  return cudaSuccess;
}

template <int NH, int EC, typename TO>
cudaError_t run_wide(const dspark_matmul_fp8_args& a, const MmParams& p, const Dev& d, cudaStream_t s) {
  using W = Wide<NH, EC>;
  CUtensorMap tmA, tmW, tmO = {};
  if (!tensor_map_2d(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a, a.K, a.M, a.lda, kKb, 128) ||
      !tensor_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, a.K, a.N, a.ldw, kKb, W::BN / 2))
    return cudaErrorInvalidValue;
  if (p.tma_out &&
      !tensor_map_2d(&tmO, sizeof(TO) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, a.out,
                     a.N, a.M, a.ldo * (int64_t)sizeof(TO), 128 / (int)sizeof(TO), 32, (int)sizeof(TO)))
    return cudaErrorInvalidValue;
  const int64_t tiles = (((int64_t)a.M + 255) / 256) * (((int64_t)a.N + W::BN - 1) / W::BN);
  if (tiles > INT32_MAX - d.pairs) return cudaErrorNotSupported;
  const void* f = (const void*)k_fp8_wide<NH, EC, TO>;
  if (const cudaError_t e = ensure_smem_limit(f, (int)W::kSmem); e != cudaSuccess) return e;
  const unsigned grid = 2 * (unsigned)std::min<int64_t>(tiles, d.pairs);
  if (const cudaError_t e = launch_overlapped(k_fp8_wide<NH, EC, TO>, grid, W::kThreads, W::kSmem, 1, s, tmA, tmW, tmO, p);
      e != cudaSuccess)
    return e;
  count_launches(1);
  return cudaGetLastError();
}

// Clusters of 2, 4 and 8 CTAs of the narrow kernel that the device runs at the
// same time (a cluster stays inside a group of SMs, so fewer than the SMs allow):
// looked up once per device.
struct Fit {
  int n[3];
};
template <int NT, typename TO>
cudaError_t clusters_fit(Fit* out) {
  constexpr int kMaxDev = 64;
  static Fit cache[kMaxDev];
  static bool have[kMaxDev] = {};
  static std::mutex mu;
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDev) return cudaErrorNotSupported;
  std::lock_guard<std::mutex> lock(mu);
  if (!have[dev]) {
    const void* f = (const void*)k_fp8_narrow<NT, TO>;
    for (int i = 0; i < 3; ++i) {
      const unsigned split = 2u << i, smem = Narrow<NT>::smem(true);
      if (const cudaError_t e = ensure_smem_limit(f, (int)smem); e != cudaSuccess) return e;
      cudaLaunchConfig_t c = {};
      cudaLaunchAttribute at[1];
      cluster_config(&c, at, split, split, Narrow<NT>::kThreads, smem, nullptr);
      if (const cudaError_t e = cudaOccupancyMaxActiveClusters(&cache[dev].n[i], f, &c); e != cudaSuccess) return e;
    }
    have[dev] = true;
  }
  *out = cache[dev];
  return cudaSuccess;
}

// CTAs of a cluster over K.  One CTA an SM: the largest cluster with which all run
// at the same time and each has a block at least (16 tiles of 64 rows, K = 4096: 7.2 us
// in clusters of 4 and 10.7 in clusters of 8, of which 15 fit).  With up to 16 rows two
// CTAs fit an SM (36 clusters of 8 and 74 of 4 ran at once, though the device's count is
// that of the other forms); that pays up to some 1.6 CTAs an SM, with two blocks or more
// a CTA.  Larger against next smaller cluster, over K = 1024 to 8192 and 1 to 16 rows:
// 20 tiles, 8 against 4: 5.5 and 5.5 us at K = 2560, 7.9 and 9.0 at 8192; 30 tiles: 5.6 to
// 6.3 and 5.8 to 6.3 at 2560, 8.9 and 10.0 at 8192 (but 5.1 and 4.8 at 1024, a block a CTA);
// 48 tiles, 4 against 2: 4.7 to 5.3 and 5.0 to 5.7 at 1024, 12.6 and 15.5 at 8192; past it 36 tiles,
// 8 against 4: 6.3 to 7.3 and 6.0 to 6.5 at 2560.  Clusters of 2 gain nothing there: 84
// tiles 5.9 against 5.4 undivided at 1024, 8.8 to 9.6 against 8.9 to 9.3 at 2560.
int narrow_split(int64_t tiles, int kb, int nt, int sms, const Fit& fit) {
  for (int i = 2; i >= 0; --i) {
    const int split = 2 << i;
    const int64_t ctas = tiles * split;
    if (nt <= 16 ? ctas <= sms || (split > 2 && 5 * ctas <= 8 * sms && kb >= 2 * split) : ctas <= sms && tiles <= fit.n[i])
      if (kb >= split) return split;
  }
  return 1;
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
  Fit fit;
  if (const cudaError_t e = clusters_fit<NT, TO>(&fit); e != cudaSuccess) return e;
  const int split = narrow_split(tiles, p.kb, NT, d.sms, fit);
  const uint32_t smem = C::smem(split > 1);
  const void* f = (const void*)k_fp8_narrow<NT, TO>;
  if (const cudaError_t e = ensure_smem_limit(f, (int)smem); e != cudaSuccess) return e;
  const unsigned grid = (unsigned)(split > 1 ? tiles * split : std::min<int64_t>(tiles, d.sms));
  const cudaError_t e =
      launch_overlapped(k_fp8_narrow<NT, TO>, grid, C::kThreads, smem, (unsigned)split, s, tmA, tmW, p, split, mt);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

template <typename TO>
cudaError_t run(const dspark_matmul_fp8_args& a, const MmParams& p, const Dev& d, cudaStream_t s) {
  if (a.M <= 16) return run_narrow<16, TO>(a, p, d, s);
  if (a.M <= 32) return run_narrow<32, TO>(a, p, d, s);
  if (a.M <= 64) return run_narrow<64, TO>(a, p, d, s);
  // few tiles and a long K: four CTAs or more a tile, or two where K is very long
  // (128 x 4096 x 1024: 7.2 against 10.1 us, 512 x 4096 x 512 7.6 against 10.1, 128 x 7168 x 4096
  // 14.4 against 16.1; not 128 x 2560 x 2560, 8.2 against 7.5)
  const int64_t few = ((a.M + 63) / 64) * (((int64_t)a.N + 127) / 128);
  if (a.M <= 512 && ((p.kb >= 16 && few * 4 <= d.sms) || (p.kb >= 48 && few * 2 <= d.sms)))
    return run_narrow<64, TO>(a, p, d, s);
  // waves of pairs times a tile's columns; a column of a 128-column tile costs
  // 1.25 of a 256-column tile's (2048 x 4096 x 151936: 1.06 ms, when this was 0.89), which
  // pays where the wider tiles leave pairs idle (512 x 4096 x 4096: 14.3 against
  // 24.8 us)
  const int64_t mt = ((int64_t)a.M + 255) / 256;
  const auto cost = [&](int bn) { return (double)((mt * ((a.N + bn - 1) / bn) + d.pairs - 1) / d.pairs * bn); };
  if (1.25 * cost(128) >= cost(256)) return run_wide<2, 64, TO>(a, p, d, s);
  if constexpr (sizeof(TO) == 4)
    if (!p.tma_out) return run_wide<1, 32, TO>(a, p, d, s);
  return run_wide<1, 64, TO>(a, p, d, s);
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
  if (((uintptr_t)a.out % 16) == 0 && (a.M == 1 || (a.ldo * esize) % 16 == 0))
    p.tma_out = ((int64_t)a.N * esize) % 16 == 0 ? 2 : 1;
  p.a_vec = ((uintptr_t)a.a_scale % 16) == 0;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  return a.out_dtype == DSPARK_BF16 ? run<__nv_bfloat16>(a, p, d, s) : run<float>(a, p, d, s);
}

}  // namespace dspark

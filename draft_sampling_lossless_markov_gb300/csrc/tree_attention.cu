// Attention of every request's drafted rows over its cached context and the drafted
// rows they descend from, read from the paged cache, on the tensor cores.
//
// An item is a request, a kv head and up to NQ of its columns: column c is row c / group
// of the request and query head c % group of the kv head.  An item runs over tiles of 128
// tokens.  Both products have the tokens' side large and the columns' side small, so the
// cache is the A operand and no tensor-core row is idle however few rows there are:
//     S [128 tokens, NQ]   = K tile . Q^T
//     O [D, NQ]           += (V tile)^T . P     (V read as it lies, MN-major)
// Tokens are the TMEM lanes of S: a lane's scales are one register each, and the weights
// are written as rows of the (MN-major) operand P by 16-byte stores.
//
// e4m3 codes are used as they are.  A column of q is scaled by a power of two and split
// into two e4m3 pieces whose sum is q exactly (8 significant bits; elements below 2^-10 of
// the column's largest to 2^-18 of it): S = K . Q1 + K . Q2.  A weight p times its
// token's v scale is split into three e5m2 pieces, 9 significant bits: the upper bytes of
// its fp16 form, of 2^3 times what they leave, and the rest rounded, times 2^3 again.
// Against a bf16 cache a weight is rounded to bf16, as both operands of a product have one type: 0.0019 of
// the norm off 64 bits, where weights of 32 bits leave the output's own 0.0016.
//
// Softmax: with y = score * log2 e + log2(v scale), weights are 2^(y - ref) about a
// column's reference, which is raised (O and the sums scaled down) only when a tile
// passes it by 2^15, and is set 2^6 below the largest then; fp16 holds 2^-24 to 2^16 of
// it, and the last piece's rounding is at most 2^-23, 2^-29 of the largest weight.  (e5m2
// ends at 2^-16: without the two factors weights below 2^-17 were lost, and with them a tail
// of 60000 tokens whose scores are 16 below a first one's.  The factors cost 1.5 %; the largest
// weight at 2^12 instead raises references so often that 256 x 8 rows take 441 us, not 369.)
// The sum of the weights themselves, 2^(y - ref) / (v scale), is kept by each lane in fp32;
// from a tile on in which a v scale is 0 or far from 1 (rows of zeros, cleared ones) its terms
// are formed from the scores alone, 2^(score * log2 e - a reference of the sum's own).
//
// A CTA is one pair of softmax warpgroups (two CTAs an SM) or two pairs, which take tiles in
// turn, each with its own references, sums and O, joined at the end of an item; a pair's
// warpgroups take half of the columns each.  Four more warps load, issue S, issue O and plan.
//
// The tiles of all items are one list, dealt out evenly to the CTAs with a fixed cost for
// each item: an item that several CTAs share leaves its parts in the workspace, and a second
// kernel joins them in order.
//
// What bounds it: the cache's bytes while a row's columns are few, the softmax's instructions
// beyond.  Of the measured copy rate it reads, with contexts that differ,
//     256 requests x 4 rows x 4 heads a kv head, e4m3, 128:  346 us, 0.95
//     256 requests x 8 rows x 4                              375 us, 0.89
//     one request x 8 rows x 4, 250001 tokens                 94 us, 0.83
//     64 requests x 16 rows x 4, bf16                        101 us, 0.80
//     16 requests x 64 rows x 8 (512 columns)                204 us, 0.09
// With 16, 32 and 64 columns a tile takes 1270, 1530 and 2490 cycles of an SM from L2; the
// loads alone would be 1455 at the copy rate.  A tile is some 1500 instructions and 15.5 for each
// column and warp of tokens, which at 64 columns fill 55 % of the issue slots; the tensor
// pipe is 18 % busy there.
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "kv_pool.cuh"
#include "launch.h"
#include "tc_ptx.cuh"
#include "tensor_map.h"

namespace dspark {

namespace {

constexpr int kTile = 128;           // tokens
constexpr int kMaxCtas = 320;        // parts the workspace holds: two a CTA
// A column's largest exponent when its reference is set, and the exponent that raises it: 2^15 is in
// fp16's range; bf16 weights stay below 1, as in a softmax, so that O overflows no sooner than the sum over v
// of weights up to 1 would.
template <bool kCodes>
constexpr float kHead = kCodes ? 6.f : -10.f;
template <bool kCodes>
constexpr float kRaise = kCodes ? 15.f : 0.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPiece = 8.f;  // a piece's factor over the one before, which leaves less than 2^12 of less than 2^15
// v scales with which the sums keep the weights' reference, 2^-40 to 2^38: a term is below 2^(15 + 40), and one whose
// weight rounds to 0 (below 2^-126) is below 2^-86 in a sum that holds one of 2^(6 - 38) or more.
constexpr uint32_t kLeastScale = (127u - 40) << 23, kMostScale = (127u + 38) << 23;
constexpr float kLeastNormal = 1.1754943508222875e-38f;
constexpr float kRaiseSum = 60.f;  // the exponent that raises a sum's own reference

// An item that begins in a CTA and goes on in others: where its rows and columns are, and its parts (0: there is
// none).  first: the CTA that the item of this CTA's first part begins in, -1 if that is this one.
struct Shared {
  int32_t lo, head, col0, columns, parts, first;
};

static_assert((64ll * kMaxTreeGroup + 64) * kMaxTreeGroup < 1ll << 32, "columns divided by a multiplication");
struct TreeArgs {
  KvPool pool;
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const int32_t* offsets;
  const int32_t* base;
  const uint64_t* tree;
  int64_t ldq, ldo;
  int32_t N, group, max_tree;
  // ceil(2^32 / group): c / group is c group_inv >> 32 for the columns c < 64 group + 64, as c group
  // is below 2^32 (kMaxTreeGroup)
  uint64_t group_inv;
  float scale;
  WsHeader* hdr;
  Shared* meta;   // [CTAs]
  float4* stat;   // [2 CTAs, NQ] a part's references, sums and the sums' references
  float* part;    // [2 CTAs, NQ, D] a part's O
};

template <bool kCodes, int D, int NQ>
struct Form {
  static constexpr int kColumns = NQ;
  // What an item costs beside its tiles, in tiles (3, 4, 5, 6, 8, 10 tried, head sizes 128 and 64, long and short contexts:
  // 16 requests x 64 nodes 234, 209, 203, 203, 207, 213 us, 256 x 8 rows 380, 374, 376, 378, 382, 388, at head size 64
  // 349, 342, 343, 346, 352, 358, 64 x 16 rows bf16 132, 120, 113, 109, 104, 105, at head size 64 100, 92, 86, 84, 77, 80)
  static constexpr int kItemCost = NQ < 64 ? 4 : kCodes ? 5 : 8;
  // Sums with references of their own in line, where the registers do without: with a row of zeros in a thousand 256 x 8
  // rows take 470 us, and 1340 through a function's arguments in local memory (376 us without such rows, either way);
  // in line at 64 columns 16 x 64 nodes go from 203 to 223 us, at head size 64 256 x 8 rows from 344 to 354.
  static constexpr bool kApartInline = kCodes && D == 128 && NQ <= 32;
  static constexpr int kElem = kCodes ? 1 : 2;
  static constexpr int kRow = D * kElem < 128 ? D * kElem : 128;  // bytes of an operand row
  static constexpr int kParts = D * kElem / kRow;                 // of a token's row
  static constexpr uint32_t kPart = kTile * kRow;
  static constexpr uint32_t kOperand = kPart * kParts;            // a tile of k or v
  static constexpr int kQPieces = kCodes ? 2 : 1, kPPieces = kCodes ? 3 : 1;
  static constexpr uint32_t kQPart = NQ * kRow;
  static constexpr uint32_t kQ = kQPart * kParts * kQPieces;
  // P's rows: the pieces side by side in 128 bytes; of 64 columns the third in rows of 64 bytes behind them
  static constexpr int kPWide = NQ * kPPieces * kElem <= 128 ? NQ * kPPieces : 128 / kElem;
  static constexpr int kPRest = NQ * kPPieces - kPWide;
  static constexpr uint32_t kPCol = kTile * 128;
  static constexpr uint32_t kP = kPCol + (kPRest > 0 ? kTile * 64 : 0);
  static constexpr uint32_t kScales = kCodes ? 2 * kTile * 4 : 0;
  static constexpr int kO = NQ * kPPieces;                         // columns of O: the pieces side by side
  // One pair of warpgroups a CTA and two CTAs an SM where they fit (what one waits for at an item's end
  // the other fills), else two pairs a CTA.  q of this part of an item and of the next.
  static constexpr bool kSmall = NQ <= 32 && kP + 2 * kQ + 4 * kOperand + 2 * kScales <= 104 * 1024 && NQ + kO <= 256;
  static constexpr int kPairs = kSmall ? 1 : 2;
  // Tiles of k and of v have rings of their own: one of k is free again as soon as S is formed (with one
  // ring a tile's loads waited for O two tiles before: 256 x 8 rows 415 us, with two 382).  What the softmax reads, scales and the pages that
  // are there, has a ring of kNotes: when k of tile n is loaded, S of tile n - kStagesK has been formed, so
  // S of every tile up to n - kStagesK - 3 has been read.
  static constexpr int kNotes = 8;
  static constexpr uint32_t kFixed = kPairs * kP + 2 * kQ + kNotes * kScales;
  static constexpr int kSlots = (int)std::min<uint32_t>(10, ((kSmall ? 106 : 212) * 1024 - kFixed) / kOperand);
  static constexpr int kStagesK = kSlots / 2, kStagesV = kSlots - kStagesK;
  static constexpr uint32_t kSmem = kFixed + kSlots * kOperand + 1024;
  static constexpr int kCols = kPairs * (NQ + kO);                 // S and O of the pairs
  static constexpr uint32_t kTmemCols = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static constexpr int kSoftWarps = 8 * kPairs, kSoft = 32 * kSoftWarps;
  static constexpr int kThreads = kSoft + 128;                     // and the warps for loads, S, O and q
  static constexpr int kCtas = kSmall ? 2 : 1;                     // an SM
  // registers of the softmax's threads and of the others, of the 80 or 96 a thread at launch
  static constexpr int kRegs = kSmall ? 80 : 96, kRegsHigh = kSmall ? 96 : 104, kRegsLow = kSmall ? 48 : 64;
  static_assert(kSoft * kRegsHigh + 128 * kRegsLow <= kThreads * kRegs, "registers");
  static_assert(kStagesK >= 2 && kStagesK + 3 <= kNotes && kCols <= 512 && kCtas * kTmemCols <= 512, "shared memory and TMEM");
};

template <int kRow>
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lbo) {
  return kRow == 128 ? ptx::smem_desc_sw128(addr, lbo, 1024) : ptx::smem_desc_sw64(addr, lbo, 512);
}
// the place of byte `a` of an operand with rows of kRow bytes
template <int kRow>
__device__ __forceinline__ uint32_t swizzled(uint32_t a) {
  return a ^ ((a >> 3) & (kRow == 128 ? 0x70u : 0x30u));
}

// A request's rows and tiles; its units are the costs of all its items: their tiles, behind the units of an item itself.
struct Request {
  int32_t lo, rows, base, tiles, chunks;
  int64_t units;
};
template <typename F>
__device__ __forceinline__ Request request_at(const TreeArgs& a, int r, bool* bad) {
  Request q;
  const int32_t lo = a.offsets[r], hi = a.offsets[r + 1];
  q.base = a.base[r];
  const int64_t held = (int64_t)q.base + hi - lo;
  *bad = lo < 0 || hi < lo || hi > a.N || hi - lo > a.max_tree || q.base < 0 ||
         held > (int64_t)a.pool.max_pages << a.pool.shift;
  q.lo = lo;
  q.rows = *bad ? 0 : hi - lo;
  q.tiles = q.rows ? (int32_t)((held + kTile - 1) / kTile) : 0;
  q.chunks = (q.rows * a.group + F::kColumns - 1) / F::kColumns;
  q.units = q.tiles ? (int64_t)(q.tiles + F::kItemCost) * q.chunks * a.pool.heads : 0;
  return q;
}

// Where a CTA's share begins: the request, the item and the unit within it.
struct Start {
  int r, head, chunk, x;
  Request q;
};
// (32-bit division where the numbers allow: a 64-bit one takes some 300 cycles)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// The parts of items in a CTA's share of the units, one after the other; the warps that need them walk by themselves.
template <typename F>
struct Walk {
  int r, head, chunk, x;  // the next unit: x of that item
  int64_t left;           // units
  Request q;
  // the part
  int tile, tiles;    // first tile, their number
  bool begins, ends;  // the item's first and last tile are in it
  __device__ __forceinline__ void start(const Start& at, int64_t n) {
    left = n;
    if (n > 0) r = at.r, head = at.head, chunk = at.chunk, x = at.x, q = at.q;
  }
  __device__ __forceinline__ bool next(const TreeArgs& a, volatile int* state) {
#pragma unroll 1
    while (left > 0) {
      if (x == q.tiles + F::kItemCost) {
        x = 0;
        if (++chunk == q.chunks) {
          chunk = 0;
          if (++head == a.pool.heads) {
            head = 0;
            do {
              if (++r >= a.pool.n_req) return false;
              ptx::mbar_progress(state);  // there may be any number of empty ones
              bool bad;
              q = request_at<F>(a, r, &bad);
            } while (q.units == 0);
          }
        }
      }
      const int y = (int)min((int64_t)(q.tiles + F::kItemCost), x + left);
      tile = max(0, x - F::kItemCost);
      tiles = max(0, y - F::kItemCost) - tile;
      left -= y - x;
      x = y;
      if (tiles == 0) continue;  // nothing but the item's own cost: it begins in the next CTA
      begins = tile == 0;
      ends = tile + tiles == q.tiles;
      return true;
    }
    return false;
  }
};

// A part as the planning warp hands it on; no tiles: the last was the one before.
struct Part {
  int32_t r, lo, base, rows, head, tile, tiles, col0, columns;  // col0: the chunk's first column
  int32_t slot;                                                 // of the workspace; -1: the item is whole
};
constexpr int kPlans = 4;  // parts planned ahead

// x, which the compiler does not know: a loop whose first round is special is not cut in two (the copy
// would be fetched anew for every part)
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

// v[i] combined over the warp's lanes: lane l ends with column l % n's
template <int n, typename Op>
__device__ __forceinline__ float over_lanes(float (&v)[n], Op op) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o >= n; o >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] = op(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1) {
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float mine = (lane & o) ? v[i + o] : v[i], send = (lane & o) ? v[i] : v[i + o];
      v[i] = op(mine, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return v[0];
}

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }
__device__ __forceinline__ __half2 bits_half2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t e5m2x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
// what the upper bytes of two halves leave of them, times the next piece's factor
__device__ __forceinline__ uint32_t left_of(uint32_t h) {
  return half2_bits(__hmul2(__hsub2(bits_half2(h), bits_half2(h & 0xFF00FF00u)), __float2half2_rn(kPiece)));
}
__device__ __forceinline__ uint32_t e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ __half2 e4m3x2_halves(uint32_t c) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3));
}
// a word's non-finite elements: all ones in their place
template <bool kCodes>
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
  if (kCodes) return ((((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 255u;
  return ((((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u) >> 15) * 65535u;
}

// q of a part as operand pieces, eight lanes a column: this lane's elements (16 or 8) of column c.
template <int D>
struct QColumn {
  static constexpr int E = D / 8, V = E / 8;
  uint4 v[V];
  __device__ __forceinline__ void load(const TreeArgs& a, const Part& p, int c) {
    const int col = p.col0 + c, j = (int)((uint32_t)col * a.group_inv >> 32);
    const __nv_bfloat16* src =
        a.q + (int64_t)(p.lo + j) * a.ldq + (p.head * a.group + col - j * a.group) * D + (threadIdx.x & 7) * E;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = c < p.columns ? *reinterpret_cast<const uint4*>(src + i * 8) : make_uint4(0, 0, 0, 0);
  }
  // to the operand at dst, the column's factor and its place in out
  template <bool kCodes, int NQ>
  __device__ __forceinline__ void store(const TreeArgs& a, const Part& p, int c, uint8_t* dst, float* qs, int64_t* out_at) {
    using F = Form<kCodes, D, NQ>;
    const int l = threadIdx.x & 7;
    uint32_t* x = reinterpret_cast<uint32_t*>(v);
    uint32_t top = 0;  // the largest magnitude's bits; infinities and NaN are above all others
#pragma unroll
    for (int i = 0; i < E / 2; ++i) top = __vmaxu2(top, x[i] & 0x7FFF7FFFu);
    top = max(top & 0xFFFFu, top >> 16);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool fin = top < 0x7F80u;
    if (!fin) {  // the column's scores are NaN through its factor
#pragma unroll
      for (int i = 0; i < E / 2; ++i) x[i] = 0;
      top = 0;
    }
    float unit = a.scale * kLog2e;
    if constexpr (kCodes) {
      // top 2^k in 128 .. 256, k up to 120 so that both powers are normal
      const int k = top ? min(7 - ((int)(top >> 7) - 127), 120) : 0;
      const float up = __uint_as_float((uint32_t)(127 + k) << 23);
      unit *= __uint_as_float((uint32_t)(127 - k) << 23);
      uint32_t p1[E / 4], p2[E / 4];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {  // below 2^8 the eight bits are exact in fp16, whose step is 2^-24 at the bottom
        const __half2 y = __floats2half2_rn(__uint_as_float(x[i] << 16) * up, __uint_as_float(x[i] & 0xFFFF0000u) * up);
        const uint32_t c1 = e4m3x2(half2_bits(y));
        const uint32_t c2 = e4m3x2(half2_bits(__hsub2(y, e4m3x2_halves(c1))));
        p1[i / 2] = (i & 1) ? __byte_perm(p1[i / 2], c1, 0x5410) : c1;
        p2[i / 2] = (i & 1) ? __byte_perm(p2[i / 2], c2, 0x5410) : c2;
      }
      const uint32_t at = swizzled<F::kRow>(c * F::kRow + l * E);
      if constexpr (E == 16) {
        *reinterpret_cast<uint4*>(dst + at) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
        *reinterpret_cast<uint4*>(dst + F::kQPart + at) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
      } else {
        *reinterpret_cast<uint2*>(dst + at) = make_uint2(p1[0], p1[1]);
        *reinterpret_cast<uint2*>(dst + F::kQPart + at) = make_uint2(p2[0], p2[1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int byte = l * E * 2 + i * 16;
        *reinterpret_cast<uint4*>(dst + byte / F::kRow * F::kQPart + swizzled<F::kRow>(c * F::kRow + byte % F::kRow)) = v[i];
      }
    }
    if (l == 0) {
      const int col = p.col0 + c, j = (int)((uint32_t)col * a.group_inv >> 32);
      qs[c] = c < p.columns ? (fin ? unit : NAN) : 0.f;
      out_at[c] = (int64_t)(p.lo + j) * a.ldo + (p.head * a.group + col - j * a.group) * D;
    }
  }
};

template <int n>
__device__ __forceinline__ void load_columns(uint32_t taddr, float* v) {
#pragma unroll
  for (int i = 0; i < n; i += 8) ptx::tmem_ld8(taddr + i, v + i);
}
// eight columns of O, its pieces summed (the smallest first)
template <int kPieces>
__device__ __forceinline__ void load_sum(uint32_t taddr, int apart, float (&v)[8]) {
  float u[kPieces][8];
#pragma unroll
  for (int p = 0; p < kPieces; ++p) ptx::tmem_ld8(taddr + p * apart, u[p]);
#pragma unroll
  for (int p = 0; p < kPieces; ++p) ptx::tmem_ld_wait<8>(u[p]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = u[kPieces - 1][i];
#pragma unroll
    for (int p = kPieces - 2; p >= 0; --p) v[i] = fmaf(v[i], 1.f / kPiece, u[p][i]);
  }
}

// Sums with references of their own take the weights of the scores alone: their exponents are x = y - ref, less log2 of
// the v scale and by the difference of the references (at).  v_inv is the scale's inverse, or the scale negated where it
// is far from 1.
__device__ __forceinline__ bool zero_scale(float v_inv) { return !(v_inv > 0.f) && -v_inv < kLeastNormal; }
__device__ __forceinline__ float less_scale(float v_inv) {
  const float v = fabsf(v_inv), log = __log2f(zero_scale(v_inv) ? kLeastNormal : v);
  return !(v == v) ? 0.f : v_inv > 0.f ? log : -log;  // (NaN is in x where the token is seen)
}
__device__ __forceinline__ float2 sum_exponents(uint64_t x, float less, const float* at) {
  return ptx::unpack2(ptx::add2(x, ptx::add2(ptx::pack2(less, less), *reinterpret_cast<const uint64_t*>(at))));
}
template <int HQ>
__device__ __forceinline__ float highest_apart(const uint64_t (&x)[HQ / 2], float v_inv, const float* at) {
  const float less = less_scale(v_inv);
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < HQ / 2; ++i) {
    const float2 e = sum_exponents(x[i], less, at + 2 * i);
    top = fmaxf(top, fmaxf(e.x, e.y));
  }
  return top;
}
template <int HQ>
__device__ __forceinline__ void add_apart(uint64_t (&x)[HQ / 2], uint64_t (&l)[HQ / 2], float v_inv, const float* at) {
  const float less = less_scale(v_inv);
  const bool zero = zero_scale(v_inv);
#pragma unroll
  for (int i = 0; i < HQ / 2; ++i) {
    const float2 e = sum_exponents(x[i], less, at + 2 * i);
    l[i] = ptx::add2(l[i], ptx::pack2(ptx::ex2(e.x), ptx::ex2(e.y)));
    if (zero) x[i] = ptx::pack2(-INFINITY, -INFINITY);  // codes of scale 0 are 0
  }
}
// the same with the references raised first (set: there is one; top: room for each warp's largest)
template <int HQ>
__device__ __forceinline__ void raise_apart(uint64_t (&x)[HQ / 2], uint64_t (&l)[HQ / 2], float v_inv, float* at,
                                            float* factor, bool* set, float (*top)[HQ], int bar) {
  const int lane = threadIdx.x & 31, token = threadIdx.x & 127;
  const float less = less_scale(v_inv);
  const bool zero = zero_scale(v_inv);
  float m = -INFINITY;  // of column `lane`
#pragma unroll
  for (int i = 0; i < HQ / 2; ++i) {
    const float2 e = sum_exponents(x[i], less, at + 2 * i);
    const float m0 = ptx::warp_max_redux(e.x), m1 = ptx::warp_max_redux(e.y);
    m = lane == 2 * i ? m0 : lane == 2 * i + 1 ? m1 : m;
  }
  if (lane < HQ) top[token / 32][lane] = m;
  ptx::named_sync(bar, 128);
  if (token < HQ) {
    m = fmaxf(fmaxf(top[0][token], top[1][token]), fmaxf(top[2][token], top[3][token]));
    const bool was = set[token];
    const float d = (was ? m > kRaiseSum : m > -INFINITY) ? m : 0.f;
    set[token] = was || m > -INFINITY;
    at[token] -= d;
    factor[token] = was ? ptx::ex2(-d) : 1.f;  // (a sum without a reference is 0 or NaN)
  }
  ptx::named_sync(bar, 128);
#pragma unroll
  for (int i = 0; i < HQ / 2; ++i) {
    const float2 e = sum_exponents(x[i], less, at + 2 * i);
    l[i] = ptx::fma2(l[i], *reinterpret_cast<const uint64_t*>(&factor[2 * i]), ptx::pack2(ptx::ex2(e.x), ptx::ex2(e.y)));
    if (zero) x[i] = ptx::pack2(-INFINITY, -INFINITY);  // codes of scale 0 are 0
  }
}

template <int HQ>
__device__ __noinline__ void raise_apart_out_of_line(uint64_t (&x)[HQ / 2], uint64_t (&l)[HQ / 2], float v_inv, float* at,
                                                     float* factor, bool* set, float (*top)[HQ], int bar) {
  raise_apart<HQ>(x, l, v_inv, at, factor, set, top, bar);
}

// What turns O into the result is 2^(O's reference less the sum's) / sum, 0 where nothing was summed, as two factors:
// neither they nor O times the first leave fp32's normal range where the result does not.
__device__ __forceinline__ float2 inverse(float sum, float apart) {
  const float half = sum == 0.f ? 0.f : ptx::ex2(0.5f * apart);
  return make_float2(sum == 0.f ? 0.f : __frcp_rn(sum) * half, half);
}

// Adds the non-finite elements of v that columns c0 .. c1 see of the drafted rows `nodes` to what was
// written for them (element d of the head).
template <bool kCodes, int D, int NQ>
__device__ __noinline__ void add_non_finite(const TreeArgs& a, const Part& p, const uint64_t* seers, const int64_t* out_at,
                                            unsigned long long nodes, int c0, int c1, int d) {
  for (; nodes; nodes &= nodes - 1) {
    const int node = __ffsll((long long)nodes) - 1;
    const int32_t row = pool_row(a.pool, p.r, (int64_t)p.base + node);
    if (row < 0) continue;
    const int64_t at = ((int64_t)row + ((int64_t)p.head << a.pool.shift)) * D + d;
    const float x = kCodes ? ((a.pool.v[at] & 0x7F) == 0x7F ? NAN : 0.f)
                           : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(a.pool.v)[at]);
    if (fabsf(x) < INFINITY) continue;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      if (!((seers[node] >> c) & 1)) continue;
      if (p.slot < 0) {
        __nv_bfloat16* o = a.out + out_at[c] + d;
        *o = __float2bfloat16_rn(__bfloat162float(*o) + x);
      } else {
        a.part[((int64_t)p.slot * NQ + c) * D + d] += x;
      }
    }
  }
}

template <bool kCodes, int D, int NQ>
__global__ void __launch_bounds__(Form<kCodes, D, NQ>::kThreads, Form<kCodes, D, NQ>::kCtas)
    k_tree_attention(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ TreeArgs a) {
  using F = Form<kCodes, D, NQ>;
  constexpr int kSoftWarps = F::kSoftWarps, kSoft = F::kSoft, kThreads = F::kThreads, kPairs = F::kPairs;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sP = sm;                  // [pairs] P
  uint8_t* sQ = sm + kPairs * F::kP;  // [2][pieces][parts]
  uint8_t* sK = sm + F::kFixed;  // [stages] tiles
  uint8_t* sV = sK + F::kStagesK * F::kOperand;
  float* sScale = reinterpret_cast<float*>(sQ + 2 * F::kQ);  // [notes] of k, of v
  __shared__ uint64_t kfull[F::kStagesK], kempty[F::kStagesK], noted[F::kNotes], vfull[F::kStagesV], vempty[F::kStagesV], sfull[kPairs], sfree[kPairs],
      pready[kPairs], pdone[kPairs], qfull[2], planned[kPlans], ended[kPlans];
  __shared__ uint32_t tmem_slot, okmask[F::kNotes];
  __shared__ int abort_s[2], never_s[2];  // mbar_wait_paced
  __shared__ Start start;
  __shared__ int64_t sums[kThreads / 32 + 1];
  // the parts planned and the columns that see each drafted row; of this part and the next the drafted rows
  // with non-finite v, each column's place in out and its factor
  __shared__ Part parts[kPlans];
  __shared__ uint64_t seers[kPlans][DSPARK_MAX_TREE];
  __shared__ unsigned long long hidden[2];
  __shared__ int64_t out_at[2][NQ];
  __shared__ __align__(16) float qs[2][NQ];
  __shared__ __align__(16) float nref[kPairs][NQ], delta[kPairs][NQ], factor[kPairs][NQ];
  __shared__ float warp_top[kSoftWarps][NQ / 2], coef[kPairs][NQ], unit[NQ];
  __shared__ bool set[kPairs][NQ];
  // the sums' references: whether there is one, and how far below the weights' it is (0 while they share it)
  __shared__ bool sum_set[kPairs][NQ];
  __shared__ __align__(16) float sum_at[kPairs][NQ];
  __shared__ bool odd_scale[kPairs][2];  // a warpgroup has met a v scale far from 1 in this part
  volatile int* abort_flag = abort_s;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < F::kStagesK; ++i) {
      ptx::mbar_init(&kfull[i], 1);
      ptx::mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < F::kNotes; ++i) ptx::mbar_init(&noted[i], kCodes ? 33 : 1);  // and every lane's copies of scales
    for (int i = 0; i < F::kStagesV; ++i) {
      ptx::mbar_init(&vfull[i], 1);
      ptx::mbar_init(&vempty[i], 1);
    }
    for (int i = 0; i < kPairs; ++i) {
      ptx::mbar_init(&sfull[i], 1);
      ptx::mbar_init(&sfree[i], 8);
      ptx::mbar_init(&pready[i], 8);
      ptx::mbar_init(&pdone[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&qfull[i], kSoftWarps);
      hidden[i] = 0;
    }
    for (int i = 0; i < kPlans; ++i) {
      ptx::mbar_init(&planned[i], 1);
      ptx::mbar_init(&ended[i], kSoftWarps);
    }
    ptx::fence_mbar_init();
    abort_s[0] = never_s[0] = 0;
    ptx::mbar_progress(abort_s);
    ptx::prefetch_map(&tmK);
    ptx::prefetch_map(&tmV);
  }
  if (warp == kSoftWarps + 1) {
    ptx::tmem_alloc(&tmem_slot, F::kTmemCols);
    ptx::tmem_relinquish();
  }
  ptx::launch_dependents();
  ptx::grid_wait();
  auto fail = [&](int what) { *abort_flag = what; };  // reported at the end

  // this CTA's share of the units: a scan over the requests, a run of them a thread
  const int per = (a.pool.n_req + kThreads - 1) / kThreads, from = threadIdx.x * per, to = min(a.pool.n_req, from + per);
  int64_t mine = 0;
  Request q;  // the run's last
  q.units = 0;
#pragma unroll 1
  for (int r = from; r < to; ++r) {
    bool bad;
    q = request_at<F>(a, r, &bad);
    mine += q.units;
    if (bad && blockIdx.x == 0 && a.hdr) report_error(a.hdr, DSPARK_BAD_INPUT, r);
  }
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  if (lane == 31) sums[warp] = before;
  before -= mine;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
  int64_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  const int ctas = (int)min((int64_t)gridDim.x, total), cta = blockIdx.x;
  // CTA c's units: an even share, the first total % ctas of the CTAs one more
  const int64_t each = ctas ? quotient(total, ctas) : 0, rest = total - each * ctas;
  const int64_t u0 = cta < ctas ? each * cta + min((int64_t)cta, rest) : 0;
  const int64_t u1 = cta < ctas ? u0 + each + (cta < rest) : 0;
  if (u1 > u0 && before <= u0 && u0 < before + mine) {
    int r = from;
    int64_t at = u0 - before;
#pragma unroll 1
    for (; r < to - 1; ++r) {
      bool bad;
      const Request p = request_at<F>(a, r, &bad);
      if (at < p.units) {
        q = p;
        break;
      }
      at -= p.units;
    }
    const int cost = q.tiles + F::kItemCost;
    const int64_t item = quotient(at, cost);
    start = Start{r, (int)((uint32_t)item / (uint32_t)q.chunks), (int)((uint32_t)item % (uint32_t)q.chunks), (int)(at - item * cost), q};
  }
  if (threadIdx.x == 0) {
    a.meta[cta].parts = 0;
    a.meta[cta].first = -1;
    ptx::mbar_progress(abort_flag);
  }
  __syncthreads();
  Walk<F> walk;
  walk.start(start, u1 - u0);
  if (warp >= kSoftWarps) {
  ptx::reg_dec<F::kRegsLow>();
  if (warp == kSoftWarps) {
    // ---- loads: a lane a page of k or v, four tokens' scales a lane; the page numbers a tile ahead, v a
    // tile behind k but at a part's end ----
    const uint64_t policy = a.group * a.max_tree > NQ ? ptx::policy_evict_normal() : ptx::policy_evict_first();
    const int box_shift = min(a.pool.shift, 7), box = 1 << box_shift, boxes = kTile >> box_shift;
    const int i = lane & 7;
    uint32_t n = 0, nv = 0;  // tiles of k, of v
    uint32_t sk = 0, phk = 1, sv = 0, phv = 1;
    int32_t row = -1;        // of the lane's page (lanes 0-7: k, 8-15: v), of the last tile of k
    uint32_t bytes = 0;
    bool ok = true;
    const auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait_paced(bar, parity, abort_flag));
      if (!ok && lane == 0) fail(1);
      return ok;
    };
    const auto load = [&](uint8_t* tile, const CUtensorMap* map, uint64_t* full) {
#pragma unroll
      for (int p = 0; p < F::kParts; ++p)
        ptx::tma_load_2d(tile + p * F::kPart + i * box * F::kRow, map, full, p * (F::kRow / F::kElem), row, policy);
    };
    const auto load_v = [&] {
      if (!wait(&vempty[sv], phv)) return;
      if (lane == 0) ptx::mbar_expect_tx(&vfull[sv], bytes);
      __syncwarp();
      if (row >= 0 && lane >= 8 && lane < 16) load(sV + sv * F::kOperand, &tmV, &vfull[sv]);
      __syncwarp();
      ++nv;
      if (++sv == (uint32_t)F::kStagesV) sv = 0, phv ^= 1;
    };
    while (ok && walk.next(a, abort_flag)) {
      const int len = walk.q.base + walk.q.rows;
      const int32_t* table = a.pool.table + walk.r * a.pool.table_ld;
      int pos = walk.tile * kTile + (i << box_shift);
      // (positions below len have an entry: request_at)
      int32_t page = i < boxes && pos < len ? table[pos >> a.pool.shift] : -1;
#pragma unroll 1
      for (int t = 0; t < walk.tiles; ++t) {
        const int32_t here = page, at = pos;
        pos += kTile;
        page = i < boxes && pos < len && t + 1 < walk.tiles ? table[pos >> a.pool.shift] : -1;
        if (!wait(&kempty[sk], phk)) break;
        const bool wanted = i < boxes && at < len;
        const bool live = wanted && here >= 0 && here < a.pool.n_pages;
        if (wanted && !live && a.hdr) report_error(a.hdr, DSPARK_BAD_INPUT, walk.r);
        const int32_t row_v = row;
        const uint32_t bytes_v = bytes;
        row = live ? ((here * a.pool.heads + walk.head) << a.pool.shift) + (at & ((1 << a.pool.shift) - 1)) : -1;
        const uint32_t mask = __ballot_sync(0xffffffffu, live) & 0xFFu;
        bytes = __popc(mask) * (box * D * F::kElem);
        if (lane == 0) {
          ptx::mbar_progress(abort_flag);
          ptx::mbar_expect_tx(&kfull[sk], bytes);
          okmask[n % F::kNotes] = mask;
          ptx::mbar_arrive(&noted[n % F::kNotes]);
        }
        __syncwarp();
        if (live && lane < 8) load(sK + sk * F::kOperand, &tmK, &kfull[sk]);
        if constexpr (kCodes) {
          const int32_t from = __shfl_sync(0xffffffffu, row, (4 * lane) >> box_shift);
          if (from >= 0) {
            const int32_t first = from + ((4 * lane) & (box - 1));
            float* dst = sScale + n % F::kNotes * 2 * kTile + 4 * lane;
            ptx::cp_async16_cg(dst, a.pool.k_scale + first);
            ptx::cp_async16_cg(dst + kTile, a.pool.v_scale + first);
          }
          ptx::cp_async_arrive(&noted[n % F::kNotes]);
        }
        __syncwarp();
        ++n;
        if (++sk == (uint32_t)F::kStagesK) sk = 0, phk ^= 1;
        if (t > 0) {  // v of the tile before
          const int32_t row_k = row;
          const uint32_t bytes_k = bytes;
          row = row_v, bytes = bytes_v;
          load_v();
          row = row_k, bytes = bytes_k;
        }
        if (t + 1 == walk.tiles) load_v();
        if (!ok) break;
      }
    }
    // nothing may be in flight when the CTA leaves
    ptx::mbar_progress(never_s);
    for (uint32_t j = n > (uint32_t)F::kNotes ? n - F::kNotes : 0; kCodes && j < n; ++j)
      ptx::mbar_wait_paced(&noted[j % F::kNotes], (j / F::kNotes) & 1, never_s);
    for (uint32_t j = n > (uint32_t)F::kStagesK ? n - F::kStagesK : 0; j < n; ++j)
      ptx::mbar_wait_paced(&kfull[j % F::kStagesK], (j / F::kStagesK) & 1, never_s);
    for (uint32_t j = nv > (uint32_t)F::kStagesV ? nv - F::kStagesV : 0; j < nv; ++j)
      ptx::mbar_wait_paced(&vfull[j % F::kStagesV], (j / F::kStagesV) & 1, never_s);
    __syncwarp();
  } else if (warp < kSoftWarps + 3) {
    // ---- MMAs: one warp for S, up to two tiles ahead, and one for O (one warp's waits and issues for
    // both took 1850 cycles a tile) ----
    constexpr uint32_t idesc_s = kCodes ? ptx::idesc_e4m3_f32(128, NQ) : ptx::idesc_bf16_f32(128, NQ, false, false);
    constexpr uint32_t idesc_o = kCodes ? ptx::idesc_e4m3_e5m2_mn_f32(128, F::kPWide) : ptx::idesc_bf16_f32(128, NQ, true, true);
    constexpr int kStepsS = D * F::kElem / 32, kStepTokens = 32 / F::kElem, kStepsO = kTile / kStepTokens;
    // of D = 64 the tile's 64 columns serve as both halves of the 128 rows
    constexpr uint32_t kLboV = F::kParts > 1 ? F::kPart : 0;
    // descriptors of the first stage and buffer; all others are so many 16-byte units further
    const uint64_t dk0 = operand_desc<F::kRow>(ptx::smem_u32(sK), 16);
    const uint64_t dv0 = operand_desc<F::kRow>(ptx::smem_u32(sV), kLboV);
    const uint64_t dq0 = operand_desc<F::kRow>(ptx::smem_u32(sQ), 16);
    const uint64_t dp0 = ptx::smem_desc_sw128(ptx::smem_u32(sP), 16, 1024);
    const uint64_t dr0 = ptx::smem_desc_sw64(ptx::smem_u32(sP) + F::kPCol, 16, 512);
    const bool is_s = warp == kSoftWarps + 1;
    const uint32_t stages = is_s ? F::kStagesK : F::kStagesV;
    auto wait = [&](uint64_t* bar, uint32_t parity, int what) {
      const bool got = __all_sync(0xffffffffu, ptx::mbar_wait_paced(bar, parity, abort_flag));
      if (!got && lane == 0) fail(what);
      return got;
    };
    uint32_t s = 0, ph = 0, turns = 0;  // the tile's stage and phase, the phases of the pairs of warpgroups
    bool ok = true;
    for (uint32_t part = 0; ok; ++part) {
      const int qb = part & 1;
      ok = wait(&qfull[qb], (part >> 1) & 1, 2);
      if (!ok) break;
      const int tiles = parts[part % kPlans].tiles;
      if (tiles == 0) break;
      for (int t = 0; t < tiles; ++t) {
        const int w = t % kPairs;
        if (is_s) {
          ok = wait(&sfree[w], (~turns >> w) & 1, 3) && wait(&kfull[s], ph, 4);
          if (!ok) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint64_t dk = dk0 + s * (F::kOperand >> 4), dq = dq0 + qb * (F::kQ >> 4);
            const uint32_t d = tmem + w * NQ;
#pragma unroll
            for (int p = 0; p < F::kQPieces; ++p)
#pragma unroll
              for (int k = 0; k < kStepsS; ++k) {
                const int row = k * 32 / F::kRow, off = k * 32 % F::kRow;
                const uint64_t da = dk + ((row * F::kPart + off) >> 4), db = dq + (((p * F::kParts + row) * F::kQPart + off) >> 4);
                if constexpr (!kCodes)
                  ptx::tc_mma(d, da, db, idesc_s, k > 0);
                else if (p + k == 0)
                  ptx::tc_mma_fp8<0>(d, da, db, idesc_s);
                else
                  ptx::tc_mma_fp8<1>(d, da, db, idesc_s);
              }
            ptx::tc_commit(&sfull[w]);
            ptx::tc_commit(&kempty[s]);
          }
        } else {
          ok = wait(&pready[w], (turns >> w) & 1, 5) && wait(&vfull[s], ph, 6);
          if (!ok) break;
          ptx::tc_fence_after();
          if (ptx::elect_one()) {
            const uint64_t dv = dv0 + s * (F::kOperand >> 4), dp = dp0 + w * (F::kP >> 4);
            const uint32_t d = tmem + kPairs * NQ + w * F::kO, more = t >= kPairs;
#pragma unroll
            for (int k = 0; k < kStepsO; ++k) {
              const uint64_t da = dv + (k * kStepTokens * F::kRow >> 4), db = dp + (k * kStepTokens * 128 >> 4);
              if constexpr (!kCodes)
                ptx::tc_mma(d, da, db, idesc_o, k > 0 ? 1 : more);
              else if (k == 0)
                ptx::tc_mma_fp8_if(d, da, db, idesc_o, more);
              else
                ptx::tc_mma_fp8<1>(d, da, db, idesc_o);
            }
            if constexpr (F::kPRest > 0) {
              const uint64_t dr = dr0 + w * (F::kP >> 4);
#pragma unroll
              for (int k = 0; k < kStepsO; ++k)
                ptx::tc_mma_fp8_if(d + F::kPWide, dv + (k * kStepTokens * F::kRow >> 4), dr + (k * kStepTokens * 64 >> 4),
                                   ptx::idesc_e4m3_e5m2_mn_f32(128, F::kPRest), k > 0 ? 1 : more);
            }
            ptx::tc_commit(&vempty[s]);
            ptx::tc_commit(&pdone[w]);
          }
        }
        __syncwarp();
        turns ^= 1u << w;
        if (++s == stages) s = 0, ph ^= 1;
      }
    }
    __syncwarp();
  } else {
    // ---- the parts, ahead of the softmax ----
    const auto owner = [&](int64_t unit) {  // the CTA that has it
      const int64_t wide = (each + 1) * rest;
      return (int)(unit < wide ? quotient(unit, each + 1) : rest + quotient(unit - wide, each));
    };
    for (uint32_t part = 0;; ++part) {
      const int b = part % kPlans;
      const bool more = walk.next(a, abort_flag);
      if (!__all_sync(0xffffffffu, ptx::mbar_wait_paced(&ended[b], ~(part / kPlans) & 1, abort_flag))) {
        if (lane == 0) fail(7);
        break;
      }
      if (more) {
        // bits of the chunk's columns, row after row: those of row j begin at j group - col0
        const int col0 = walk.chunk * NQ;
        const int j0 = (int)((uint32_t)col0 * a.group_inv >> 32);
        const int j1 = min(walk.q.rows, (int)((uint32_t)(col0 + NQ - 1) * a.group_inv >> 32) + 1);
        uint64_t see0 = 0, see1 = 0;    // of nodes `lane` and lane + 32
        uint64_t mine0 = 0, mine1 = 0;  // the words of rows `lane` and lane + 32
        if (a.tree) {
          if (lane < walk.q.rows) mine0 = a.tree[walk.q.lo + lane];
          if (lane + 32 < walk.q.rows) mine1 = a.tree[walk.q.lo + lane + 32];
        } else {
          mine0 = ~0ull >> (63 - lane);
          mine1 = ~0ull >> (31 - lane);
        }
#pragma unroll 1
        for (int j = j0; j < j1; ++j) {
          const uint64_t word = __shfl_sync(0xffffffffu, j < 32 ? mine0 : mine1, j & 31);
          const int first = max(0, j * a.group - col0), last = min(NQ, (j + 1) * a.group - col0);
          const uint64_t bits = (~0ull >> (64 - (last - first))) << first;
          if ((word >> lane) & 1) see0 |= bits;
          if ((word >> (lane + 32)) & 1) see1 |= bits;
        }
        seers[b][lane] = see0;
        seers[b][lane + 32] = see1;
      }
      if (lane == 0) {
        Part p;
        p.tiles = 0;
        if (more) {
          p.r = walk.r, p.lo = walk.q.lo, p.base = walk.q.base, p.rows = walk.q.rows, p.head = walk.head;
          p.tile = walk.tile, p.tiles = walk.tiles, p.col0 = walk.chunk * NQ;
          p.columns = min(NQ, walk.q.rows * a.group - p.col0);
          p.slot = walk.begins && walk.ends ? -1 : 2 * cta + walk.begins;
          if (walk.begins && !walk.ends) {  // so it is the last part here; which CTA has the item's last unit:
            Shared* m = &a.meta[cta];
            m->lo = p.lo, m->head = p.head, m->col0 = p.col0, m->columns = p.columns;
            m->parts = owner(u1 + walk.q.tiles - walk.tiles - 1) - cta + 1;
          }
        }
        parts[b] = p;
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&planned[b]);
      if (!more) break;
    }
    // the first part's item began elsewhere (said last: nobody here waits for it)
    if (lane == 0 && u1 > u0 && start.x > F::kItemCost) a.meta[cta].first = owner(u0 - start.x + F::kItemCost);
    __syncwarp();
  }
  } else {
    ptx::reg_inc<F::kRegsHigh>();
    // ---- softmax: tiles w, w + 2, .. of a part and half of the columns a warpgroup ----
    constexpr int HQ = NQ / 2, kAll = 5;
    const int wg = warp >> 2, w = wg >> 1, h = wg & 1, quarter = warp & 3, token = quarter * 32 + lane;
    const int own = 1 + wg;  // its barrier
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16), tS = lanes + w * NQ + h * HQ, tO = lanes + kPairs * NQ;
    const int box_shift = min(a.pool.shift, 7);
    const uint32_t all_ok = (1u << (kTile >> box_shift)) - 1;
    uint32_t n0 = opaque(0), turn = opaque(0);  // the CTA's tiles before this part, this warpgroup's so far
    auto wait = [&](uint64_t* bar, uint32_t parity, int what) {
      if (!ptx::mbar_wait_paced(bar, parity, abort_flag)) fail(what);  // the loops run on: every later wait ends at once
    };
    // q of part `part`: four columns a warp, loaded before it is needed
    QColumn<D> q;
    const int qc = warp * 4 + (lane >> 3);
    static_assert(NQ <= 4 * kSoftWarps, "four columns a warp");
    const auto same = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };  // of a value that the warp shares
    const auto load_q = [&](int part) {
      const bool got = __all_sync(0xffffffffu, ptx::mbar_wait_paced(&planned[part % kPlans], (part / kPlans) & 1, abort_flag));
      if (!got) fail(8);
      if (got && same(parts[part % kPlans].tiles) > 0 && warp * 4 < NQ) q.load(a, parts[part % kPlans], qc);
    };
    const auto store_q = [&](int part) {
      if (same(*abort_flag) == 0 && same(parts[part % kPlans].tiles) > 0 && warp * 4 < NQ) {
        q.template store<kCodes, NQ>(a, parts[part % kPlans], qc, sQ + (part & 1) * F::kQ, qs[part & 1], out_at[part & 1]);
        ptx::fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&qfull[part & 1]);
    };
    int stored = opaque(0), last = opaque(0), loaded = opaque(0);  // parts whose q is in place, ..
    for (int part = opaque(0);; ++part) {
      const int b = part & 1;
      const Part& now = parts[part % kPlans];
      // q of this part and the next (this part's is there already but for the first)
#pragma unroll 1
      while (stored < part + 2 && !last) {
        if (!loaded) load_q(stored);
        loaded = 0;
        store_q(stored);
        last = same(parts[stored % kPlans].tiles) <= 0;
        ++stored;
      }
      // this warpgroup's references and their like
      float* my_nref = &nref[w][h * HQ];
      float* my_delta = &delta[w][h * HQ];
      float* my_factor = &factor[w][h * HQ];
      float* my_sum_at = &sum_at[w][h * HQ];
      if (token < HQ) my_nref[token] = my_sum_at[token] = 0.f, set[w][h * HQ + token] = sum_set[w][h * HQ + token] = false;
      if (token == 0) odd_scale[w][h] = false;
      const bool got = ptx::mbar_wait_paced(&qfull[b], (part >> 1) & 1, abort_flag);
      if (!got) fail(10);
      // after a fault all leave together (q is counted as ready, and the plans are no more than they were)
      if (same(ptx::named_any(kAll, kSoft, !got || *abort_flag != 0))) break;
      const int tiles = same(now.tiles), tile0 = same(now.tile);
      if (tiles == 0) break;
      const int base = same(now.base), len = base + same(now.rows);

      uint64_t l2[HQ / 2];
#pragma unroll
      for (int i = 0; i < HQ / 2; ++i) l2[i] = 0;
      int mode = opaque(1);  // 1: a column has no reference yet, 2: the sums have their own
#pragma unroll 1
      for (int t = opaque(w); t < tiles; t += kPairs) {
        const uint32_t n = n0 + t, note = n % F::kNotes;
        wait(&noted[note], (n / F::kNotes) & 1, 11);  // (not k itself: S may have let it go)
        const int pos0 = (tile0 + t) * kTile, pos = pos0 + token;
        const uint32_t have = okmask[note];
        const bool masked = pos0 + kTile > base || have != all_ok;
        const bool held = pos < len && ((have >> (token >> box_shift)) & 1);  // looked at where masked
        float k_scale = 1.f, v_scale = 1.f;
        if (kCodes) {
          k_scale = sScale[note * 2 * kTile + token];
          v_scale = sScale[note * 2 * kTile + kTile + token];
        }
        if (masked) {
          // what no row or only some see must not reach the others through 0 * NaN
          // (the tile before is in O first: until v of tile n - kStagesV has arrived, vfull's phase is one of
          // the same parity two back)
          if (turn > 0) wait(&pdone[w], (turn + 1) & 1, 12);
          wait(&vfull[n % F::kStagesV], (n / F::kStagesV) & 1, 12);
          uint8_t* row = sV + n % F::kStagesV * F::kOperand + token * F::kRow;
          if (!held || pos >= base) {
            uint32_t any = 0;
            // half of the row a warpgroup, neighbouring tokens' 16-byte units in different banks
            constexpr int kUnits = F::kParts * F::kRow / 16, kRowUnits = F::kRow / 16;
            const int turned = (kRowUnits == 8 ? token : token >> 1) & (kRowUnits - 1);
#pragma unroll 1
            for (int u = h * (kUnits / 2); u < (h + 1) * (kUnits / 2); ++u) {
              const int i = u ^ (turned & (kUnits / 2 - 1));
              uint4* at = reinterpret_cast<uint4*>(row + i * 16 / F::kRow * F::kPart + i * 16 % F::kRow);
              if (held) {
                const uint4 x = *at;
                const uint4 m = make_uint4(non_finite<kCodes>(x.x), non_finite<kCodes>(x.y), non_finite<kCodes>(x.z),
                                           non_finite<kCodes>(x.w));
                if (m.x | m.y | m.z | m.w) {
                  *at = make_uint4(x.x & ~m.x, x.y & ~m.y, x.z & ~m.z, x.w & ~m.w);
                  any = 1;
                }
              } else {
                *at = make_uint4(0, 0, 0, 0);
              }
            }
            if (any) atomicOr(&hidden[b], 1ull << (pos - base));
          }
        }
        wait(&sfull[w], turn & 1, 13);
        ++turn;
        ptx::tc_fence_after();
        // y, less the reference so far: S (qs ks) + (log2 vs - ref); both factors are formed while S arrives
        uint64_t x2[HQ / 2];
        constexpr int L = HQ < 16 ? HQ : 16;  // columns at a time
        float v[HQ / L][L], v_inv = 1.f;
        load_columns<L>(tS, v[0]);
        uint64_t ks2 = 0, vl2 = 0;
        if (kCodes) {
          if (masked && !held) v_scale = 1.f;  // what is no token's scale
          const float least = v_scale < kLeastNormal ? kLeastNormal : v_scale;  // 0 of a cache that was cleared
          const float v_log = __log2f(least);
          // a scale far from 1 (0 and NaN too) stands in the place of its inverse, negated
          v_inv = __float_as_uint(v_scale) - kLeastScale > kMostScale - kLeastScale ? -v_scale : ptx::rcp(least);
          ks2 = ptx::pack2(k_scale, k_scale);
          vl2 = ptx::pack2(v_log, v_log);
        }
#pragma unroll
        for (int c = 0; c < HQ; c += L) {
          uint64_t f[L / 2], g[L / 2];
#pragma unroll
          for (int i = 0; i < L / 2; i += 2) {
            const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&qs[b][h * HQ + c + 2 * i]);
            const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(&my_nref[c + 2 * i]);  // 0 before they are set
            f[i] = kCodes ? ptx::mul2(u.x, ks2) : u.x, f[i + 1] = kCodes ? ptx::mul2(u.y, ks2) : u.y;
            g[i] = kCodes ? ptx::add2(r.x, vl2) : r.x, g[i + 1] = kCodes ? ptx::add2(r.y, vl2) : r.y;
          }
          ptx::tmem_ld_wait<L>(v[c / L]);
          if (c + L < HQ) load_columns<L>(tS + c + L, v[c / L + (c + L < HQ)]);
          if (c + L == HQ) {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&sfree[w]);
          }
#pragma unroll
          for (int i = 0; i < L / 2; ++i) x2[c / 2 + i] = ptx::fma2(ptx::pack2(v[c / L][2 * i], v[c / L][2 * i + 1]), f[i], g[i]);
        }
        if (masked) {
          const uint32_t see = !held ? 0u : pos < base ? ~0u : (uint32_t)(seers[part % kPlans][pos - base] >> (h * HQ));
#pragma unroll
          for (int i = 0; i < HQ / 2; ++i) {
            const float2 x = ptx::unpack2(x2[i]);
            x2[i] = ptx::pack2((see >> (2 * i)) & 1 ? x.x : -INFINITY, (see >> (2 * i + 1)) & 1 ? x.y : -INFINITY);
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < HQ / 2; ++i) {
          const float2 x = ptx::unpack2(x2[i]);
          top = fmaxf(top, fmaxf(x.x, x.y));
        }
        const bool raise = ptx::named_any(own, 128, top > kRaise<kCodes> || !(v_inv > 0.f)) || mode;
        if (turn > 1) {  // the tile before is in O, and its weights have been read
          wait(&pdone[w], turn & 1, 14);
          ptx::tc_fence_after();
        }
        bool full = raise;
        if (F::kApartInline && mode == 2) {  // most often no reference is to be raised
          full = ptx::named_any(own, 128, top > kRaise<kCodes> || highest_apart<HQ>(x2, v_inv, my_sum_at) > kRaiseSum);
          if (!full) {
            add_apart<HQ>(x2, l2, v_inv, my_sum_at);
            v_inv = 0.f;
          }
        }
        if (full) {
          // the columns' largest, new references, what was summed so far brought to them
#pragma unroll 1
          for (bool sums = kCodes;; sums = false) {
            float m = -INFINITY;  // of column `lane`
#pragma unroll
            for (int i = 0; i < HQ / 2; ++i) {
              const float2 x = ptx::unpack2(x2[i]);
              const float m0 = ptx::warp_max_redux(x.x), m1 = ptx::warp_max_redux(x.y);
              m = lane == 2 * i ? m0 : lane == 2 * i + 1 ? m1 : m;
            }
            if (lane < HQ) warp_top[warp][lane] = m;
            if (!(v_inv > 0.f)) odd_scale[w][h] = true;
            ptx::named_sync(own, 128);
            if (!sums || !odd_scale[w][h]) break;
            // this tile's sums first, which changes x2
            if constexpr (F::kApartInline) {
              raise_apart<HQ>(x2, l2, v_inv, my_sum_at, my_factor, &sum_set[w][h * HQ], &warp_top[wg * 4], own);
            } else {
              uint64_t x[HQ / 2], l[HQ / 2];
#pragma unroll
              for (int i = 0; i < HQ / 2; ++i) x[i] = x2[i], l[i] = l2[i];
              raise_apart_out_of_line<HQ>(x, l, v_inv, my_sum_at, my_factor, &sum_set[w][h * HQ], &warp_top[wg * 4], own);
#pragma unroll
              for (int i = 0; i < HQ / 2; ++i) x2[i] = x[i], l2[i] = l[i];
            }
            v_inv = 0.f;
          }
          const bool apart = kCodes && odd_scale[w][h];  // the sums have references of their own
          bool none = false;
          if (token < HQ) {
            const float m = fmaxf(fmaxf(warp_top[wg * 4][token], warp_top[wg * 4 + 1][token]),
                                  fmaxf(warp_top[wg * 4 + 2][token], warp_top[wg * 4 + 3][token]));
            float d = 0.f;
            const bool was = set[w][h * HQ + token];
            if (was)
              d = fmaxf(0.f, m - kHead<kCodes>);
            else if (m > -INFINITY)
              d = m - kHead<kCodes>, set[w][h * HQ + token] = true, sum_set[w][h * HQ + token] |= !apart;
            else
              none = true;
            my_delta[token] = -d;
            my_factor[token] = was ? ptx::ex2(-d) : 1.f;  // (nothing was summed before the first reference, however low that is)
            my_nref[token] -= d;
            if (apart) my_sum_at[token] += d;
          }
          mode = (ptx::named_any(own, 128, none) ? 1 : 0) | (apart ? 2 : 0);
#pragma unroll
          for (int i = 0; i < HQ / 2; ++i) {
            x2[i] = ptx::add2(x2[i], *reinterpret_cast<const uint64_t*>(&my_delta[2 * i]));
            if (t >= kPairs && !apart) l2[i] = ptx::mul2(l2[i], *reinterpret_cast<const uint64_t*>(&my_factor[2 * i]));
          }
          if (t >= kPairs) {
#pragma unroll 1
            for (int p = 0; p < F::kPPieces; ++p)
#pragma unroll 1
              for (int c = 0; c < HQ; c += 8) {
                const uint32_t at = tO + w * F::kO + p * NQ + h * HQ + c;
                float v[8];
                ptx::tmem_ld8(at, v);
                ptx::tmem_ld_wait<8>(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= my_factor[c + i];
                ptx::tmem_st8(at, v);
              }
            ptx::tmem_st_wait();
          }
        }
        // weights, their sums and their pieces
        uint8_t* prow = sP + w * F::kP + token * 128;
        const uint64_t vi2 = ptx::pack2(v_inv, v_inv);
        constexpr int G = HQ < 16 ? HQ : 16;  // columns at a time
#pragma unroll
        for (int c = 0; c < HQ; c += G) {
          uint32_t hh[G / 2], r1[G / 2], c3[G / 2];
#pragma unroll
          for (int i = 0; i < G / 2; ++i) {
            const float2 x = ptx::unpack2(x2[c / 2 + i]);
            const float p0 = ptx::ex2(x.x), p1 = ptx::ex2(x.y);
            const uint64_t p2 = ptx::pack2(p0, p1);
            uint64_t& l = l2[c / 2 + i];
            l = kCodes ? ptx::fma2(p2, vi2, l) : ptx::add2(l, p2);
            if constexpr (kCodes) {
              hh[i] = half2_bits(__floats2half2_rn(p0, p1));
              r1[i] = left_of(hh[i]);
              c3[i] = e5m2x2(left_of(r1[i]));
            } else {
              const __nv_bfloat162 o = __floats2bfloat162_rn(p0, p1);
              hh[i] = *reinterpret_cast<const uint32_t*>(&o);
            }
          }
          // (16-byte unit u of row r lies at u ^ (r % 8))
          auto place = [&](uint32_t byte) { return prow + (((byte >> 4) ^ (token & 7)) << 4) + (byte & 15); };
          if constexpr (kCodes) {
            const uint32_t byte = h * HQ + c;
            uint32_t b1[G / 4], b2[G / 4], b3[G / 4];
#pragma unroll
            for (int i = 0; i < G / 4; ++i) {
              b1[i] = __byte_perm(hh[2 * i], hh[2 * i + 1], 0x7531);
              b2[i] = __byte_perm(r1[2 * i], r1[2 * i + 1], 0x7531);
              b3[i] = __byte_perm(c3[2 * i], c3[2 * i + 1], 0x5410);
            }
            uint8_t* third = place(2 * NQ + byte);
            if constexpr (F::kPRest > 0) third = sP + w * F::kP + F::kPCol + swizzled<64>(token * 64 + byte);
            if constexpr (G == 16) {
              *reinterpret_cast<uint4*>(place(byte)) = make_uint4(b1[0], b1[1], b1[2], b1[3]);
              *reinterpret_cast<uint4*>(place(NQ + byte)) = make_uint4(b2[0], b2[1], b2[2], b2[3]);
              *reinterpret_cast<uint4*>(third) = make_uint4(b3[0], b3[1], b3[2], b3[3]);
            } else {
              *reinterpret_cast<uint2*>(place(byte)) = make_uint2(b1[0], b1[1]);
              *reinterpret_cast<uint2*>(place(NQ + byte)) = make_uint2(b2[0], b2[1]);
              *reinterpret_cast<uint2*>(third) = make_uint2(b3[0], b3[1]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < G / 8; ++i)
              *reinterpret_cast<uint4*>(place((h * HQ + c + 8 * i) * 2)) = make_uint4(hh[4 * i], hh[4 * i + 1], hh[4 * i + 2], hh[4 * i + 3]);
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&pready[w]);
      }

      // ---- the part's end: sums of both tile sequences, O joined and written ----
      n0 += tiles;
      if (!last) {
        load_q(stored);
        loaded = 1;
      }
      const bool two = kPairs > 1 && tiles > 1;  // both pairs have a tile
      if (w == 0 || two) wait(&pdone[w], (turn - 1) & 1, 15);
      {
        float v[HQ];
#pragma unroll
        for (int i = 0; i < HQ / 2; ++i) {
          const float2 x = ptx::unpack2(l2[i]);
          v[2 * i] = x.x;
          v[2 * i + 1] = x.y;
        }
        const float sum = over_lanes<HQ>(v, [](float x, float y) { return x + y; });
        if (lane < HQ) warp_top[warp][lane] = sum;
      }
      ptx::named_sync(kAll, kSoft);
      ptx::tc_fence_after();
      const unsigned long long bad_rows = hidden[b];
      if (threadIdx.x == 0) hidden[b ^ 1] = 0;
      const int slot = same(now.slot), columns = same(now.columns);
      const bool whole = slot < 0;
      if (threadIdx.x < NQ) {
        const int c = threadIdx.x, half = c / HQ, i = c % HQ;
        float ref[kPairs], sum_ref[kPairs], l[kPairs];
#pragma unroll
        for (int g = 0; g < kPairs; ++g) {
          const int first = (g * 2 + half) * 4;
          ref[g] = set[g][c] ? -nref[g][c] : -INFINITY;
          sum_ref[g] = sum_set[g][c] ? -(nref[g][c] + sum_at[g][c]) : -INFINITY;
          l[g] = (warp_top[first][i] + warp_top[first + 1][i]) + (warp_top[first + 2][i] + warp_top[first + 3][i]);
        }
        float m = ref[0], sum_m = sum_ref[0], sum = l[0], f[kPairs] = {1.f};
        if constexpr (kPairs > 1) {
          f[1] = 0.f;
          if (two) {
            m = fmaxf(ref[0], ref[1]);
            sum_m = fmaxf(sum_ref[0], sum_ref[1]);
            sum = 0.f;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              f[g] = ref[g] == m ? 1.f : ptx::ex2(ref[g] - m);
              sum += (sum_ref[g] == sum_m ? 1.f : ptx::ex2(sum_ref[g] - sum_m)) * l[g];
            }
          }
        }
        const float2 inv = whole ? inverse(sum, m - sum_m) : make_float2(1.f, 1.f);
#pragma unroll
        for (int g = 0; g < kPairs; ++g) coef[g][c] = f[g] * inv.x;
        unit[c] = inv.y;
        if (!whole) a.stat[(int64_t)slot * NQ + c] = make_float4(m, sum, sum_m, 0.f);
      }
      ptx::named_sync(kAll, kSoft);
      // its share of the columns a warpgroup, eight at a time (a loop: straight-line code this rarely
      // run waits for its instructions, 8700 cycles for 16 columns)
      constexpr int W = NQ / (2 * kPairs) >= 8 ? NQ / (2 * kPairs) : 8;
      const int d = quarter * 32 + lane;
      if (quarter * 32 < D) {
#pragma unroll 1
        for (int c0 = wg * W; c0 < min(columns, (wg + 1) * W); c0 += 8) {
          float v[8], u[8];
          load_sum<F::kPPieces>(tO + c0, NQ, v);
          if (two) load_sum<F::kPPieces>(tO + (kPairs - 1) * F::kO + c0, NQ, u);
          const int n = min(8, columns - c0);
          const float* f0 = &coef[0][c0];
          const float* f1 = &coef[kPairs - 1][c0];
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = (two ? fmaf(f1[i], u[i], f0[i] * v[i]) : f0[i] * v[i]) * unit[c0 + i];
          if (whole) {
            // two elements a store: even lanes take columns 0-3 of two lanes, odd ones 4-7
            const bool odd = lane & 1;
            const int64_t* at = &out_at[b][c0 + 4 * odd];
            __nv_bfloat16* dst = a.out + (d & ~1);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float mine = odd ? v[i + 4] : v[i], other = __shfl_xor_sync(0xffffffffu, odd ? v[i] : v[i + 4], 1);
              const __nv_bfloat162 x = __floats2bfloat162_rn(odd ? other : mine, odd ? mine : other);
              if (i + 4 * odd < n) *reinterpret_cast<__nv_bfloat162*>(dst + at[i]) = x;
            }
          } else {
            float* at = a.part + ((int64_t)slot * NQ + c0) * D + d;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (i < n) at[i * D] = v[i];
          }
        }
        __syncwarp();  // (an element may have been written by the lane beside)
        if (bad_rows && d < D)
          add_non_finite<kCodes, D, NQ>(a, now, seers[part % kPlans], out_at[b], bad_rows, wg * W, min(columns, (wg + 1) * W), d);
      }
      ptx::tc_fence_before();
      ptx::named_sync(kAll, kSoft);  // O may be written again
      if (lane == 0) ptx::mbar_arrive(&ended[part % kPlans]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && abort_s[0] && a.hdr) report_error(a.hdr, DSPARK_TIMEOUT, abort_s[0]);
  if (warp == kSoftWarps + 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, F::kTmemCols);
  }
}

// The items that several CTAs share: part 0 is the second slot of the CTA they begin in,
// the others the first slots of those behind it.  The blocks of CTA blockIdx.x / (NQ / 8) take eight
// columns each of the item that begins in it and goes on, a warp a column, D / 32 elements a lane; of
// more than eight parts one column each, a warp every eighth part, and the blocks of the seven CTAs
// behind it the other columns.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
template <int D, int NQ>
__global__ void __launch_bounds__(kJoinThreads) k_tree_join(const TreeArgs a) {
  static_assert(kJoinWarps == 8, "columns of a block");
  constexpr int E = D / 32;
  __shared__ float sums[8], os[8][D];
  ptx::launch_dependents();
  ptx::grid_wait();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int cta = blockIdx.x / (NQ / 8), c = blockIdx.x % (NQ / 8) * 8;
  Shared m = a.meta[cta];
  if (m.parts <= 1) {
    const int behind = cta - m.first;
    if (m.first < 0 || behind > 7) return;
    cta = m.first, c += behind;
    m = a.meta[cta];
    if (m.parts <= 8) return;
  }
  const bool team = m.parts > 8;
  if (!team) c += warp;
  if (c >= m.columns) return;
  const auto slot = [&](int p) { return (int64_t)(p ? 2 * (cta + p) : 2 * cta + 1) * NQ + c; };
  float ref = -INFINITY, sum_ref = -INFINITY;
  for (int p = lane; p < m.parts; p += 32) {
    const float4 s = a.stat[slot(p)];
    ref = fmaxf(ref, s.x), sum_ref = fmaxf(sum_ref, s.z);
  }
  ref = warp_max(ref);
  sum_ref = warp_max(sum_ref);
  float sum = 0.f, o[E] = {};
  const auto add = [&](float g, int p) {
    const float* src = a.part + slot(p) * D + lane * E;
    if constexpr (E == 4) {
      const float4 x = *reinterpret_cast<const float4*>(src);
      o[0] = fmaf(g, x.x, o[0]), o[1] = fmaf(g, x.y, o[1]), o[2] = fmaf(g, x.z, o[2]), o[3] = fmaf(g, x.w, o[3]);
    } else {
      const float2 x = *reinterpret_cast<const float2*>(src);
      o[0] = fmaf(g, x.x, o[0]), o[1] = fmaf(g, x.y, o[1]);
    }
  };
  const auto factor = [&](int p) {  // of part p, whose sum is added
    if (p >= m.parts) return 0.f;
    const float4 s = a.stat[slot(p)];
    sum += (s.z == sum_ref ? 1.f : exp2f(s.z - sum_ref)) * s.y;
    return s.x == ref ? 1.f : exp2f(s.x - ref);
  };
  if (!team) {
    const float f = factor(lane);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float g = __shfl_sync(0xffffffffu, f, p);
      if (p < m.parts) add(g, p);
    }
    sum = warp_sum(sum);
  } else {
    for (int p0 = warp; p0 < m.parts; p0 += 32 * 8) {  // this warp's parts p0, p0 + 8, ..
      const float f = factor(p0 + lane * 8);
      const int count = min(32, (m.parts - p0 + 7) / 8);
#pragma unroll 4
      for (int i = 0; i < count; ++i) add(__shfl_sync(0xffffffffu, f, i), p0 + i * 8);
    }
    sum = warp_sum(sum);
    if (lane == 0) sums[warp] = sum;
#pragma unroll
    for (int e = 0; e < E; ++e) os[warp][lane * E + e] = o[e];
    __syncthreads();
    if (warp > 0) return;
    sum = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int w = 0; w < 8; ++w) {
      sum += sums[w];
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += os[w][lane * E + e];
    }
  }
  const float2 inv = inverse(sum, ref - sum_ref);
  uint32_t out[E / 2];
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const __nv_bfloat162 x = __floats2bfloat162_rn(o[e] * inv.x * inv.y, o[e + 1] * inv.x * inv.y);
    out[e / 2] = *reinterpret_cast<const uint32_t*>(&x);
  }
  const int col = m.col0 + c, row = (int)((uint32_t)col * a.group_inv >> 32);
  __nv_bfloat16* dst = a.out + (int64_t)(m.lo + row) * a.ldo + (m.head * a.group + col - row * a.group) * D + lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else
    *reinterpret_cast<uint32_t*>(dst) = out[0];
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
struct Layout {
  size_t meta, stat, part, total;
};
int columns_of(int max_tree, int group) {
  const int n = max_tree * group;
  return n <= 16 ? 16 : n <= 32 ? 32 : 64;
}
Layout layout(int max_tree, int group, int head_dim) {
  const size_t nq = columns_of(max_tree, group);
  Layout l;
  l.meta = align_up(sizeof(WsHeader), 256);
  l.stat = align_up(l.meta + kMaxCtas * sizeof(Shared), 256);
  l.part = align_up(l.stat + 2 * kMaxCtas * nq * sizeof(float4), 256);
  l.total = l.part + 2 * kMaxCtas * nq * head_dim * sizeof(float);
  return l;
}

struct Dev {
  int sms = 0;
  bool sm103 = false;
};
// The kernel's warps trade registers among themselves: what the softmax's warps ask for
// has to be there, or they would wait for ever.
template <typename F>
cudaError_t check_registers(const void* f) {
  cudaFuncAttributes at;
  if (const cudaError_t e = cudaFuncGetAttributes(&at, f); e != cudaSuccess) return e;
  return at.numRegs * F::kThreads < F::kSoft * F::kRegsHigh + 128 * F::kRegsLow ? cudaErrorNotSupported : cudaSuccess;
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
    cache[dev] = d;
    have[dev] = true;
  }
  *out = cache[dev];
  return cudaSuccess;
}

template <bool kCodes, int D, int NQ>
cudaError_t run(const dspark_kv_cache& c, const TreeArgs& t, const Dev& dev, cudaStream_t s) {
  using F = Form<kCodes, D, NQ>;
  CUtensorMap tmK, tmV;
  const int64_t rows = (int64_t)c.n_pages * c.n_kv_heads * c.page_size;
  const CUtensorMapDataType dt = kCodes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int box = std::min(c.page_size, kTile);
  if (!tensor_map_2d(&tmK, dt, c.k, D, rows, D * F::kElem, F::kRow / F::kElem, box, F::kElem) ||
      !tensor_map_2d(&tmV, dt, c.v, D, rows, D * F::kElem, F::kRow / F::kElem, box, F::kElem))
    return cudaErrorInvalidValue;
  const auto f = k_tree_attention<kCodes, D, NQ>;
  static const cudaError_t registers = check_registers<F>((const void*)f);
  if (registers != cudaSuccess) return registers;
  if (const cudaError_t e = ensure_smem_limit((const void*)f, (int)F::kSmem); e != cudaSuccess) return e;
  const unsigned grid = (unsigned)std::min(dev.sms * F::kCtas, kMaxCtas);
  if (const cudaError_t e = launch_overlapped(f, grid, F::kThreads, F::kSmem, 1, s, tmK, tmV, t); e != cudaSuccess) return e;
  count_launches(1);
  const cudaError_t e = launch_overlapped(k_tree_join<D, NQ>, grid * (NQ / 8), kJoinThreads, 0, 1, s, t);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

template <bool kCodes, int D>
cudaError_t run_columns(const dspark_kv_cache& c, const TreeArgs& t, const Dev& dev, cudaStream_t s) {
  switch (columns_of(t.max_tree, t.group)) {
    case 16: return run<kCodes, D, 16>(c, t, dev, s);
    case 32: return run<kCodes, D, 32>(c, t, dev, s);
    default: return run<kCodes, D, 64>(c, t, dev, s);
  }
}

}  // namespace

size_t tree_attention_ws(int max_tree, int n_q_heads, int n_kv_heads, int head_dim) {
  return layout(max_tree, n_q_heads / n_kv_heads, head_dim).total;
}

cudaError_t launch_tree_attention(const dspark_tree_attention_args& a, uint8_t* ws, cudaStream_t s) {
  Dev dev;
  if (const cudaError_t e = device(&dev); e != cudaSuccess) return e;
  if (!dev.sm103) return cudaErrorNotSupported;
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
  t.group = a.n_q_heads / a.cache.n_kv_heads;
  t.group_inv = ((1ull << 32) + t.group - 1) / t.group;
  t.max_tree = a.max_tree;
  t.scale = a.scale;
  t.hdr = reinterpret_cast<WsHeader*>(ws);
  const Layout l = layout(a.max_tree, t.group, a.cache.head_dim);
  t.meta = reinterpret_cast<Shared*>(ws + l.meta);
  t.stat = reinterpret_cast<float4*>(ws + l.stat);
  t.part = reinterpret_cast<float*>(ws + l.part);
  const bool small = a.cache.head_dim == 64;
  if (a.cache.dtype == DSPARK_E4M3)
    return small ? run_columns<true, 64>(a.cache, t, dev, s) : run_columns<true, 128>(a.cache, t, dev, s);
  return small ? run_columns<false, 64>(a.cache, t, dev, s) : run_columns<false, 128>(a.cache, t, dev, s);
}

}  // namespace dspark

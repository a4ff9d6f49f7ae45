// Attention of groups of queries over a shared prefix on the tcgen05 tensor
// cores (bf16 cache at head dim 64 or 128, E4M3 cache at 128).
//
// With n requests behind one prefix the n G rows (query, head of the kv head's G)
// are the M dimension of ordinary matrix products over the prefix, so each key and value
// is read once for a block of 256 rows.  A worker (one CTA an SM) takes the
// plan's items one after another, each a range of key tiles of one block:
//   warps 0-15  softmax: warp w takes rows [32 (w % 4), +32) of chain t = (w / 4) % 2
//               and, with h = w / 8, one half of its score columns and of O's dims
//   warp 16     TMA producer: K_j and V_j [128 keys x D] into a ring of slots,
//               V_(j-1) and K_j as one unit under one barrier
//   warp 17     MMA issuer (one elected lane) and TMEM owner
//   warp 18     relay: clears the rows of V behind a shard's last key and adds one
//               arrival on each chain's P barrier once the step's unit has landed,
//               so that the issuer's wait for P covers the unit
// Two chains keep the tensor cores and the exponentials busy in turn.  A block
// of more than 128 rows: chain t is M tile t, both share the step's K and V.  A
// block of up to 128 rows (WIDE = false): chain t takes keys [64 t, 64 t + 64) of every
// tile, and the two results combine in shared memory at the end: a single chain
// would wait for its own exponentials in every step.
// TMEM (512 columns): chain t holds S in columns [256 t, +128) (or 64) and O in
// [256 t + 128, +D).  Each half of a row writes its P (bf16 pairs) over the first
// half of its own S columns.  The running max moves only when a row's max grows by
// more than 2^8; any running max gives the exact result (O = sum e^(s-m) v / sum e^(s-m)).
// P is rounded to bf16 for its product, its sum is not.
// E4M3 (F8): S multiplies K's codes as they are stored, with the queries as two E4M3
// numbers each, hi + lo of the row times a power of two that brings its largest element
// to [128, 256): 4 + 4 significant bits hold bf16's 8 down to 2^-9 of the largest, and
// smaller elements are off by up to 2^-17 of it (E4M3's least step, 2^-9, halved); V's
// codes become bf16 (exact; a NaN code NaN), since P needs the range that bf16 has: warps 18-21 convert them
// and take the relay's part, but in blocks of up to 64 rows the softmax warps without rows
// convert.  A token's scale multiplies its column of S and, once P's sum is taken, of P.
// What bounds it: 64 requests x 32 heads behind 32,768 keys of 8 kv heads (134 MB) take
// 48-50 us with the merge, 0.4 of HBM: 14 tiles of 1.5 us, at HBM's rate, and some 20 us of
// plan and first loads, the last product, fp32 parts and merge.  300 x 64 heads behind
// 85,000 keys in five groups: 119 us.  131,072 E4M3 keys: 16 x 32 heads 95 us, a chain of
// 54 tiles of 1.4 us; 32 x 32 heads 136 us and 64 x 32 heads 182, bound by V's conversion (four warps).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstring>

#include "early_launch.cuh"
#include "internal.h"
#include "page_count.cuh"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {
using namespace tc;

constexpr int BM = 128;  // rows of an M tile
constexpr int BN = 128;  // keys of a K/V tile
constexpr int kSoftmaxWarps = 16;
constexpr int kWarpTma = kSoftmaxWarps, kWarpMma = kSoftmaxWarps + 1, kWarpRelay = kSoftmaxWarps + 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;
// E4M3: in a block of up to so many rows half of the softmax warps have none, and convert V
// instead of the relay's four (32 heads behind 131,072 tokens: one request 133 us without
// them and 92 with, 16 requests 135 and 95; behind 16,384 35 and 33).  Larger blocks leave a
// quarter without rows at most.
constexpr int kHelpRows = 64;

template <int D, bool F8>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kQBytes = BM * D * 2;    // (E4M3: hi, then lo)
  static constexpr int kSlotBytes = BN * D * 2;
  static constexpr int kSlots = F8 ? 2 : D == 128 ? 5 : 10;  // of the K/V ring (E4M3: of V as bf16)
  static constexpr int kRing = 2 * kQBytes;
  // E4M3: rings of code tiles behind it
  static constexpr int kKSlots = 3, kCodeTiles = kKSlots + 2, kCodeBytes = BN * D;
  static constexpr int kCodes = kRing + kSlots * kSlotBytes;
  static constexpr int kTiles = kCodes + (F8 ? kCodeTiles * kCodeBytes : 0);
  static constexpr int kThreads = 32 * (kSoftmaxWarps + (F8 ? 6 : 3));
  static constexpr int kRelays = F8 ? 4 : 1;  // arrivals of the relay's part
};

// K and V of up to MAXC shards; a pool has one map of each, with 64-row boxes.
template <int MAXC>
struct Maps {
  CUtensorMap k[MAXC], v[MAXC];
};

struct Params {
  PrefixArgs a;
  FastDiv by_g;  // rows of a block to query rows
  float scale_log2;
  unsigned* status;
  unsigned long long wait_ns;
  int stall_test;  // test hook: the MMA thread waits on a barrier nobody arrives at
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0, float c1) {
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d0), "=f"(d1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Four E4M3 codes as bf16, two words of two.  With the code's exponent and mantissa at
// bf16's place a code is 2^-120 of its value (subnormal codes are subnormal bf16),
// and the product with 2^120 is exact.
// top: the largest magnitude so far, of two columns of codes in the upper bytes of halves.
__device__ __forceinline__ void bf16_of_codes(uint32_t codes, uint32_t& lo, uint32_t& hi, uint32_t& top) {
  const uint32_t a = __byte_perm(codes, 0, 0x1404), b = __byte_perm(codes, 0, 0x3424);  // codes in the upper bytes of halves
  const uint32_t m = a & 0x7f007f00u, n = b & 0x7f007f00u;
  const uint32_t x = (a & 0x80008000u) | (m >> 4), y = (b & 0x80008000u) | (n >> 4);
  const uint32_t k = 0x7b807b80u;  // 2^120 twice
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(k));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(k));
  top = __vimax3_u16x2(top, m, n);
}
// Eight elements of a query row, whose 16 lanes stand side by side, as E4M3 hi and lo of
// the row times 2^(7 - e), its largest magnitude in [2^e, 2^(e+1)); *inv = 2^(e - 7).  lo at
// hi's own scale, so that both products add up in one accumulator.
__device__ __forceinline__ void put_codes(const uint4& x, uint8_t* row, int swizzle, int piece, float* inv) {
  const uint32_t k = 0x7fff7fffu;  // magnitudes are ordered like their bits, two bf16 at a time
  uint32_t m = __vmaxu2(__vmaxu2(x.x & k, x.y & k), __vmaxu2(x.z & k, x.w & k));
  m = max(m & 0xffff0000u, m << 16);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  const int e = max(-100, (int)(m >> 23) - 127);
  const float f = __uint_as_float((uint32_t)(7 - e + 127) << 23);
  // an infinite element would become 448: the row's scores are NaN instead
  if (piece == 0) *inv = __uint_as_float(e < 128 ? (uint32_t)(e - 7 + 127) << 23 : 0x7fffffffu);
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float v0 = __uint_as_float(in[i] << 16) * f, v1 = __uint_as_float(in[i] & 0xffff0000u) * f;
    uint16_t h, l;
    uint32_t b;
    float h0, h1;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(v1), "f"(v0));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(h));
    asm("{\n .reg .f16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}" : "=f"(h0), "=f"(h1) : "r"(b));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l) : "f"(v1 - h1), "f"(v0 - h0));
    hi[i >> 1] |= (uint32_t)h << (16 * (i & 1));
    lo[i >> 1] |= (uint32_t)l << (16 * (i & 1));
  }
  uint8_t* at = row + (((piece >> 1) ^ swizzle) << 4) + 8 * (piece & 1);
  *reinterpret_cast<uint2*>(at) = make_uint2(hi[0], hi[1]);
  *reinterpret_cast<uint2*>(at + BM * 128) = make_uint2(lo[0], lo[1]);
}
// Chunks [c0, c0 + N) of 16 codes of a V tile's row as bf16, both 128-byte-swizzled; `to`
// is the row in the first of the bf16 tile's two 64-dim chunks of BN rows.  A NaN code
// (0x7F, 0xFF) becomes +-480 here; true if there is one (nan_codes puts it right).
template <int N>
__device__ __forceinline__ bool convert_row(const uint8_t* from, uint8_t* to, int row, int c0) {
  const uint4* src = reinterpret_cast<const uint4*>(from);
  uint32_t top = 0;
#pragma unroll 4
  for (int c = c0; c < c0 + N; ++c) {
    const uint4 x = src[c ^ (row & 7)];
    uint32_t o[8];
    bf16_of_codes(x.x, o[0], o[1], top);
    bf16_of_codes(x.y, o[2], o[3], top);
    bf16_of_codes(x.z, o[4], o[5], top);
    bf16_of_codes(x.w, o[6], o[7], top);
    uint8_t* chunk = to + (c >> 2) * (BN * 128);
    const int unit = 2 * (c & 3);
    *reinterpret_cast<uint4*>(chunk + ((unit ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4*>(chunk + (((unit + 1) ^ (row & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
  return (top & 0xffffu) == 0x7f00u || top >> 16 == 0x7f00u;
}
// The NaN codes of those chunks as bf16 NaN: hardly ever called.
__device__ __noinline__ void nan_codes(const uint8_t* from, uint8_t* to, int row, int c0, int n) {
#pragma unroll 1
  for (int d = 16 * c0; d < 16 * (c0 + n); ++d) {
    if ((from[((d >> 4 ^ (row & 7)) << 4) + (d & 15)] & 0x7f) != 0x7f) continue;
    const int at = (((d >> 3 & 7) ^ (row & 7)) << 4) + 2 * (d & 7);
    *reinterpret_cast<uint16_t*>(to + (d >> 6) * (BN * 128) + at) = 0x7fff;
  }
}
__device__ __forceinline__ void mbar_inval(uint32_t bar) { asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory"); }

__device__ void report_timeout(unsigned* status, unsigned site, volatile int* abort) {
  *abort = 1;
  if (atomicCAS(status, 0u, 1u) == 0u) {
    status[1] = kKernPrefixTc;
    status[2] = site;
    status[3] = blockIdx.x;
    __threadfence();
  }
}

// The walk over an item's key tiles: shard, first row in the shard, keys in use.
struct Walk {
  const int32_t* off;  // [C + 1] first tile of every shard
  int r, t;
  __device__ __forceinline__ Walk(const int32_t* o, int first) : off(o), r(0), t(first) {
    while (off[r + 1] <= t) ++r;
  }
  __device__ __forceinline__ void next() {
    ++t;
    while (off[r + 1] <= t) ++r;  // not past the last tile: the caller stops there
  }
};

struct alignas(16) Shared {
  // E4M3: unit[0..2] K tiles landed, unit[3..5] V tiles landed, unit[6..8] V tiles converted,
  // rel[4..6] a tile's scales written
  uint64_t bar_unit[10], bar_rel[10], bar_s[2], bar_p[2], bar_o[2], bar_never, bar_drain;
  uint32_t tmem_slot;
  volatile int abort_flag;
  volatile int zero_flag;  // never set: drains ignore the abort flag
  int32_t tile_off[CP_MAX_SHARDS + 2];
  int32_t rows[CP_MAX_SHARDS], row_off[CP_MAX_SHARDS];
  cp_prefix_item item;
};
struct alignas(16) Scales {  // behind Shared, for an E4M3 cache only
  float scale[3][BN];  // the tokens' of the last three tiles, read in pieces of four
  float inv[2 * BM];   // what undoes the rows' powers of two
};

template <int D, bool WIDE, int MAXC, bool F8>
__device__ __noinline__ void process(const Params& p, const Maps<MAXC>& maps, Shared& sh, uint8_t* sQ,
                                        uint32_t tmem) {
  using C = Cfg<D, F8>;
  uint8_t* sKV = sQ + C::kRing;
  constexpr int kUnitBars = C::kSlots;
  // E4M3: V's code tiles, the third one where a second M tile of queries would be
  constexpr int kVSlots = WIDE ? 2 : 3;
  auto v_codes = [&](int j) {
    const int slot = j % kVSlots;
    return sQ + (slot < 2 ? C::kCodes + (C::kKSlots + slot) * C::kCodeBytes : C::kQBytes);
  };
  // keys of the item's tile j, where a row of it has a NaN code (rows behind them may have
  // any, and meet weights of 0: they stay finite)
  auto keys_of = [&](int j) {
    const Walk w(sh.tile_off, sh.item.tile_begin + j);
    return sh.rows[w.r] - (w.t - w.off[w.r]) * BN;
  };
  constexpr int kRels = F8 ? 3 : C::kSlots;  // barriers of the releases
  constexpr int NS = WIDE ? 128 : 64;  // score columns of a chain
  constexpr int NC = NS / 2;           // of one half of a row
  // Score columns in registers at a time: all of a half's and their P need more registers than
  // a thread has (80 over E4M3, with its further warps: 64 x 32 heads behind 131,072 tokens took
  // 516 us and take 182, 16 x 32 heads 117 and 95; bf16, 96 registers: 300 x 64 heads 124 and 119)
  constexpr int NB = 16;
  // a half row's P sum that can hide a P above 2^8
  constexpr float kSpecSum = NC * 256.f;
  const PrefixArgs& a = p.a;
  const cp_prefix_item& it = sh.item;
  Scales& sc = *reinterpret_cast<Scales*>(&sh + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nK = it.tile_end - it.tile_begin;
  volatile int* abort = &sh.abort_flag;

  if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3, t = (warp >> 2) & 1, half = warp >> 3;
    const int i = quarter * 32 + lane;  // row within the M tile = TMEM lane
    const int pbar = 2 + t * 4 + quarter;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t colS = t * 256 + NC * half, colO = t * 256 + 128 + (D / 2) * half;
    const int row = (WIDE ? t * BM : 0) + i;  // row of the block
    const bool releaser = t == 1 && quarter == 0 && half == 0;  // frees K/V slots
    // value of the other half of this row, through the last of its S columns, which
    // P never covers and which S no longer needs once a tile's values are in registers
    auto exchange = [&](float v) -> float {
      tmem_st1(lane_addr + t * 256 + NC * half + NC - 1, __float_as_uint(v));
      tmem_st_wait();
      tc_fence_before();
      named_bar_sync(pbar, 64);
      tc_fence_after();
      const uint32_t o = tmem_ld1(lane_addr + t * 256 + NC * (half ^ 1) + NC - 1);
      tmem_ld_wait();
      return __uint_as_float(o);
    };
    // rows of the block in use by this warp (a single chain's block may leave quarters empty)
    const bool idle = !WIDE && quarter * 32 >= it.m_rows;
    const float inv_row = F8 ? sc.inv[row] : 1.f;
    const float sl2 = p.scale_log2 * inv_row;
    float m_used = -INFINITY, l = 0.f;
    bool ok = true, first = true;  // first: no key of this chain so far
    int keys = 0;                  // of this half's columns, those in use in this tile
    const float* scales = nullptr;  // E4M3: of this half's columns
    auto load_s = [&](int c0, uint32_t (&sr)[NB]) {  // columns [c0, c0 + NB) of the half
      tmem_ld16(lane_addr + colS + c0, sr);
      tmem_ld_wait();
      if constexpr (F8) {
#pragma unroll
        for (int e = 0; e < NB; e += 4) {
          const float4 k = *reinterpret_cast<const float4*>(scales + c0 + e);
          sr[e] = __float_as_uint(__uint_as_float(sr[e]) * k.x);
          sr[e + 1] = __float_as_uint(__uint_as_float(sr[e + 1]) * k.y);
          sr[e + 2] = __float_as_uint(__uint_as_float(sr[e + 2]) * k.z);
          sr[e + 3] = __float_as_uint(__uint_as_float(sr[e + 3]) * k.w);
        }
      }
      if (keys < c0 + NB) {
#pragma unroll
        for (int e = 0; e < NB; ++e)
          if (c0 + e >= keys) sr[e] = __float_as_uint(-INFINITY);
      }
    };
    auto exps = [&](int c0, const uint32_t (&sr)[NB], uint32_t (&pk)[NC / 2]) -> float {
      const float neg = -m_used * sl2;
      float s0sum = 0.f, s1sum = 0.f;
#pragma unroll
      for (int e = 0; e < NB / 2; ++e) {
        float u0, u1;
        fma2(u0, u1, __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]), sl2, sl2, neg, neg);
        const float p0 = ex2(u0), p1 = ex2(u1);
        add2(s0sum, s1sum, s0sum, s1sum, p0, p1);
        if constexpr (F8) {
          const float2 k = *reinterpret_cast<const float2*>(scales + c0 + 2 * e);
          pk[c0 / 2 + e] = pack_bf16x2(p0 * k.x, p1 * k.y);
        } else {
          pk[c0 / 2 + e] = pack_bf16x2(p0, p1);
        }
      }
      return s0sum + s1sum;
    };
    const bool helps = F8 && !WIDE && it.m_rows <= kHelpRows && quarter >= 2;
    if (helps) {
      // 32 of the chain's 64 rows of V, one half of the dims.  V_(j+1) goes where V_(j-1) was, and
      // the chain's product with that one is complete when its S_j is; this warp's arrival on
      // P_(j+1) covers it.
      const int vrow = 64 * t + (quarter - 2) * 32 + lane;
      for (int j = -1; j < nK; ++j) {
        bool got = j < 0 || mbar_wait(smem_u32(&sh.bar_s[t]), j & 1, p.wait_ns, abort);
        if (got && j >= 0) mbar_arrive(smem_u32(&sh.bar_p[t]));
        const int v = j + 1;
        if (got && v < nK) got = mbar_wait(smem_u32(&sh.bar_unit[3 + v % kVSlots]), (v / kVSlots) & 1, p.wait_ns, abort);
        got = __all_sync(0xffffffffu, got);
        if (!got) {
          if (lane == 0) report_timeout(p.status, 6, abort);
          ok = false;
          break;
        }
        if (v == nK) break;
        uint8_t* to = sKV + (v % C::kSlots) * C::kSlotBytes + vrow * 128;
        if (convert_row<4>(v_codes(v) + vrow * 128, to, vrow, 4 * half) && vrow < keys_of(v)) nan_codes(v_codes(v) + vrow * 128, to, vrow, 4 * half, 4);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sh.bar_unit[6 + v % kVSlots]));
      }
    }
    Walk w(sh.tile_off, it.tile_begin);
    for (int j = helps ? nK : 0; j < nK && ok; ++j) {
      const int nv = min(BN, sh.rows[w.r] - (w.t - w.off[w.r]) * BN);  // keys of the tile
      const int chain = WIDE ? nv : nv - 64 * t;                      // of the chain
      keys = chain - NC * half;
      if (j + 1 < nK) w.next();
      bool got = mbar_wait(smem_u32(&sh.bar_s[t]), j & 1, p.wait_ns, abort);
      if constexpr (F8) {
        got = got && mbar_wait(smem_u32(&sh.bar_rel[4 + j % 3]), (j / 3) & 1, p.wait_ns, abort);
        scales = sc.scale[j % 3] + (WIDE ? 0 : 64 * t) + NC * half;
      }
      got = __all_sync(0xffffffffu, got);
      if (idle) {  // no row of the block: O of these lanes is never read; no votes
        if (!got) {
          if (lane == 0) report_timeout(p.status, 1, abort);
          ok = false;
          break;
        }
        mbar_arrive(smem_u32(&sh.bar_p[t]));
        continue;
      }
      if (got && releaser && lane == 0) mbar_arrive(smem_u32(&sh.bar_rel[j % kRels]));
      tc_fence_after();
      uint32_t sr[NB], pk[NC / 2];
      float part = 0.f;
      const bool fresh = WIDE ? j == 0 : first;
      bool slow = WIDE ? fresh : fresh && chain > 0;
      if (!fresh) {
        // P with the running max as it stands: a half whose P sums past NC x 2^8
        // holds a P above 2^8 (or a NaN), and the row takes the exact path
#pragma unroll
        for (int c0 = 0; c0 < NC; c0 += NB) {
          load_s(c0, sr);
          part += exps(c0, sr, pk);
        }
        slow = bar_red_or(pbar, 64, !got || !(part <= kSpecSum));
      } else if (!WIDE && chain <= 0) {  // nothing to weigh yet
        if (bar_red_or(pbar, 64, !got)) slow = true;
#pragma unroll
        for (int e = 0; e < NC / 2; ++e) pk[e] = 0;
      }
      if (slow) {
        // both warps of these rows leave together: one that gave up meets the other at this vote
        if (bar_red_or(pbar, 64, !got)) {
          if (!got) report_timeout(p.status, 1, abort);
          ok = false;
          break;
        }
        float mx = -INFINITY;
#pragma unroll
        for (int c0 = 0; c0 < NC; c0 += NB) {
          load_s(c0, sr);
#pragma unroll
          for (int e = 0; e < NB / 2; ++e) mx = fmax3(mx, __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
        }
        const float mrow = fmaxf(mx, exchange(mx));
        if (fresh) {
          m_used = mrow;
          first = false;
        } else {
          // Each row moves its own max; the wait and the pair's barrier are taken by every lane
          const bool need = (mrow - m_used) * sl2 > kRescaleLog2;
          const float alpha = need ? ex2((m_used - mrow) * sl2) : 1.f;
          if (need) {
            l *= alpha;
            m_used = mrow;
          }
          const bool landed = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.bar_o[t]), (j - 1) & 1, p.wait_ns, abort));
          if (bar_red_or(pbar, 64, !landed)) {
            if (!landed) report_timeout(p.status, 2, abort);
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[16];
            tmem_ld16(lane_addr + colO + c * 16, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st16(lane_addr + colO + c * 16, r);
          }
        }
        // the last columns, whose place in TMEM the exchange took, are still in registers; the
        // sum goes by rising column as above, so that a row's bits do not depend on whether
        // another row of the warp takes this path
        const float last = exps(NC - NB, sr, pk);
        part = 0.f;
#pragma unroll
        for (int c0 = 0; c0 < NC - NB; c0 += NB) {
          load_s(c0, sr);
          part += exps(c0, sr, pk);
        }
        part += last;
      }
      l += part;
      if constexpr (NC == 64) tmem_st32(lane_addr + colS, pk);
      else tmem_st16(lane_addr + colS, pk);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(smem_u32(&sh.bar_p[t]));
    }
    // ------------------------------------------------------------ epilogue
    const bool landed = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.bar_o[t]), (nK - 1) & 1, p.wait_ns, abort));
    const bool failed = bar_red_or(1, kSoftmaxWarps * 32, !landed);
    if (failed) {
      if (ok && !landed) report_timeout(p.status, 3, abort);
    } else {
      tc_fence_after();

      float lt = l + exchange(l);
      float w0 = 1.f;
      // Every product of the item is complete (both chains' last ones were waited for), so the
      // K/V ring is free.  O of chain 1 [dim][row], its running max and sum; the block's results
      float* other = reinterpret_cast<float*>(sKV);
      float *other_m = other + D * BM, *other_l = other_m + BM;
      float4* out = reinterpret_cast<float4*>(sKV + (WIDE ? 0 : (D + 2) * BM * 4));
      float* out_lse = reinterpret_cast<float*>(out + (WIDE ? 2 : 1) * BM * (D / 4));
      if (!WIDE) {
        if (t == 1) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[16];
            tmem_ld16(lane_addr + colO + c * 16, r);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) other[((D / 2) * half + c * 16 + e) * BM + i] = __uint_as_float(r[e]);
          }
          if (half == 0) {
            other_m[i] = m_used;
            other_l[i] = lt;
          }
        }
        named_bar_sync(1, kSoftmaxWarps * 32);
      }
      if (WIDE || t == 0) {
        float w1 = 0.f;
        if (!WIDE) {
          // either chain may have had no key (max -inf, sum 0)
          const float m1 = other_m[i], mm = fmaxf(m_used, m1);
          w0 = m_used == -INFINITY ? 0.f : ex2((m_used - mm) * sl2);
          w1 = m1 == -INFINITY ? 0.f : ex2((m1 - mm) * sl2);
          lt = lt * w0 + other_l[i] * w1;
          m_used = mm;
        }
        const float inv = 1.f / lt;
        w0 *= inv;
        w1 *= inv;
        // O and the LSE of this half of the row to shared memory, pieces of four dims
        // rotated by the row (a column of pieces would share its banks).  This code runs
        // once an item, out of the instruction cache: short loops.
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t r[16];
          tmem_ld16(lane_addr + colO + c * 16, r);
          tmem_ld_wait();
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[e] = __uint_as_float(r[4 * v + e]) * w0;
              if (!WIDE) x[e] += other[((D / 2) * half + c * 16 + 4 * v + e) * BM + i] * w1;
            }
            const int piece = (D / 8) * half + c * 4 + v;
            out[row * (D / 4) + (piece ^ (i & 7))] = make_float4(x[0], x[1], x[2], x[3]);
          }
        }
        if (half == 0) out_lse[row] = m_used * (a.sm_scale * inv_row) + logf(lt);
        // ... and from there whole rows at a time to global memory: the two warps of these
        // 32 rows take every other one
        named_bar_sync(pbar, 64);
        constexpr int kLanes = D / 4, kRows = 32 / kLanes;  // lanes a row, rows a warp at a time
        constexpr int kSteps = 16 / kRows, kBatch = 4;
        const int piece = lane % kLanes, x0 = half * kRows + lane / kLanes;
        const int base = row - i + quarter * 32, rows = min(32, it.m_rows - base);
        const bool direct = it.alone && a.P == 0;
#pragma unroll 1
        for (int b = 0; b < kSteps; b += kBatch) {
          float4 v[kBatch];
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int x = x0 + 2 * kRows * (b + k);
            v[k] = out[(base + x) * (D / 4) + (piece ^ (x & 7))];
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int x = x0 + 2 * kRows * (b + k);
            if (x >= rows) continue;
            if (!direct) {
              const long long at = (long long)it.part * kPrefixRows + base + x;
              reinterpret_cast<float4*>(a.ws_o + at * D)[piece] = v[k];
              if (piece == 0) a.ws_lse[at] = out_lse[base + x];
            } else {
              const int m = it.m0 + base + x, n = p.by_g(m);
              const long long at = (long long)(it.row0 + n) * a.Hq + it.kv_head * a.G + m - n * a.G;
              if (a.o_bf16)
                reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at * D)[piece] = make_uint2(pack_bf16x2(v[k].x, v[k].y), pack_bf16x2(v[k].z, v[k].w));
              else
                reinterpret_cast<float4*>(static_cast<float*>(a.o) + at * D)[piece] = v[k];
              if (piece == 0) a.lse[at] = out_lse[base + x];
            }
          }
        }
      }
    }
  } else if (warp == kWarpTma) {
    // ------------------------------------------------------------ TMA producer
    int last_unit = 0;  // K_0: loaded before the block's barrier
    bool ok = true;
    int v0 = 0, v1 = 0, vr = 0;  // V's: the K of the unit before
    // The rows to load are known before the wait that frees their slots: a tile's
    // coordinates come from shared memory or the page table while the one before it is
    // on its way, and V's are K's of the step before.
    Walk w(sh.tile_off, it.tile_begin);
    int y0 = 0, y1 = 0, yr = 0;  // of tile w.t: its rows' coordinate (of both halves in a pool) and shard
    auto locate = [&]() {
      const int row = (w.t - w.off[w.r]) * BN;
      yr = w.r;
      if (!a.rm.table) {
        y0 = sh.row_off[w.r] + row;
      } else {
        // two 64-row halves, each inside one page; a half behind the pair's rows lies past
        // the pool and reads zeros
        const int pair = w.r * a.R + it.group;
        y0 = (int)map_row_early(a.rm, pair, 0, row);
        y1 = row + 64 < sh.rows[w.r] ? (int)map_row_early(a.rm, pair, 0, row + 64) : (int)a.rm.pool_rows;
        yr = 0;
      }
    };
    auto load = [&](const CUtensorMap* map, int c0, int c1, uint32_t dst, uint32_t full) {
      // a code row is one chunk of 128 bytes
#pragma unroll
      for (int c = 0; c < (F8 ? 1 : C::kChunks); ++c) {
        tma_load_3d(dst + c * (BN * 128), map, c * 64, it.kv_head, c0, full);
        if (a.rm.table) tma_load_3d(dst + c * (BN * 128) + 64 * 128, map, c * 64, it.kv_head, c1, full);
      }
    };
    if constexpr (F8) {
      uint8_t* codes = sQ + C::kCodes;
      locate();
      int nk = 1, nv = 0;  // tiles loaded (K_0 before the block's barrier)
      int v0 = y0, v1 = y1, vr = yr;
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        if (__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.wait_ns, abort))) return true;
        if (lane == 0) report_timeout(p.status, 4, abort);
        return false;
      };
      for (int j = 0; j < nK; ++j) {  // V_j, then K_(j+1)
        if (nv >= kVSlots && !wait_all(&sh.bar_unit[6 + nv % kVSlots], (nv / kVSlots - 1) & 1)) break;
        if (elect_one()) {
          const uint32_t full = smem_u32(&sh.bar_unit[3 + nv % kVSlots]);
          mbar_expect_tx(full, C::kCodeBytes);
          load(&maps.v[vr], v0, v1, smem_u32(v_codes(nv)), full);
        }
        __syncwarp();
        ++nv;
        if (nk == nK) continue;
        w.next();
        locate();
        v0 = y0;
        v1 = y1;
        vr = yr;
        // K_(nk - 3) is read once S_(nk - 3) is complete
        if (nk >= C::kKSlots && !wait_all(&sh.bar_rel[(nk - C::kKSlots) % 3], ((nk - C::kKSlots) / 3) & 1)) break;
        if (elect_one()) {
          const uint32_t full = smem_u32(&sh.bar_unit[nk % C::kKSlots]);
          mbar_expect_tx(full, C::kCodeBytes);
          load(&maps.k[yr], y0, y1, smem_u32(codes + nk % C::kKSlots * C::kCodeBytes), full);
        }
        __syncwarp();
        ++nk;
      }
      // never leave with a copy in flight: the last fill of every slot
      for (int u = max(0, nk - C::kKSlots); u < nk; ++u)
        mbar_wait(smem_u32(&sh.bar_unit[u % C::kKSlots]), (u / C::kKSlots) & 1, 1000000000ull, &sh.zero_flag);
      for (int u = max(0, nv - kVSlots); u < nv; ++u)
        mbar_wait(smem_u32(&sh.bar_unit[3 + u % kVSlots]), (u / kVSlots) & 1, 1000000000ull, &sh.zero_flag);
      __syncwarp();
      return;
    }
    locate();
    v0 = y0;
    v1 = y1;
    vr = yr;
    if (nK > 1) {
      w.next();
      locate();
    }
    for (int k = 1; k <= nK && ok; ++k) {
      // load u = 2j (K_j) or 2j + 1 (V_j) goes to slot u % kSlots; unit k = {V_(k-1), K_k}
      const int u0 = 2 * k - 1, u1 = k == nK ? 2 * k - 1 : 2 * k;
      for (int u = u0; u <= u1 && ok; ++u) {
        if (u < C::kSlots) continue;             // the slot's first load
        const int r = (u - C::kSlots + 1) >> 1;  // the release of load u - kSlots
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.bar_rel[r % C::kSlots]), (r / C::kSlots) & 1, p.wait_ns, abort))) {
          if (lane == 0) report_timeout(p.status, 4, abort);
          ok = false;
        }
      }
      if (!ok) break;
      const uint32_t full = smem_u32(&sh.bar_unit[k % kUnitBars]);
      const uint32_t v_slot = smem_u32(sKV + ((2 * k + C::kSlots - 1) % C::kSlots) * C::kSlotBytes);
      const uint32_t k_slot = smem_u32(sKV + ((2 * k) % C::kSlots) * C::kSlotBytes);
      if (elect_one()) {
        mbar_expect_tx(full, (u1 - u0 + 1) * C::kSlotBytes);
        load(&maps.v[vr], v0, v1, v_slot, full);
        if (k < nK) load(&maps.k[yr], y0, y1, k_slot, full);
      }
      __syncwarp();
      v0 = y0;
      v1 = y1;
      vr = yr;
      if (k + 1 < nK) {
        w.next();
        locate();
      }
      last_unit = k;
    }
    // never leave with a copy in flight: the last unit of every barrier
    for (int k = max(0, last_unit - kUnitBars + 1); k <= last_unit; ++k)
      mbar_wait(smem_u32(&sh.bar_unit[k % kUnitBars]), (k / kUnitBars) & 1, 1000000000ull, &sh.zero_flag);
    __syncwarp();
  } else if (F8 && warp >= kWarpRelay) {
    // ------------------------------------------------------------ V's codes to bf16 (a thread a row)
    bool ok = true;
    const int row = (warp - kWarpRelay) * 32 + lane;
    Walk w(sh.tile_off, it.tile_begin);
    auto scale_of = [&]() -> float {  // of this row of tile w.t; 0 behind the shard's last key
      const int in_pair = (w.t - w.off[w.r]) * BN + row, pair = w.r * a.R + it.group;
      if (in_pair >= sh.rows[w.r]) return 0.f;
      return __ldcg(a.sc.p[w.r] + (a.rm.table ? map_row_early(a.rm, pair, 0, in_pair) : (long long)sh.row_off[w.r] + in_pair));
    };
    auto put_scale = [&](int j, float x) {
      sc.scale[j % 3][row] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.bar_rel[4 + j % 3]));
    };
    put_scale(0, scale_of());
    for (int j = 0; j < nK && ok; ++j) {
      float scale = 0.f;
      if (j + 1 < nK) {
        w.next();
        scale = scale_of();
      }
      // V_j has landed; its bf16 slot's V_(j-2) is read (release j - 1: S_(j-1) is complete)
      ok = mbar_wait(smem_u32(&sh.bar_unit[3 + j % kVSlots]), (j / kVSlots) & 1, p.wait_ns, abort);
      if (ok && j >= C::kSlots) ok = mbar_wait(smem_u32(&sh.bar_rel[(j - 1) % kRels]), ((j - 1) / kRels) & 1, p.wait_ns, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) report_timeout(p.status, 5, abort);
        break;
      }
      // rows behind the shard's last key meet weights of 0: any finite value will do (a NaN code's, too)
      if (it.m_rows > kHelpRows) {
        uint8_t* to = sKV + (j % C::kSlots) * C::kSlotBytes + row * 128;
        if (convert_row<8>(v_codes(j) + row * 128, to, row, 0) && row < keys_of(j)) nan_codes(v_codes(j) + row * 128, to, row, 0, 8);
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sh.bar_unit[6 + j % kVSlots]));
      if (j + 1 < nK) {
        // V_(j-2) was free: both chains are done with P_(j-2), whose scales these replace
        put_scale(j + 1, scale);
        ok = mbar_wait(smem_u32(&sh.bar_unit[(j + 1) % C::kKSlots]), ((j + 1) / C::kKSlots) & 1, p.wait_ns, abort);
      }
      // V_j and K_(j+1) are in place: this warp's arrival on both chains' P_j
      for (int t = 0; t < 2; ++t) {
        if (j > 0) ok = ok && mbar_wait(smem_u32(&sh.bar_p[t]), (j - 1) & 1, p.wait_ns, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane == 0) mbar_arrive(smem_u32(&sh.bar_p[t]));
      }
      if (!ok && lane == 0) report_timeout(p.status, 17, abort);
    }
  } else if (warp == kWarpRelay) {
    // ------------------------------------------------------------ relay
    bool ok = true;
    Walk w(sh.tile_off, it.tile_begin);
    for (int j = 0; j < nK && ok; ++j) {
      const int nv = sh.rows[w.r] - (w.t - w.off[w.r]) * BN;
      if (j + 1 < nK) w.next();
      ok = __all_sync(0xffffffffu,
                      mbar_wait(smem_u32(&sh.bar_unit[(j + 1) % kUnitBars]), ((j + 1) / kUnitBars) & 1, p.wait_ns, abort));
      if (ok && nv < BN) {
        // rows of V behind the shard's last key: another group's, or a page's tail; they
        // meet weights of 0 and must not be infinite or NaN
        uint8_t* v = sKV + ((2 * j + 1) % C::kSlots) * C::kSlotBytes;
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c)
          for (int x = nv * 8 + lane; x < BN * 8; x += 32)
            reinterpret_cast<uint4*>(v + c * (BN * 128))[x] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      }
      for (int t = 0; t < 2 && ok; ++t) {
        if (j > 0) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&sh.bar_p[t]), (j - 1) & 1, p.wait_ns, abort));
        if (ok && lane == 0) mbar_arrive(smem_u32(&sh.bar_p[t]));
        __syncwarp();
      }
      if (!ok && lane == 0) report_timeout(p.status, 17, abort);
    }
  } else {
    // ------------------------------------------------------------ MMA issuer
    constexpr unsigned kAll = 0xffffffffu;
    const uint32_t idS = F8 ? idesc_e4m3_f32(BM, NS, 0, 0) : idesc_bf16_f32(BM, NS, 0, 0);
    const uint32_t idPV = idesc_bf16_f32(BM, D, 0, 1);
    auto fail = [&](unsigned site) {
      if (lane == 0) report_timeout(p.status, site, abort);
    };
    auto wait_all = [&](uint64_t* bar, uint32_t parity) {
      return __all_sync(kAll, mbar_wait(smem_u32(bar), parity, p.wait_ns, abort));
    };
    const uint64_t dQ0 = smem_desc(smem_u32(sQ), 16, 1024);
    const uint64_t dK0 = smem_desc(smem_u32(sKV), 16, 1024);
    const uint64_t dV0 = smem_desc(smem_u32(sKV), BN * 128, 1024);
    auto issue_s = [&](int t, int j) {
      const uint64_t a0 = dQ0 + (uint64_t)((WIDE ? t * C::kQBytes : 0) >> 4);
      // the chain's 64 keys are the tile's rows 64 t on: 8 KB into every chunk
      const int chain = WIDE ? 0 : t * 64 * 128;
      if (elect_one()) {
        if constexpr (F8) {  // hi, then lo, which stands behind it
          const uint64_t b0 = dQ0 + (uint64_t)((C::kCodes + j % C::kKSlots * C::kCodeBytes + chain) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss_f8(tmem + t * 256, a0 + (((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4), b0 + (((kk & 3) * 32) >> 4), idS, kk > 0);
        } else {
          const uint64_t b0 = dK0 + (uint64_t)((((2 * j) % C::kSlots) * C::kSlotBytes + chain) >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
            mma_ss(tmem + t * 256, a0 + off, b0 + off, idS, kk > 0);
          }
        }
        mma_commit(smem_u32(&sh.bar_s[t]));
      }
      __syncwarp();
    };
    auto issue_pv = [&](int t, int j, bool acc) {
      const int slot = (F8 ? j : 2 * j + 1) % C::kSlots;
      const uint64_t v0 = dV0 + (uint64_t)((slot * C::kSlotBytes + (WIDE ? 0 : t * 64 * 128)) >> 4);
      const uint32_t pa = tmem + t * 256, d = tmem + t * 256 + 128;
      if (elect_one()) {
        // P of a half's NC keys sits over the first NC / 2 of its NC columns
        constexpr int kHalf = NC / 16;
#pragma unroll
        for (int kk = 0; kk < NS / 16; ++kk)
          mma_ts(d, pa + (kk / kHalf) * NC + (kk % kHalf) * 8, v0 + (uint64_t)((kk * 16 * 128) >> 4), idPV, (acc || kk > 0) ? 1u : 0u);
        mma_commit(smem_u32(&sh.bar_o[t]));
      }
      __syncwarp();
    };
    bool ok = true;
    if (p.stall_test && !wait_all(&sh.bar_never, 0)) {
      fail(10);
      ok = false;
    }
    if (ok && !wait_all(&sh.bar_unit[0], 0)) {
      fail(12);
      ok = false;
    }
    if (ok) {
      tc_fence_after();
      issue_s(0, 0);
      issue_s(1, 0);
    }
    for (int j = 0; j < nK && ok; ++j) {
      for (int t = 0; t < 2 && ok; ++t) {
        // V_j and K_(j+1) are in place once the chain's P_j has completed (the relay's arrival)
        if (!wait_all(&sh.bar_p[t], j & 1)) {
          fail(14 + t);
          ok = false;
          break;
        }
        tc_fence_after();
        issue_pv(t, j, j > 0);
        if (j + 1 < nK) issue_s(t, j + 1);
      }
    }
    // never go on under a running product
    if (elect_one()) mma_commit(smem_u32(&sh.bar_drain));
    __syncwarp();
    mbar_wait(smem_u32(&sh.bar_drain), 0, 1000000000ull, &sh.zero_flag);
  }
}

// the tiles and what stands behind them: at most 227 KB a block
template <int D, bool F8>
constexpr int kSmem = Cfg<D, F8>::kTiles + (int)sizeof(Shared) + (F8 ? (int)sizeof(Scales) : 0);
static_assert(kSmem<128, false> <= 232448 && kSmem<64, false> <= 232448 && kSmem<128, true> <= 232448, "shared memory");

template <int D, int MAXC, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ Maps<MAXC> maps, const __grid_constant__ Params p) {
  using C = Cfg<D, F8>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::kTiles);
  const PrefixArgs& a = p.a;
  const int warp = threadIdx.x >> 5;
  if (warp == kWarpTma)  // the descriptors' own latency, before the first load needs them
    for (int r = threadIdx.x & 31; r < (a.rm.table ? 1 : a.C); r += 32) {
      prefetch_tmap(&maps.k[r]);
      prefetch_tmap(&maps.v[r]);
    }
  const int w0 = a.plan[a.off_worker + blockIdx.x], w1 = a.plan[a.off_worker + blockIdx.x + 1];
  if (w0 == w1) return;
  constexpr int kBars = (int)(offsetof(Shared, tmem_slot) / 8);  // a lane each
  static_assert(kBars <= 32, "barriers");
  if (warp == kWarpMma) tmem_alloc(smem_u32(&sh.tmem_slot), 512);
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    sh.zero_flag = 0;
  }
  // the plan comes by copies, never from a kernel: it may be read before the kernel
  // before this one ends
  cp_prefix_item it = reinterpret_cast<const cp_prefix_item*>(a.plan + a.off_item)[w0];
  wait_for_earlier_kernels();
  for (int wi = w0; wi < w1; ++wi) {
    // What an item's first product waits for comes in one step after the item itself:
    // the first K tile, the block's queries and the group's tables.
    if (wi > w0) it = reinterpret_cast<const cp_prefix_item*>(a.plan + a.off_item)[wi];
    if (warp == kWarpTma) {
      const int lane = threadIdx.x & 31;
      if (lane < kBars) {
        uint64_t* b = reinterpret_cast<uint64_t*>(&sh) + lane;
        if (wi > w0) mbar_inval(smem_u32(b));
        const bool is_p = b == &sh.bar_p[0] || b == &sh.bar_p[1];
        const bool converted = F8 && b >= &sh.bar_unit[6] && b <= &sh.bar_unit[8], scaled = F8 && b >= &sh.bar_rel[4] && b <= &sh.bar_rel[6];
        mbar_init(smem_u32(b), is_p ? 2 * BM + C::kRelays : converted ? (it.m_rows <= kHelpRows ? 12 : 4) : scaled ? 4 : 1);
        mbar_init_fence();
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        // K_0 (more of the ring here would hold up the block's barrier)
        int y0 = it.first_y, y1 = 0;
        if (a.rm.table) {
          const int pair = it.first_shard * a.R + it.group;
          y0 = (int)map_row_early(a.rm, pair, 0, it.first_row);
          y1 = it.first_row + 64 < it.first_rows ? (int)map_row_early(a.rm, pair, 0, it.first_row + 64) : (int)a.rm.pool_rows;
        }
        const CUtensorMap* map = &maps.k[a.rm.table ? 0 : it.first_shard];
        const uint32_t full = smem_u32(&sh.bar_unit[0]), dst = smem_u32(F8 ? sQ + C::kCodes : sQ + C::kRing);
        mbar_expect_tx(full, F8 ? C::kCodeBytes : C::kSlotBytes);
#pragma unroll
        for (int c = 0; c < (F8 ? 1 : C::kChunks); ++c) {
          tma_load_3d(dst + c * (BN * 128), map, c * 64, it.kv_head, y0, full);
          if (a.rm.table) tma_load_3d(dst + c * (BN * 128) + 64 * 128, map, c * 64, it.kv_head, y1, full);
        }
        sh.item = it;
      }
    } else if (warp < kSoftmaxWarps) {
      // queries to shared memory (128-byte-swizzled K-major): 16 bytes a thread, a row's
      // pieces side by side, four loads before their stores
      constexpr int kPieces = D / 8, kStep = kSoftmaxWarps * 32, kBatch = 4;
      const int count = (it.m_rows > BM ? 2 * BM : BM) * kPieces;
#pragma unroll 1
      for (int e0 = threadIdx.x; e0 < count; e0 += kBatch * kStep) {
        uint4 val[kBatch];
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int e = e0 + x * kStep, r = e / kPieces, m = it.m0 + r, n = p.by_g(m);
          val[x] = make_uint4(0, 0, 0, 0);
          if (r < it.m_rows)
            val[x] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                           ((long long)(it.row0 + n) * a.Hq + it.kv_head * a.G + m - n * a.G) * D) + e % kPieces);
        }
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const int e = e0 + x * kStep, r = e / kPieces, c = e % kPieces;
          if (e >= count) continue;
          if constexpr (F8) {
            put_codes(val[x], sQ + (r >> 7) * C::kQBytes + (r & 127) * 128, r & 7, c, &reinterpret_cast<Scales*>(&sh + 1)->inv[r]);
          } else {
            *reinterpret_cast<uint4*>(sQ + (r >> 7) * C::kQBytes + (c >> 3) * (BM * 128) + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4)) = val[x];
          }
        }
      }
      fence_proxy_async_smem();
    } else {
      for (int r = threadIdx.x - kWarpMma * 32; r <= a.C; r += C::kThreads - kWarpMma * 32) {
        sh.tile_off[r] = a.plan[a.off_tiles + it.group * (a.C + 1) + r];
        if (r < a.C) {
          const cp_pair_desc* pd = reinterpret_cast<const cp_pair_desc*>(a.plan + a.off_pair) + r * a.R + it.group;
          sh.rows[r] = pd->rows;
          sh.row_off[r] = pd->row_off;
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_slot;
    if (sh.item.m_rows > BM) process<D, true, MAXC, F8>(p, maps, sh, sQ, tmem);
    else process<D, false, MAXC, F8>(p, maps, sh, sQ, tmem);
    fence_proxy_async_smem();  // the next item's copies come after this one's reads and writes
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (sh.abort_flag) break;
  }
  if (warp == kWarpMma) tmem_dealloc(sh.tmem_slot, 512);
}

// [rows, H, D] as 3-D (D, H, rows); boxes of 128-byte rows, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, long long rows, int H, int D, int box_rows, bool f8) {
  if (f8) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)H, (uint64_t)rows}, strides[2] = {(uint64_t)D, (uint64_t)H * D};
    const uint32_t box[3] = {(uint32_t)D, 1, (uint32_t)box_rows};
    return encode_tensor_map_u8_3d(m, base, dims, strides, box);
  }
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)H, (uint64_t)rows};
  const uint64_t strides[2] = {(uint64_t)D * 2, (uint64_t)H * D * 2};
  const uint32_t box[3] = {64, 1, (uint32_t)box_rows};
  return encode_tensor_map_bf16(m, base, 3, dims, strides, box, D == 128);
}

template <int D, int MAXC, bool F8>
cudaError_t launch_c(const Params& p, const long long* shard_rows, int workers, cudaStream_t s) {
  const PrefixArgs& a = p.a;
  Maps<MAXC> maps;
  memset(&maps, 0, sizeof(maps));
  if (a.rm.table) {
    if (!make_map(&maps.k[0], a.k.p[0], a.rm.pool_rows, a.Hkv, D, 64, F8) || !make_map(&maps.v[0], a.v.p[0], a.rm.pool_rows, a.Hkv, D, 64, F8))
      return cudaErrorInvalidValue;
  } else {
    for (int r = 0; r < a.C; ++r)
      if (shard_rows[r] > 0 &&
          (!make_map(&maps.k[r], a.k.p[r], shard_rows[r], a.Hkv, D, BN, F8) || !make_map(&maps.v[r], a.v.p[r], shard_rows[r], a.Hkv, D, BN, F8)))
        return cudaErrorInvalidValue;
  }
  const cudaError_t e = cudaFuncSetAttribute(prefix_tc_kernel<D, MAXC, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D, F8>);
  if (e != cudaSuccess) return e;
  return launch_early(prefix_tc_kernel<D, MAXC, F8>, (unsigned)workers, Cfg<D, F8>::kThreads, kSmem<D, F8>, s, 1, maps, p);
}

}  // namespace

bool prefix_tc_supported(cp_dtype kv, int D) { return kv == CP_BF16 ? D == 64 || D == 128 : kv == CP_FP8_E4M3 && D == 128; }

cudaError_t launch_prefix_tc(const PrefixArgs& a, cp_dtype kv, const long long* shard_rows, int workers, bool stall_test, cudaStream_t s) {
  Params p = {a, FastDiv(a.G), 0.f, nullptr, 0, 0};
  p.scale_log2 = a.sm_scale * kLog2e;
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInvalidDevice;
  p.wait_ns = stall_test ? 50000000ull : wait_limit_ns();
  p.stall_test = stall_test ? 1 : 0;
  // the maps travel as kernel arguments: 2 KB of them where eight shards are enough
  const bool few = a.rm.table || a.C <= 8;
  if (kv == CP_FP8_E4M3)
    return few ? launch_c<128, 8, true>(p, shard_rows, workers, s) : launch_c<128, CP_MAX_SHARDS, true>(p, shard_rows, workers, s);
  if (a.D == 128)
    return few ? launch_c<128, 8, false>(p, shard_rows, workers, s) : launch_c<128, CP_MAX_SHARDS, false>(p, shard_rows, workers, s);
  return few ? launch_c<64, 8, false>(p, shard_rows, workers, s) : launch_c<64, CP_MAX_SHARDS, false>(p, shard_rows, workers, s);
}

}  // namespace cpattn

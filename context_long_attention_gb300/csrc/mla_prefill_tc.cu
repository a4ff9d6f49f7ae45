// Causal prefill of multi-head latent attention in its expanded form, on the
// tcgen05 tensor cores (bf16 in, fp32 accumulate).
//
// For a query at position p of its request and head h
//   s_t = sm_scale (q_h[0:128] . k_nope_{t,h} + q_h[128:192] . k_rope_t), t = 0..p
//   LSE = ln sum_t exp(s_t);  O_h = sum_t exp(s_t - LSE) v_{t,h}
// k_nope and v are the two halves of a token's 256-wide row for the head (the
// product of its latent vector with the up-projection, cp_mla_expand); the
// 64 rotated key dims are one vector per token that all heads read ("How GPUs
// Share a Long Context During LLM Inference" §1.2, §1.3: one 576-wide cache
// entry, the latent part and the shared positional part).
//
// The work of one CTA, or of a pair of CTAs, is up to 256 (512) consecutive
// queries for one head, as two M tiles of 128 (256) rows that share every K/V
// tile of 128 keys.  For one rank they are a segment's; a call over all ranks
// takes the requests' tokens as they come (a short request cut into 2 C blocks,
// or a rank's every C-th token, would leave most of a tile empty or masked) and
// writes each row where its rank's order has it.  CTA c of a pair has rows 128 c ..
// 128 c + 127 of each M tile, half of each K tile's keys and half of each V
// tile's dims.  The products of a pair are issued by its even CTA
// (cta_group::2).
//   warps 0-15  softmax: two warps per 32 rows of an M tile, each with half of
//               a row's 128 scores and half of its 128 output dims
//   warp 16     TMA producer
//   warp 17     MMA issuer (of a pair: the even CTA's) and TMEM owner
//   warp 18     relay: adds an arrival to the P barrier of a step once the
//               step's K/V tiles have landed in this CTA, so that the issuer's
//               one wait covers them (a wait costs the issuing thread ~140 clk
//               while the tensor pipe runs dry); clears the last V tile's rows
//               past the last key (another request's rows: a zero weight
//               times a NaN there would be NaN)
// TMEM (512 columns): tile t holds S_t in columns [256t, 256t + 128), O_t in
// [256t + 128, 256t + 256); P (bf16 pairs) goes over the first 32 of a half's
// 64 score columns.
//
// P is rounded to bf16, the type of its product with V on the tensor cores; the
// row's sum, in fp32, takes it before that.  A weight is then off by at most
// 2^-8 of itself and O by 2^-8 of the weights' mean of |v| (relative error against
// 64 bits on the long prompt 0.0023; with the output's rounding alone 0.0017).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "early_launch.cuh"
#include "internal.h"
#include "tc_pair.cuh"

namespace cpattn {
namespace {
using namespace tc;

constexpr int BM = 128;     // query rows of an M tile in one CTA
constexpr int BN = 128;     // keys per K/V tile
constexpr int kNope = 128;  // per-head key dims
constexpr int kRope = 64;   // key dims shared by the heads
constexpr int kDqk = kNope + kRope;
constexpr int kDv = 128;
constexpr int kSoftmaxWarps = 16;
constexpr int kThreads = 32 * (kSoftmaxWarps + 3);
constexpr int kWarpTma = kSoftmaxWarps;
constexpr int kWarpMma = kSoftmaxWarps + 1;
constexpr int kWarpRelay = kSoftmaxWarps + 2;
constexpr int kLaunchBoundThreads = 640;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;      // move the running max when it grows by > 2^8
constexpr float kSpecSum = 64.f * 256.f;  // a half row's P sum that may hide a P above 2^8

constexpr int kQBytes = BM * kDqk * 2;
constexpr int kPiece = BN * 128;  // bytes of 64 dims of a tile's keys
constexpr long long kGroupBytes = 80ll << 20;  // keys and values of a head group: the L2 (129 MB) holds them beside Q and O

template <bool PAIR>
struct Cfg {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kRows = BM * kCtas;                 // rows of an M tile
  static constexpr int kKeys = BN / kCtas;                 // keys of a K tile in one CTA
  static constexpr int kDims = kDv / kCtas;                // dims of a V tile in one CTA
  static constexpr int kKBytes = kKeys * kDqk * 2;
  static constexpr int kVBytes = BN * kDims * 2;
  // Beside Q a pair's halves fit three times.  Whole tiles do not fit twice:
  // one CTA keeps a ring of eight pieces of [128 keys x 64 dims], a step's V_j
  // (two) and K_(j+1) (three) and three of the next step.
  static constexpr int kSlots = PAIR ? 3 : 2;  // barriers in turn; for a pair also tiles
  static constexpr int kRing = PAIR ? kSlots * (kKBytes + kVBytes) : 8 * kPiece;
  static constexpr int kSmem = 2 * kQBytes + kRing + 1024;
};

struct Params {
  const int32_t* plan;
  int off_seg;
  int off_rank;  // all ranks: the ranks' first rows
  int C, R;
  int zigzag;
  int all;        // all ranks: the tile list holds cp_req_tile
  int split;      // one rank of an interleave plan (below)
  int tile_list;
  int n_tiles;
  int row_sub;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  int H;
  int head_group;  // heads whose units run together, tile by tile
  float sm_scale, scale_log2;
  unsigned* status;
  unsigned long long wait_ns;
  int stall_test;  // test hook: the issuer waits on a barrier that nobody arrives at yet
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1,
                                     float c0, float c1) {
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

__device__ void report_timeout(unsigned* status, unsigned site, volatile int* abort) {
  *abort = 1;
  if (atomicCAS(status, 0u, 1u) == 0u) {
    status[1] = kKernMlaPrefill;
    status[2] = site;
    status[3] = blockIdx.x;
    __threadfence();
  }
}

template <bool PAIR>
__global__ void __launch_bounds__(kLaunchBoundThreads, 1)
    mla_prefill_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap ropemap,
                       const Params p) {
  using C = Cfg<PAIR>;
  constexpr int KS = C::kSlots, MT = C::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = smem + 2 * kQBytes;
  uint8_t* sV = sK + KS * C::kKBytes;  // (pair)
  // one CTA: piece g of the order K_0, V_0, K_1, V_1, ... (K_j: 5j .. 5j + 2, V_j: 5j + 3, 5j + 4)
  auto piece = [&](int g) { return sK + (g & 7) * kPiece; };
  // bar_k, bar_v [j % KS]: this CTA's part of K_j (V_j) has landed; waited for
  // tile after tile by the relay (V, and a pair's K) and by the issuer (K of
  // one CTA).  bar_rel[j % KS]: a softmax thread saw S_j of the step's last
  // tile complete, so K_j and V_(j-1) are read (products complete in order).
  // A pair loads K_(j+3) and V_(j+2) after release j.  One CTA loads V_j and
  // the first piece of K_(j+1), which take the pieces of K_(j-1), after release
  // j - 1, and K_(j+1)'s other pieces, which take V_(j-1)'s, after the last
  // P_(j-1) V_(j-1) (bar_o).  Every barrier that the producer waits for comes
  // round again only after products that need the load it is waiting to make,
  // and every landing barrier after products that its waiter lets through: no
  // phase completes unobserved.  (bar_o alternates between two for that.)
  // bar_q, bar_k0, bar_p are waited for by the issuer and live in its CTA;
  // warps arrive there from both CTAs.
  __shared__ __align__(8) uint64_t bar_k[KS], bar_v[KS], bar_rel[KS], bar_k0;
  // bar_ql: a tile's Q rows are in this CTA's shared memory (by TMA, or
  // written by its eight warps); in pairs the relays pass that on to bar_q.
  __shared__ __align__(8) uint64_t bar_ql[2], bar_q[2], bar_s[2], bar_p[2], bar_o[2][2], bar_drain;
  __shared__ int s_row[2][BM];  // output row of each query, -1 past the unit's last (kept here: the loop has no register to spare)
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ volatile int zero_flag;

  wait_for_earlier_kernels();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = PAIR ? (int)cluster_ctarank() : 0;
  const int unit = PAIR ? blockIdx.x >> 1 : blockIdx.x;
  // Units go head group by head group, in a group tile by tile (longest
  // first) over its heads: the keys and values in use stay in the L2, and the
  // long tiles of no head come last.
  const int per_group = p.n_tiles * p.head_group, g0 = unit / per_group, rem = unit - g0 * per_group;
  const int group = min(p.head_group, p.H - g0 * p.head_group);
  const int tile_i = rem / group, h = g0 * p.head_group + rem - tile_i * group;
  cp_tile_desc td;
  cp_seg_desc sg;
  if (p.all) {
    const int4* tile = reinterpret_cast<const int4*>(p.plan + p.tile_list) + 2 * tile_i;  // a cp_req_tile
    const int4 a = tile[0], b = tile[1];
    td.seg = a.x;
    td.q_off = a.y;
    sg.count = a.z;
    sg.first_pos = a.w;
    sg.first_f = b.x;
    sg.kv_base = b.y;
    sg.stride = 1;
  } else {
    td = reinterpret_cast<const cp_tile_desc*>(p.plan + p.tile_list)[tile_i];
    // a pair takes two plan tiles, from every even one of a segment
    if (PAIR && (td.q_off & (2 * MT - 1))) return;
    sg = reinterpret_cast<const cp_seg_desc*>(p.plan + p.off_seg)[td.seg];
  }
  const bool split = p.split;

  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(smem_u32(&bar_k[s]), 1);
      mbar_init(smem_u32(&bar_v[s]), 1);
      mbar_init(smem_u32(&bar_rel[s]), 1);
    }
    mbar_init(smem_u32(&bar_k0), C::kCtas);
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&bar_ql[t]), split ? 8 : 1);
      mbar_init(smem_u32(&bar_q[t]), C::kCtas);
      mbar_init(smem_u32(&bar_p[t]), (8 + 1) * C::kCtas);  // and the relay
      mbar_init(smem_u32(&bar_s[t]), 1);
      for (int k = 0; k < 2; ++k) mbar_init(smem_u32(&bar_o[t][k]), 1);
    }
    mbar_init(smem_u32(&bar_drain), 1);
    abort_flag = 0;
    zero_flag = 0;
    mbar_init_fence();
  }
  if (warp == kWarpMma) {
    if constexpr (PAIR) tmem_alloc_pair(smem_u32(&tmem_slot), 512);
    else tmem_alloc(smem_u32(&tmem_slot), 512);
  }
  if (warp == kWarpTma && lane == 0) {
    prefetch_tmap(&qmap);
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
    prefetch_tmap(&ropemap);
  }

  // Query (from the unit's first) of row i of M tile t.  A block's queries are
  // neighbours and the second tile reads a tile or two of keys more; an
  // interleave run's lie C apart and it would read C / 2 tiles more all alone
  // (a step takes as long for one M tile as for two), so the tiles take every
  // other query.
  auto query = [&](int t, int i) { return split ? 2 * i + t : t * MT + i; };
  const int n_q = min(2 * MT, sg.count - td.q_off);
  const int rows0 = split ? (n_q + 1) / 2 : min(MT, n_q), rows1 = n_q - rows0;
  const int nkv0 = (sg.first_pos + (td.q_off + query(0, rows0 - 1)) * sg.stride + BN) / BN;
  const int nkv1 = rows1 > 0 ? (sg.first_pos + (td.q_off + query(1, rows1 - 1)) * sg.stride + BN) / BN : 0;
  const int nK = max(nkv0, nkv1);
  const int last_t = nkv1 > 0 ? 1 : 0;  // the tile whose products come last in every step
  // rows of V from here on are not the unit's request's (one rank: not its last query's)
  const int n_keys = sg.first_pos + (p.all ? sg.count : (td.q_off + n_q - 1) * sg.stride + 1);
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers are set up
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // One arrival of a whole warp at a barrier of the issuer's CTA.
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) {
      if constexpr (PAIR) mbar_arrive_cluster(map_to_rank(smem_u32(bar), 0));
      else mbar_arrive(smem_u32(bar));
    }
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.wait_ns, &abort_flag)) != 0;
  };

  if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3;
    const int t = (warp >> 2) & 1;
    const int half = warp >> 3;
    const int i = quarter * 32 + lane;  // row within the CTA's part of the M tile = TMEM lane
    const int row = cta * BM + i;       // row within the M tile
    const int pbar = 2 + t * 4 + quarter;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t colS = t * 256 + 64 * half, colO = t * 256 + 128 + (kDv / 2) * half;
    const int rows_t = t ? rows1 : rows0;
    const bool valid = row < rows_t;
    const bool releaser = t == last_t && quarter == 0 && half == 0;
    // value of the other half of this row, through column 63 of each half's
    // scores (P never covers it, and the scores are in registers by then)
    auto exchange = [&](float v) -> float {
      tmem_st1(lane_addr + t * 256 + 64 * half + 63, __float_as_uint(v));
      tmem_st_wait();
      tc_fence_before();
      named_bar_sync(pbar, 64);
      tc_fence_after();
      const uint32_t o = tmem_ld1(lane_addr + t * 256 + 64 * (half ^ 1) + 63);
      tmem_ld_wait();
      return __uint_as_float(o);
    };
    // An interleave run's queries lie C rows apart and come by ordinary loads
    // (others by TMA): this warp's 32 rows of Q, its half of their 24 16-byte
    // pieces, to shared memory (128-byte-swizzled, K-major), neighbouring lanes
    // reading neighbouring pieces, so that a row's 192 bytes come at once.
    if (split) {
      constexpr int kHalf = kDqk / 16;
      uint4 val[kHalf];
#pragma unroll
      for (int k = 0; k < kHalf; ++k) {
        const int e = k * 32 + lane, r = quarter * 32 + e / kHalf, c = half * kHalf + e % kHalf;
        const long long f = (long long)sg.first_f + (long long)(td.q_off + query(t, cta * BM + r)) * sg.stride;
        val[k] = make_uint4(0, 0, 0, 0);
        if (cta * BM + r < rows_t) val[k] = __ldcg(reinterpret_cast<const uint4*>(p.q + (f * p.H + h) * kDqk) + c);
      }
#pragma unroll
      for (int k = 0; k < kHalf; ++k) {
        const int e = k * 32 + lane, r = quarter * 32 + e / kHalf, c = half * kHalf + e % kHalf;
        *reinterpret_cast<uint4*>(sQ + t * kQBytes + (c >> 3) * (BM * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = val[k];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bar_ql[t]));
    }
    const int n_t = t ? nkv1 : nkv0;
    if (n_t > 0) {
      // Rows past the unit's last query see no key: what Q holds there (the
      // next request's queries) must not choose this unit's path.
      const int my_row = min(row, rows_t - 1);
      const int pos = row < rows_t ? sg.first_pos + (td.q_off + query(t, row)) * sg.stride : -1;
      if (half == 0) {
        const int q = td.q_off + query(t, my_row);
        int to;
        if (!p.all) {
          to = sg.local_start + q - p.row_sub;
        } else if (p.zigzag) {  // block b of 2 C, the first n mod 2 C one longer; rank b or 2 C - 1 - b
          const int blocks = 2 * p.C, base = sg.count / blocks, rem = sg.count - base * blocks;
          const int big = rem * (base + 1);
          const int b = q < big ? q / (base + 1) : rem + (q - big) / base;
          const int r = b < p.C ? b : blocks - 1 - b;
          const cp_seg_desc* s =
              reinterpret_cast<const cp_seg_desc*>(p.plan + p.off_seg) + (r * p.R + td.seg) * 2 + (b >= p.C);
          to = s->local_start + q - s->q_start;
        } else {  // flattened token f: rank f mod C, its f / C-th row
          const int f = sg.first_f + q;
          to = p.plan[p.off_rank + f % p.C] + f / p.C;
        }
        s_row[t][i] = valid ? to : -1;  // read after the pair's first named barrier
      }
      const float sl2 = p.scale_log2;
      const float thr = kRescaleLog2 / sl2;
      float m_used = -INFINITY, l = 0.f;
      bool ok = true;
      auto load_s = [&](int j, uint32_t (&sr)[64]) {
        const int kbase = j * BN + 64 * half;
        tmem_ld32(lane_addr + colS, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(lane_addr + colS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_ld_wait();
        if (kbase + 63 > pos) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            if (kbase + e > pos) sr[e] = __float_as_uint(-INFINITY);
        }
      };
      auto exps = [&](const uint32_t (&sr)[64], uint32_t (&pk)[32]) -> float {
        const float neg = -m_used * sl2;
        float s0sum = 0.f, s1sum = 0.f;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float s0 = __uint_as_float(sr[2 * e]), s1 = __uint_as_float(sr[2 * e + 1]);
          float u0, u1;
          fma2(u0, u1, s0, s1, sl2, sl2, neg, neg);
          const float p0 = ex2(u0), p1 = ex2(u1);
          add2(s0sum, s1sum, s0sum, s1sum, p0, p1);
          pk[e] = pack_bf16x2(p0, p1);
        }
        return s0sum + s1sum;
      };
      for (int j = 0; j < n_t && ok; ++j) {
        const bool got = wait_all(&bar_s[t], j & 1);
        if (got && releaser && lane == 0) mbar_arrive(smem_u32(&bar_rel[j % KS]));
        tc_fence_after();
        uint32_t sr[64], pk[32];
        float part = 0.f;
        bool slow = j == 0;
        if (j > 0) {
          // P with the running max as it stands; a half whose sum passes
          // 64 x 2^8 may hold a P above 2^8 and sends the row down the exact
          // path (NaN too).  The result is exact for any max in use.
          load_s(j, sr);
          part = exps(sr, pk);
          slow = bar_red_or(pbar, 64, !got || !(part <= kSpecSum));
        }
        if (slow) {
          if (bar_red_or(pbar, 64, !got)) {
            if (!got) report_timeout(p.status, 1, &abort_flag);
            ok = false;
            break;
          }
          load_s(j, sr);
          float mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            mx = fmax3(mx, __uint_as_float(sr[2 * e]), __uint_as_float(sr[2 * e + 1]));
          const float mrow = fmaxf(mx, exchange(mx));
          if (j == 0) {
            m_used = pos < 0 ? 0.f : mrow;
          } else {
            const bool need = mrow > m_used + thr;
            const float alpha = need ? ex2((m_used - mrow) * sl2) : 1.f;
            if (need) {
              l *= alpha;
              m_used = mrow;
            }
            const bool landed = wait_all(&bar_o[t][(j - 1) & 1], ((j - 1) >> 1) & 1);
            if (bar_red_or(pbar, 64, !landed)) {
              if (!landed) report_timeout(p.status, 2, &abort_flag);
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kDv / 32; ++c) {
              uint32_t r[16];
              tmem_ld16(lane_addr + colO + c * 16, r);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
              tmem_st16(lane_addr + colO + c * 16, r);
            }
          }
          part = exps(sr, pk);
        }
        l += part;
        tmem_st32(lane_addr + colS, pk);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&bar_p[t]);
      }
      const bool landed = ok && wait_all(&bar_o[t][(n_t - 1) & 1], ((n_t - 1) >> 1) & 1);
      if (!bar_red_or(pbar, 64, !landed)) {
        tc_fence_after();
        const float lt = l + exchange(l);
        const float inv = 1.f / lt;
        // O through this tile's Q (no product reads it any more), each warp in
        // 4 KB of its own, so that eight lanes write a row's 128 bytes together
        uint8_t* stage = sQ + t * kQBytes + (half * 4 + quarter) * 4096;
#pragma unroll
        for (int c = 0; c < kDv / 64; ++c) {
          uint32_t r[32];
          tmem_ld32(lane_addr + colO + c * 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(r[8 * v4 + 0]) * inv, __uint_as_float(r[8 * v4 + 1]) * inv);
            w.y = pack_bf16x2(__uint_as_float(r[8 * v4 + 2]) * inv, __uint_as_float(r[8 * v4 + 3]) * inv);
            w.z = pack_bf16x2(__uint_as_float(r[8 * v4 + 4]) * inv, __uint_as_float(r[8 * v4 + 5]) * inv);
            w.w = pack_bf16x2(__uint_as_float(r[8 * v4 + 6]) * inv, __uint_as_float(r[8 * v4 + 7]) * inv);
            *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c + v4) ^ (lane & 7)) << 4)) = w;
          }
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = 4 * k + (lane >> 3), c = lane & 7;
          const long long to = s_row[t][quarter * 32 + r];
          if (to >= 0)
            reinterpret_cast<uint4*>(p.o + (to * p.H + h) * kDv + (kDv / 2) * half)[c] =
                *reinterpret_cast<const uint4*>(stage + r * 128 + ((c ^ (r & 7)) << 4));
        }
        const long long to = s_row[t][i];
        if (to >= 0 && half == 0) p.lse[to * p.H + h] = m_used * p.sm_scale + logf(lt);
      } else if (ok) {
        report_timeout(p.status, 3, &abort_flag);
      }
    }
  } else if (warp == kWarpTma) {
    // ------------------------------------------------------------ TMA producer
    int last_k = -1, last_v = -1;
    bool ok = true;
    auto load_v = [&](int j) {
      if (elect_one()) {
        const uint32_t full = smem_u32(&bar_v[j % KS]);
        mbar_expect_tx(full, C::kVBytes);
#pragma unroll
        for (int c = 0; c < C::kDims / 64; ++c)
          tma_load_3d(smem_u32(PAIR ? sV + (j % KS) * C::kVBytes : piece(5 * j + 3 + c)), &vmap,
                      kNope + cta * C::kDims + c * 64, h, sg.kv_base + j * BN, full);
      }
      __syncwarp();
      last_v = j;
    };
    auto load_k = [&](int j, int c0, int c1) {  // its 64-dim pieces c0 .. c1 - 1 (from 0 first)
      if (elect_one()) {
        const uint32_t full = smem_u32(&bar_k[j % KS]);
        if (c0 == 0) mbar_expect_tx(full, C::kKBytes);
        for (int c = c0; c < c1; ++c) {
          const uint32_t dst = smem_u32(PAIR ? sK + (j % KS) * C::kKBytes + c * C::kKeys * 128 : piece(5 * j + c));
          const int row = sg.kv_base + j * BN + cta * C::kKeys;
          if (c < 2) tma_load_3d(dst, &kmap, c * 64, h, row, full);
          else tma_load_2d(dst, &ropemap, 0, row, full);
        }
      }
      __syncwarp();
      last_k = j;
    };
    auto load_q = [&](int t) {
      if (!split && elect_one()) {
        // rows past the unit's last query are other requests' (or zeros); their
        // results are not written
        const uint32_t full = smem_u32(&bar_ql[t]);
        mbar_expect_tx(full, kQBytes);
        for (int c = 0; c < 3; ++c)
          tma_load_3d(smem_u32(sQ + t * kQBytes + c * BM * 128), &qmap, c * 64, h,
                      sg.first_f + td.q_off + t * MT + cta * BM, full);
      }
      __syncwarp();
    };
    load_q(0);
    if (nK > 0) load_k(0, 0, 3);
    if (rows1 > 0) load_q(1);  // the first tile's scores need not wait for it
    for (int j = 0; j < nK && ok; ++j) {  // V_j and K_(j+1)
      if constexpr (PAIR) {
        if (j >= KS - 1) ok = wait_all(&bar_rel[(j + 1) % KS], ((j + 1) / KS - 1) & 1);
        if (!ok) break;
        load_v(j);
        if (j + 1 < nK) load_k(j + 1, 0, 3);
      } else {
        if (j > 0) ok = wait_all(&bar_rel[(j - 1) & 1], ((j - 1) >> 1) & 1);
        if (!ok) break;
        load_v(j);
        if (j + 1 < nK) {
          load_k(j + 1, 0, 1);
          if (j > 0) ok = wait_all(&bar_o[last_t][(j - 1) & 1], ((j - 1) >> 1) & 1);
          if (!ok) {  // give the barrier what it waits for: nobody uses the pieces any more
            load_k(j + 1, 1, 3);
            break;
          }
          load_k(j + 1, 1, 3);
        }
      }
    }
    if (!ok && lane == 0) report_timeout(p.status, 4, &abort_flag);
    // Never leave with a copy in flight.
    if (!split)
      for (int t = 0; t < (rows1 > 0 ? 2 : 1); ++t) mbar_wait(smem_u32(&bar_ql[t]), 0, 1000000000ull, &zero_flag);
    for (int k = max(0, last_k - KS + 1); k <= last_k; ++k)
      mbar_wait(smem_u32(&bar_k[k % KS]), (k / KS) & 1, 1000000000ull, &zero_flag);
    for (int k = max(0, last_v - KS + 1); k <= last_v; ++k)
      mbar_wait(smem_u32(&bar_v[k % KS]), (k / KS) & 1, 1000000000ull, &zero_flag);
    __syncwarp();
  } else if (warp == kWarpRelay) {
    // ------------------------------------------------------------ relay
    bool ok = true;
    if constexpr (PAIR) {
      ok = wait_all(&bar_ql[0], 0);
      if (ok) warp_arrive(&bar_q[0]);
      if (ok && nK > 0) {
        ok = wait_all(&bar_k[0], 0);
        if (ok) warp_arrive(&bar_k0);
      }
      if (ok && rows1 > 0) {
        ok = wait_all(&bar_ql[1], 0);
        if (ok) warp_arrive(&bar_q[1]);
      }
    }
    for (int j = 0; j < nK && ok; ++j) {
      ok = wait_all(&bar_v[j % KS], (j / KS) & 1);
      if (PAIR && ok && j + 1 < nK) ok = wait_all(&bar_k[(j + 1) % KS], ((j + 1) / KS) & 1);
      if (ok && j == nK - 1) {  // rows past the last key, four rows' 128 bytes at a time
        for (int r = n_keys - j * BN + (lane >> 3); r < BN; r += 4)
#pragma unroll
          for (int c = 0; c < C::kDims / 64; ++c) {
            uint8_t* v = PAIR ? sV + (j % KS) * C::kVBytes : piece(5 * j + 3 + c);
            *reinterpret_cast<uint4*>(v + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        fence_proxy_async_smem();
      }
      // Phase j of a tile's P barrier has begun once S_j, issued after phase
      // j - 1 was waited for, is complete; phase j + 1 of bar_s needs this
      // arrival, so none is missed.
      for (int t = 0; t < 2 && ok; ++t) {
        if (j >= (t ? nkv1 : nkv0)) continue;
        ok = wait_all(&bar_s[t], j & 1);
        if (ok) warp_arrive(&bar_p[t]);
      }
    }
    if (!ok && lane == 0) report_timeout(p.status, 5, &abort_flag);
  } else if (cta == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idS = idesc_bf16_f32(MT, BN, 0, 0);
    constexpr uint32_t idPV = idesc_bf16_f32(MT, kDv, 0, 1);
    const uint64_t dQ0 = smem_desc(smem_u32(sQ), 16, 1024);
    const uint64_t dK0 = smem_desc(smem_u32(sK), 16, 1024);
    const uint64_t dV0 = smem_desc(smem_u32(PAIR ? sV : sK), BN * 128, 1024);
    auto commit = [&](uint64_t* bar) {
      if constexpr (PAIR) mma_commit_pair(smem_u32(bar));
      else mma_commit(smem_u32(bar));
    };
    auto issue_s = [&](int t, int j) {
      const uint64_t a0 = dQ0 + (uint64_t)((t * kQBytes) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const uint64_t b0 = dK0 + (uint64_t)((PAIR ? (j % KS) * C::kKBytes + c * C::kKeys * 128
                                                     : ((5 * j + c) & 7) * kPiece) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint64_t a = a0 + ((c * (BM * 128) + kk * 32) >> 4), b = b0 + ((kk * 32) >> 4);
            if constexpr (PAIR) mma_ss_pair(tmem + t * 256, a, b, idS, c + kk > 0);
            else mma_ss(tmem + t * 256, a, b, idS, c + kk > 0);
          }
        }
        commit(&bar_s[t]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int t, int j) {
      const uint32_t pa = tmem + t * 256, d = tmem + t * 256 + 128;
      const int g = (5 * j + 3) & 7;  // one CTA: V's first piece
      const uint64_t v0 = dV0 + (uint64_t)((PAIR ? (j % KS) * C::kVBytes : g * kPiece) >> 4);
      if (elect_one()) {
        if (!PAIR && g == 7) {
          // the second piece is the ring's first: each 64 dims a product of their own
          constexpr uint32_t idHalf = idesc_bf16_f32(MT, kDv / 2, 0, 1);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
              mma_ts(d + c * 64, pa + (kk >> 2) * 64 + (kk & 3) * 8,
                     (c ? dV0 : v0) + (uint64_t)((kk * 16 * 128) >> 4), idHalf, (j > 0 || kk > 0) ? 1u : 0u);
        } else {
#pragma unroll
          for (int kk = 0; kk < BN / 16; ++kk) {
            const uint32_t a = pa + (kk >> 2) * 64 + (kk & 3) * 8;
            const uint64_t b = v0 + (uint64_t)((kk * 16 * 128) >> 4);
            if constexpr (PAIR) mma_ts_pair(d, a, b, idPV, (j > 0 || kk > 0) ? 1u : 0u);
            else mma_ts(d, a, b, idPV, (j > 0 || kk > 0) ? 1u : 0u);
          }
        }
        commit(&bar_o[t][j & 1]);
      }
      __syncwarp();
    };
    unsigned bad = 0;
    if (p.stall_test && !wait_all(&bar_drain, 0)) bad = 10;
    if (nK > 0 && !bad && !wait_all(PAIR ? &bar_k0 : &bar_k[0], 0)) bad = 12;
    for (int t = 0; t < 2 && !bad; ++t) {
      if ((t ? nkv1 : nkv0) == 0) continue;
      if (!wait_all(PAIR ? &bar_q[t] : &bar_ql[t], 0)) {
        bad = 11;
        break;
      }
      tc_fence_after();
      issue_s(t, 0);
    }
    for (int j = 0; j < nK && !bad; ++j) {
      bool k_in = PAIR;  // K_(j+1) is in place: a pair's P barrier says so
      for (int t = 0; t < 2 && !bad; ++t) {
        const int nt = t ? nkv1 : nkv0;
        if (j >= nt) continue;
        if (!wait_all(&bar_p[t], j & 1)) {  // P_j is written, V_j is in place
          bad = 14 + t;
          break;
        }
        tc_fence_after();
        issue_pv(t, j);
        if (j + 1 >= nt) continue;
        if (!k_in) {  // while P V runs
          k_in = wait_all(&bar_k[(j + 1) % KS], ((j + 1) / KS) & 1);
          if (!k_in) {
            bad = 17;
            break;
          }
          tc_fence_after();
        }
        issue_s(t, j + 1);
      }
    }
    if (bad && lane == 0) report_timeout(p.status, bad, &abort_flag);
    // Never free TMEM under a running MMA: wait for everything issued.
    if (elect_one()) commit(&bar_drain);
    __syncwarp();
    mbar_wait(smem_u32(&bar_drain), 0, 1000000000ull, &zero_flag);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // neither CTA leaves while products read its memory
  tc_fence_after();
  if (warp == kWarpMma) {
    if constexpr (PAIR) tmem_dealloc_pair(tmem, 512);
    else tmem_dealloc(tmem, 512);
  }
}

// Rows of the head's keys or values as 3-d (256 dims, heads, rows).
bool kv_map(CUtensorMap* m, const void* kv, int H, int rows, int box_rows) {
  const uint64_t dims[3] = {kNope + kDv, (uint64_t)H, (uint64_t)rows};
  const uint64_t strides[2] = {(kNope + kDv) * 2, (uint64_t)H * (kNope + kDv) * 2};
  const uint32_t box[3] = {64, 1, (uint32_t)box_rows};
  return encode_tensor_map_bf16(m, kv, 3, dims, strides, box);
}

template <bool PAIR>
cudaError_t launch(const Params& p, const void* kv, const void* k_rope, long long rope_stride, int n_q, int rows,
                   cudaStream_t s) {
  using C = Cfg<PAIR>;
  CUtensorMap qm, km, vm, rm;
  const uint64_t qdims[3] = {kDqk, (uint64_t)p.H, (uint64_t)n_q};
  const uint64_t qstrides[2] = {kDqk * 2, (uint64_t)p.H * kDqk * 2};
  const uint32_t qbox[3] = {64, 1, BM};
  const uint64_t dims[2] = {kRope, (uint64_t)rows};
  const uint64_t strides[1] = {(uint64_t)rope_stride * 2};
  const uint32_t box[2] = {64, C::kKeys};
  if (!encode_tensor_map_bf16(&qm, p.q, 3, qdims, qstrides, qbox) || !kv_map(&km, kv, p.H, rows, C::kKeys) ||
      !kv_map(&vm, kv, p.H, rows, BN) ||
      !encode_tensor_map_bf16(&rm, k_rope, 2, dims, strides, box, false))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(mla_prefill_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const long long blocks = (long long)p.n_tiles * p.H * C::kCtas;
  if (blocks > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  return launch_early(mla_prefill_kernel<PAIR>, (unsigned)blocks, kThreads, C::kSmem, s, C::kCtas, qm, km, vm, rm, p);
}

}  // namespace

cudaError_t launch_mla_prefill(const int32_t* dev_plan, const int32_t* host_plan, const cp_plan_header& h,
                               int rank, const void* q, const void* kv, const void* k_rope,
                               long long rope_stride, int H, float sm_scale, void* o, float* lse,
                               bool stall_test, cudaStream_t s) {
  Params p;
  p.plan = dev_plan;
  p.off_seg = h.off_seg;
  p.off_rank = h.off_rank;
  p.C = h.C;
  p.R = h.R;
  p.zigzag = h.kind == 0;
  p.all = rank < 0;
  p.split = rank >= 0 && h.kind == 1 && h.C > 1;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.H = H;
  p.sm_scale = sm_scale;
  p.scale_log2 = sm_scale * kLog2e;
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInvalidDevice;
  p.wait_ns = stall_test ? 50000000ull : wait_limit_ns();
  p.stall_test = stall_test;
  const long long head_bytes = (long long)h.KV * (kNope + kDv) * 2;
  const int most = (int)std::min<long long>(H, std::max<long long>(1, kGroupBytes / head_bytes));
  const int groups = (H + most - 1) / most;
  p.head_group = (H + groups - 1) / groups;
  // A pair where requests (one rank: segments) fill three quarters of its 512
  // rows or more.  Both forms take about as long for a tile step (3,000 clk for
  // a pair's 512 rows, 3,440 for one CTA's 256), so a pair whose second M tile
  // is empty wastes an SM.  16,384 tokens behind 4,096, 32 heads: pairs
  // 2,380 us, single CTAs 2,540; nine ragged requests of 1 to 2,500 tokens (48
  // quarters filled of 68), 16 heads: 96 and 77.
  const cp_seg_desc* seg = reinterpret_cast<const cp_seg_desc*>(host_plan + h.off_seg);
  const cp_req_desc* req = reinterpret_cast<const cp_req_desc*>(host_plan + h.off_req);
  long long n128 = 0, n512 = 0;
  for (int i = 0; i < (rank < 0 ? h.R : h.n_seg); ++i) {
    const int count = rank < 0 ? req[i].new_len : seg[i].rank == rank ? seg[i].count : 0;
    n128 += (count + 127) / 128;
    n512 += (count + 511) / 512;
  }
  const bool pair = n128 >= 3 * n512;
  if (rank < 0) {
    p.tile_list = h.off_run + (pair ? kReqTileWords * h.n_parts : 0);
    p.n_tiles = pair ? (int)n512 : h.n_parts;
    p.row_sub = 0;
  } else {
    const int32_t* rto = host_plan + h.off_rtile;
    p.tile_list = h.off_rtile + h.C + 1 + 2 * rto[rank];
    p.n_tiles = rto[rank + 1] - rto[rank];
    p.row_sub = host_plan[h.off_rank + rank];
  }
  if (p.n_tiles == 0) return cudaSuccess;
  return pair ? launch<true>(p, kv, k_rope, rope_stride, h.T, h.KV, s)
              : launch<false>(p, kv, k_rope, rope_stride, h.T, h.KV, s);
}

}  // namespace cpattn

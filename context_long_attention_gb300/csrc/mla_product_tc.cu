// Per-head products of multi-head latent attention on the tcgen05 tensor
// cores (bf16 in, fp32 accumulate, one rounding to bf16).
//
// With the up-projection W [H, 256, 512] (per head: 128 rows of the key part,
// then 128 rows of the value):
//   expand   kv[t, h, :]        = W[h] latent[t]                 N = 256, K = 512
//   absorb   ql[n, h, 0:512]    = W[h, 0:128]^T q[n, h, 0:128]   N = 512, K = 128
//            ql[n, h, 512:576]  = q[n, h, 128:192] (the rotated part, copied)
//   project  o[n, h, :]         = W[h, 128:256] ol[n, h, :]      N = 128, K = 512
//
// One work item = 128 tokens (the products' M) x one head x NB of its output
// columns (N); rows of a tile past the last token read as zeros and are never
// written.  Persistent CTAs take items in turn:
//   warp 0     TMA producer: stages of 64 of K, the tokens' [128 x 64] and the
//              weight's NB x 64 (absorb reads it as an MN-major operand, so
//              one layout of W serves all three; after a head's first columns
//              it also loads the query's rotated part as a stage)
//   warp 1     MMA issuer and TMEM owner, two accumulators of NB columns
//   warp 2     absorb: the rotated part's TMA store, straight from its stage
//   warps 4-11 epilogue, two groups of four warps with every other item: a
//              thread per token row, 64 columns at a time through shared
//              memory to a TMA store (rows written straight from the registers,
//              16 bytes a lane and row, took absorb over 512 tokens x 64 heads
//              twice as long)
// Tiles of 256 tokens (a third less weight read from the L2) were no faster:
// a pass of project over 1,000 tokens x 64 heads took 18.6 us either way, one
// over 300 tokens x 16 heads 8.4 instead of 6.6.
//
// A prompt's expansion runs on CTA pairs (expand_pair_kernel, below).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdlib.h>

#include "early_launch.cuh"
#include "internal.h"
#include "tc_pair.cuh"

namespace cpattn {
namespace {
using namespace tc;

constexpr int BM = 128;  // tokens per item
constexpr int kLatent = 512;
constexpr int kHeadRows = 256;  // W rows per head
constexpr int kKeyDims = 128;   // W rows of the key part; the value part follows
constexpr int kRope = 64;
constexpr int kThreads = 384;

constexpr int kOutBytes = BM * 128;  // an output piece: 128 tokens x 64 columns

enum Mode { kExpand = 0, kAbsorb = 1, kProject = 2 };

template <int MODE, int NB>
struct Cfg {
  static constexpr int kN = MODE == kExpand ? kHeadRows : MODE == kAbsorb ? kLatent : kKeyDims;  // columns per head
  static constexpr int kK = MODE == kAbsorb ? kKeyDims : kLatent;
  static constexpr int kNBlocks = kN / NB;
  static constexpr int kIters = kK / 64;
  static constexpr int kABytes = BM * 128;
  static constexpr int kBBytes = NB * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // staging pieces of an epilogue group: two, so that an item's stores do not
  // wait for each other, except where the call is bound by its writes (absorb
  // over 512 tokens x 64 heads 10.7 us with one, 11.2 with two)
  static constexpr int kBufs = MODE == kAbsorb ? 1 : NB / 64;
  static constexpr int kStages = (229376 - 2 * kBufs * kOutBytes) / kStageBytes;
  static constexpr int kSmem = kStages * kStageBytes + 2 * kBufs * kOutBytes + 1024;
  static constexpr int kTmemCols = 2 * NB;
};

struct Params {
  int H;
  int n_items;  // token tiles x heads x column blocks
  int n_tokens;
  unsigned* status;
  unsigned long long wait_ns;
  int stall_test;  // test hook: the issuer waits on a barrier that nobody arrives at yet
};

__device__ void report_timeout(unsigned* status, unsigned site, volatile int* abort) {
  *abort = 1;
  if (atomicCAS(status, 0u, 1u) == 0u) {
    status[1] = kKernMlaProduct;
    status[2] = site;
    status[3] = blockIdx.x;
    __threadfence();
  }
}

// NB columns of an accumulator to the output by four epilogue warps: 64
// columns at a time, bf16, through the group's BUFS staging pieces to TMA
// stores at columns col0 on (rows past the last token fall outside the map).
// Named barriers bar, bar + 1 are the group's.
template <int NB, int BUFS>
__device__ __forceinline__ void store_columns(uint32_t acc, uint8_t* stage, int row, const CUtensorMap* map, int col0,
                                              int h, int tok0, int n_tokens, int bar) {
#pragma unroll 1
  for (int c = 0; c < NB / 64; ++c) {
    uint32_t r[2][32];
    tmem_ld32(acc + c * 64, r[0]);
    tmem_ld32(acc + c * 64 + 32, r[1]);
    uint8_t* buf = stage + (c % BUFS) * kOutBytes;
    if (c % BUFS == 0) {  // the stores so far have read the pieces
      if (row == 0) tma_store_wait_read();
      named_bar_sync(bar, 128);
    }
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t* x = r[k >> 2] + 8 * (k & 3);
      uint4 w;
      w.x = pack_bf16x2(__uint_as_float(x[0]), __uint_as_float(x[1]));
      w.y = pack_bf16x2(__uint_as_float(x[2]), __uint_as_float(x[3]));
      w.z = pack_bf16x2(__uint_as_float(x[4]), __uint_as_float(x[5]));
      w.w = pack_bf16x2(__uint_as_float(x[6]), __uint_as_float(x[7]));
      *reinterpret_cast<uint4*>(buf + row * 128 + ((k ^ (row & 7)) << 4)) = w;
    }
    fence_proxy_async_smem();
    named_bar_sync(bar + 1, 128);
    if (row == 0) {
      if (tok0 < n_tokens) tma_store_3d(map, smem_u32(buf), col0 + c * 64, h, tok0);
      tma_store_commit();
    }
  }
}

struct Item {
  int tile, h, nb;
};
template <class C>
__device__ __forceinline__ Item item_of(int i, int H) {
  Item it;
  it.nb = i % C::kNBlocks;
  const int r = i / C::kNBlocks;
  it.h = r % H;
  it.tile = r / H;
  return it;
}
// Whether an item also carries the query's rotated part (64 columns as they are).
template <int MODE>
__device__ __forceinline__ bool rotated(const Item& it) {
  return MODE == kAbsorb && it.nb == 0;
}

template <int MODE, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    mla_product_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap omap, const Params p) {
  using C = Cfg<MODE, NB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t bar_full[C::kStages], bar_empty[C::kStages], bar_acc[2], bar_free[2], bar_drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag, zero_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      // absorb: the issuer and warp 2 each wait for every stage and release it,
      // so that neither misses a phase of a stage that the other one uses
      mbar_init(smem_u32(&bar_empty[s]), MODE == kAbsorb ? 2 : 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&bar_acc[a]), 1);
      mbar_init(smem_u32(&bar_free[a]), 128);
    }
    mbar_init(smem_u32(&bar_drain), 1);
    abort_flag = 0;
    zero_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&amap);
    prefetch_tmap(&wmap);
    prefetch_tmap(&omap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  wait_for_earlier_kernels();
  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.wait_ns, &abort_flag));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    int g = 0;  // stages filled so far
    bool ok = true;
    for (int i = blockIdx.x; i < p.n_items && ok; i += gridDim.x) {
      const Item it = item_of<C>(i, p.H);
      const int stages = C::kIters + rotated<MODE>(it);
      for (int k = 0; k < stages && ok; ++k, ++g) {
        const int s = g % C::kStages;
        if (g >= C::kStages) ok = wait_all(smem_u32(&bar_empty[s]), (g / C::kStages - 1) & 1);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t full = smem_u32(&bar_full[s]);
          const uint32_t a = smem_u32(smem + s * C::kStageBytes), b = a + C::kABytes;
          mbar_expect_tx(full, k < C::kIters ? C::kStageBytes : C::kABytes);
          if (MODE == kExpand) tma_load_2d(a, &amap, k * 64, it.tile * BM, full);
          else tma_load_3d(a, &amap, k * 64, it.h, it.tile * BM, full);
          if (MODE == kAbsorb) {  // [64 key dims x 64 latent columns] pieces
            if (k < C::kIters) {
#pragma unroll
              for (int c = 0; c < NB / 64; ++c)
                tma_load_2d(b + c * 64 * 128, &wmap, it.nb * NB + c * 64, it.h * kHeadRows + k * 64, full);
            }
          } else {  // [NB rows x 64 latent columns]
            const int row = it.h * kHeadRows + (MODE == kProject ? kKeyDims : 0) + it.nb * NB;
            tma_load_2d(b, &wmap, k * 64, row, full);
          }
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) report_timeout(p.status, 1, &abort_flag);
    // Never leave with a copy in flight.
    for (int k = max(0, g - C::kStages); k < g; ++k)
      mbar_wait(smem_u32(&bar_full[k % C::kStages]), (k / C::kStages) & 1, 1000000000ull, &zero_flag);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id = idesc_bf16_f32(BM, NB, 0, MODE == kAbsorb ? 1 : 0);
    int g = 0, n = 0;
    unsigned bad = 0;
    if (p.stall_test && !wait_all(smem_u32(&bar_drain), 0)) bad = 7;
    for (int i = blockIdx.x; i < p.n_items && !bad; i += gridDim.x, ++n) {
      const int acc = n & 1;
      if (n >= 2 && !wait_all(smem_u32(&bar_free[acc]), (n / 2 - 1) & 1)) bad = 2;
      for (int k = 0; k < C::kIters && !bad; ++k, ++g) {
        const int s = g % C::kStages;
        if (!wait_all(smem_u32(&bar_full[s]), (g / C::kStages) & 1)) {
          bad = 3;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(smem + s * C::kStageBytes), b = a + C::kABytes;
        const uint64_t da = smem_desc(a, 16, 1024);
        const uint64_t db = MODE == kAbsorb ? smem_desc(b, 64 * 128, 1024) : smem_desc(b, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const uint32_t oa = (kk * 32) >> 4;
            const uint32_t ob = MODE == kAbsorb ? (kk * 16 * 128) >> 4 : (kk * 32) >> 4;
            mma_ss(tmem + acc * NB, da + oa, db + ob, id, (k > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(smem_u32(&bar_empty[s]));
          if (k == C::kIters - 1) mma_commit(smem_u32(&bar_acc[acc]));
        }
        __syncwarp();
      }
      if (!bad && rotated<MODE>(item_of<C>(i, p.H))) {  // warp 2's stage
        const int s = g % C::kStages;
        if (!wait_all(smem_u32(&bar_full[s]), (g / C::kStages) & 1)) bad = 6;
        else if (lane == 0) mbar_arrive(smem_u32(&bar_empty[s]));
        __syncwarp();
        ++g;
      }
    }
    if (bad && lane == 0) report_timeout(p.status, bad, &abort_flag);
    if (elect_one()) mma_commit(smem_u32(&bar_drain));
    __syncwarp();
    mbar_wait(smem_u32(&bar_drain), 0, 1000000000ull, &zero_flag);
  } else if (MODE == kAbsorb && warp == 2) {
    // ------------------------------------------------------------ rotated part
    int g = 0;
    bool ok = true;
    for (int i = blockIdx.x; i < p.n_items && ok; i += gridDim.x) {
      const Item it = item_of<C>(i, p.H);
      const int stages = C::kIters + rotated<MODE>(it);
      for (int k = 0; k < stages && ok; ++k, ++g) {
        const int s = g % C::kStages;
        ok = wait_all(smem_u32(&bar_full[s]), (g / C::kStages) & 1);
        if (ok && lane == 0) {
          if (k == C::kIters) {
            tma_store_3d(&omap, smem_u32(smem + s * C::kStageBytes), kLatent, it.h, it.tile * BM);
            tma_store_commit();
            tma_store_wait_read();
          }
          mbar_arrive(smem_u32(&bar_empty[s]));
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) report_timeout(p.status, 5, &abort_flag);
    if (lane == 0) tma_store_wait_read();
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3, group = (warp >> 2) - 1;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    uint8_t* stage = smem + C::kStages * C::kStageBytes + group * C::kBufs * kOutBytes;
    int n = 0;
    for (int i = blockIdx.x; i < p.n_items; i += gridDim.x, ++n) {
      const int acc = n & 1;
      if (acc != group) continue;
      const Item it = item_of<C>(i, p.H);
      // the four warps leave together: one that gave up meets the others here
      const bool got = wait_all(smem_u32(&bar_acc[acc]), (n / 2) & 1);
      if (bar_red_or(3 + 4 * group, 128, !got)) {
        if (!got && lane == 0) report_timeout(p.status, 4, &abort_flag);
        break;
      }
      tc_fence_after();
      store_columns<NB, C::kBufs>(lane_addr + acc * NB, stage, row, &omap, it.nb * NB, it.h, it.tile * BM,
                           p.n_tokens, 1 + 4 * group);
      tc_fence_before();
      mbar_arrive(smem_u32(&bar_free[acc]));
    }
    if (row == 0) tma_store_wait_read();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// ---------------------------------------------------------------- expansion of a prompt
//
// A pair of CTAs holds 256 tokens' latent rows in shared memory (128 x 512
// each) and takes heads one after another: M = 256 tokens, N = 256 columns of
// the head, K = 512 streamed as eight [256 x 64] pieces of W, half of each in
// either CTA.  So a CTA reads 16 KB of W for 512 clk of products (32 B/clk
// through its L2 port; a single CTA's 128 x 256 tile reads 96).  Pairs take
// contiguous runs of (token tile, head) items; a new tile's rows are loaded
// piece by piece as the last head's products release the old ones.  20,480
// tokens x 32 heads in a replayed graph: 103 to 105 us = 1,650 TFLOP/s (the
// library's product of this shape: 99.5; single CTAs with tiles of 128 x 256: 117
// to 162); bound by power (0.98 of the sustained bf16 rate) and the first rows'
// read.  A call among others takes 116 to 120.
constexpr int kPieces = kLatent / 64;
constexpr int kPieceBytes = BM * 128;  // 128 rows x 64 columns, of tokens or of W
constexpr int kPairThreads = 256;  // four epilogue warps: 2,800 clk an item of 4,096 clk of products
constexpr int kWStages = 5;
constexpr int kExpandSmem = (kPieces + kWStages) * kPieceBytes + kOutBytes + 1024;

__global__ void __launch_bounds__(kPairThreads, 1)
    expand_pair_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                       const __grid_constant__ CUtensorMap omap, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sW = smem + kPieces * kPieceBytes;
  // bar_a[k], bar_w[s]: piece k of the tokens, the W piece in stage s landed in
  // both CTAs (both halves' bytes count in the even CTA, which issues the
  // products).  bar_afree, bar_wfree: read by the products (in both CTAs).
  __shared__ __align__(8) uint64_t bar_a[kPieces], bar_afree[kPieces], bar_w[kWStages], bar_wfree[kWStages];
  __shared__ __align__(8) uint64_t bar_acc[2], bar_free[2], bar_drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag, zero_flag;
  __shared__ int issued[2];  // pieces of W and of the tokens that this CTA's producer has asked for
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = (int)cluster_ctarank();
  const int pairs = gridDim.x >> 1, pair = blockIdx.x >> 1;
  const int first = (int)((long long)p.n_items * pair / pairs), last = (int)((long long)p.n_items * (pair + 1) / pairs);

  if (threadIdx.x == 0) {
    for (int k = 0; k < kPieces; ++k) {
      mbar_init(smem_u32(&bar_a[k]), 1);
      mbar_init(smem_u32(&bar_afree[k]), 1);
    }
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(smem_u32(&bar_w[s]), 1);
      mbar_init(smem_u32(&bar_wfree[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&bar_acc[a]), 1);
      mbar_init(smem_u32(&bar_free[a]), 2 * 4);  // the epilogue warps of both CTAs
    }
    mbar_init(smem_u32(&bar_drain), 1);
    abort_flag = 0;
    zero_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&tmem_slot), 512);
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&amap);
    prefetch_tmap(&wmap);
    prefetch_tmap(&omap);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  wait_for_earlier_kernels();
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.wait_ns, &abort_flag)) != 0;
  };
  auto give_up = [&](unsigned site) {  // both CTAs stop, and both know it when they meet
    report_timeout(p.status, site, &abort_flag);
    st_cluster(map_to_rank(smem_u32(const_cast<int*>(&abort_flag)), cta ^ 1), 1);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    int g = 0, pieces = 0, tiles = 0, tile = -1;
    bool ok = true;
    for (int i = first; i < last && ok; ++i) {
      const int h = i % p.H;
      const bool fresh = i / p.H != tile;
      tile = i / p.H;
      for (int k = 0; k < kPieces && ok; ++k, ++g) {
        if (fresh) {
          if (tiles > 0) ok = wait_all(&bar_afree[k], (tiles - 1) & 1);
          if (!ok) break;
          if (elect_one()) {
            if (cta == 0) mbar_expect_tx(smem_u32(&bar_a[k]), 2 * kPieceBytes);
            tma_load_2d_pair(smem_u32(sA + k * kPieceBytes), &amap, k * 64, tile * 2 * BM + cta * BM,
                             map_to_rank(smem_u32(&bar_a[k]), 0));
          }
          __syncwarp();
          ++pieces;
        }
        const int s = g % kWStages;
        if (g >= kWStages) ok = wait_all(&bar_wfree[s], (g / kWStages - 1) & 1);
        if (!ok) break;
        if (elect_one()) {
          if (cta == 0) mbar_expect_tx(smem_u32(&bar_w[s]), 2 * kPieceBytes);
          tma_load_2d_pair(smem_u32(sW + s * kPieceBytes), &wmap, k * 64, h * kHeadRows + cta * 128,
                           map_to_rank(smem_u32(&bar_w[s]), 0));
        }
        __syncwarp();
      }
      if (fresh) ++tiles;
    }
    if (!ok && lane == 0) give_up(11);
    if (lane == 0) {
      issued[0] = g;
      issued[1] = pieces;
    }
    __syncwarp();
  } else if (warp == 1 && cta == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id = idesc_bf16_f32(2 * BM, kHeadRows, 0, 0);
    const uint64_t dA = smem_desc(smem_u32(sA), 16, 1024), dW = smem_desc(smem_u32(sW), 16, 1024);
    unsigned bad = 0;
    int s = 0, tiles = 0, head = first % p.H;
    uint32_t phase = 0;  // of the W stages
    bool fresh = true;
    if (p.stall_test && !wait_all(&bar_drain, 0)) bad = 16;
    for (int n = 0; n < last - first && !bad; ++n) {
      const int acc = n & 1;
      const bool leave = head + 1 == p.H;  // this tile's last head
      const uint32_t d = tmem + acc * kHeadRows;
      if (n >= 2 && !wait_all(&bar_free[acc], (n / 2 - 1) & 1)) bad = 12;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        if (fresh && !bad && !wait_all(&bar_a[k], tiles & 1)) bad = 13;
        if (!bad && !wait_all(&bar_w[s], phase)) bad = 14;
        if (bad) break;
        tc_fence_after();
        const uint64_t a = dA + (uint64_t)((k * kPieceBytes) >> 4), b = dW + (uint64_t)((s * kPieceBytes) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_pair(d, a + ((kk * 32) >> 4), b + ((kk * 32) >> 4), id, (k > 0 || kk > 0) ? 1u : 0u);
          mma_commit_pair(smem_u32(&bar_wfree[s]));
          if (leave) mma_commit_pair(smem_u32(&bar_afree[k]));
          if (k == kPieces - 1) mma_commit_pair(smem_u32(&bar_acc[acc]));
        }
        __syncwarp();
        if (++s == kWStages) {
          s = 0;
          phase ^= 1;
        }
      }
      tiles += fresh;
      fresh = leave;
      head = leave ? 0 : head + 1;
    }
    if (bad && lane == 0) give_up(bad);
    if (elect_one()) mma_commit_pair(smem_u32(&bar_drain));
    __syncwarp();
    mbar_wait(smem_u32(&bar_drain), 0, 1000000000ull, &zero_flag);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    uint8_t* stage = sW + kWStages * kPieceBytes;
    int n = 0;
    for (int i = first; i < last; ++i, ++n) {
      const int acc = n & 1, tile = i / p.H;
      const bool got = wait_all(&bar_acc[acc], (n / 2) & 1);
      if (bar_red_or(3, 128, !got)) {
        if (!got && lane == 0) give_up(15);
        break;
      }
      tc_fence_after();
      store_columns<kHeadRows, 1>(lane_addr + acc * kHeadRows, stage, row, &omap, 0, i - tile * p.H,
                               tile * 2 * BM + cta * BM, p.n_tokens, 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(&bar_free[acc]), 0));
    }
    if (row == 0) tma_store_wait_read();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while products read its memory
  tc_fence_after();
  // Nor with a copy in flight: products waited for every piece, unless a wait ran
  // out in either CTA.  Then both stay until the last pieces that either asked for
  // have landed (the barriers of the even CTA count both halves; where only one
  // half was asked for, until it has had far more time than a copy takes).
  if (__any_sync(0xffffffffu, abort_flag)) {
    if (cta == 0 && warp == 0) {
      const uint32_t other = map_to_rank(smem_u32(issued), 1);
      const int w = max(issued[0], (int)ld_cluster(other)), a = max(issued[1], (int)ld_cluster(other + 4));
      for (int k = max(0, w - kWStages); k < w; ++k)
        mbar_wait(smem_u32(&bar_w[k % kWStages]), (k / kWStages) & 1, 10000000ull, &zero_flag);
      for (int k = max(0, a - kPieces); k < a; ++k)
        mbar_wait(smem_u32(&bar_a[k % kPieces]), (k / kPieces) & 1, 10000000ull, &zero_flag);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

cudaError_t launch_expand_pair(const CUtensorMap& am, const CUtensorMap& wm, const CUtensorMap& om, Params p, int sms,
                               cudaStream_t s) {
  const long long items = (long long)((p.n_tokens + 2 * BM - 1) / (2 * BM)) * p.H;
  if (items > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  p.n_items = (int)items;
  cudaError_t e = cudaFuncSetAttribute(expand_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmem);
  if (e != cudaSuccess) return e;
  const int pairs = (int)(items < sms / 2 ? items : sms / 2);
  return launch_early(expand_pair_kernel, 2 * pairs, kPairThreads, kExpandSmem, s, 2, am, wm, om, p);
}

template <int MODE, int NB>
cudaError_t launch(const CUtensorMap& am, const CUtensorMap& wm, const CUtensorMap& om, Params p, int sms,
                   cudaStream_t s) {
  using C = Cfg<MODE, NB>;
  const long long items = (long long)((p.n_tokens + BM - 1) / BM) * p.H * C::kNBlocks;
  if (items > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  p.n_items = (int)items;
  cudaError_t e = cudaFuncSetAttribute(mla_product_kernel<MODE, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = (int)(items < sms ? items : sms);
  return launch_early(mla_product_kernel<MODE, NB>, grid, kThreads, C::kSmem, s, 1, am, wm, om, p);
}

bool weight_map(CUtensorMap* m, const void* w, int H, int box_rows) {
  const uint64_t dims[2] = {kLatent, (uint64_t)H * kHeadRows};
  const uint64_t strides[1] = {kLatent * 2};
  const uint32_t box[2] = {64, (uint32_t)box_rows};
  return encode_tensor_map_bf16(m, w, 2, dims, strides, box);
}
// x [tokens, H, row] as 3-d, boxes of 64 columns of one head's 128 tokens
bool token_map(CUtensorMap* m, const void* x, int n, int H, int row) {
  const uint64_t dims[3] = {(uint64_t)row, (uint64_t)H, (uint64_t)n};
  const uint64_t strides[2] = {(uint64_t)row * 2, (uint64_t)H * row * 2};
  const uint32_t box[3] = {64, 1, BM};
  return encode_tensor_map_bf16(m, x, 3, dims, strides, box);
}

Params params(int n, int H) {
  const char* stall = getenv("CPATTN_TEST_STALL");  // the test hook of cp_prefill_attn
  const bool stall_test = stall && stall[0] == '1';
  return {H, 0, n, device_status_ptr(), stall_test ? 50000000ull : wait_limit_ns(), stall_test};
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

}  // namespace

cudaError_t launch_mla_expand(const void* latent, long long stride, const void* w, int T, int H, void* kv,
                              cudaStream_t s) {
  Params p = params(T, H);
  const int sms = sm_count();
  if (!p.status || !sms) return cudaErrorInvalidDevice;
  CUtensorMap am, wm, om;
  const uint64_t dims[2] = {kLatent, (uint64_t)T};
  const uint64_t strides[1] = {(uint64_t)stride * 2};
  const uint32_t box[2] = {64, BM};
  if (!encode_tensor_map_bf16(&am, latent, 2, dims, strides, box)) return cudaErrorInvalidValue;
  if (!weight_map(&wm, w, H, 128) || !token_map(&om, kv, T, H, kHeadRows)) return cudaErrorInvalidValue;
  // Measured in a replayed graph (us): r rounds of 128 x 128 tiles on single
  // CTAs take 2.7 + 2.4 r (1 round 5.2, 2 7.6, 3 10.0, 4 12.2, 12 31.5, 68 167),
  // r rounds of (256 tokens, head) items on pairs 4.6 + 3 r (1 round 7.6,
  // 2 10.6, 3 13.5, 6 21.7, 34 105).  Twice the single rounds as a rule, fewer
  // where the last 256 tokens are half empty or the last round is.
  const long long singles = ((long long)((T + BM - 1) / BM) * 2 * H + sms - 1) / sms;
  const long long pairs = ((long long)((T + 2 * BM - 1) / (2 * BM)) * H + sms / 2 - 1) / (sms / 2);
  if (10 + 15 * pairs < 12 * singles) return launch_expand_pair(am, wm, om, p, sms, s);
  return launch<kExpand, 128>(am, wm, om, p, sms, s);
}

cudaError_t launch_mla_absorb(const void* q, const void* w, int n, int H, void* ql, cudaStream_t s) {
  if (n <= kMlaSmall) return launch_mla_absorb_small(q, w, n, H, ql, s);
  Params p = params(n, H);
  const int sms = sm_count();
  if (!p.status || !sms) return cudaErrorInvalidDevice;
  CUtensorMap am, wm, om;
  if (!token_map(&am, q, n, H, kKeyDims + kRope) || !weight_map(&wm, w, H, 64) ||
      !token_map(&om, ql, n, H, kLatent + kRope))
    return cudaErrorInvalidValue;
  return launch<kAbsorb, 128>(am, wm, om, p, sms, s);
}

cudaError_t launch_mla_project(const void* ol, const void* w, int n, int H, void* o, cudaStream_t s) {
  if (n <= kMlaSmall) return launch_mla_project_small(ol, w, n, H, o, s);
  Params p = params(n, H);
  const int sms = sm_count();
  if (!p.status || !sms) return cudaErrorInvalidDevice;
  CUtensorMap am, wm, om;
  if (!token_map(&am, ol, n, H, kLatent) || !weight_map(&wm, w, H, 128) || !token_map(&om, o, n, H, kKeyDims))
    return cudaErrorInvalidValue;
  return launch<kProject, 128>(am, wm, om, p, sms, s);
}

}  // namespace cpattn

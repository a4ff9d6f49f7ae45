// The attention weights of a prompt batch on the tcgen05 tensor cores (bf16, head
// dim 64 or 128).
//
// One pass: with the LSE at hand a weight is exp(score - LSE) at once, so there is
// no second product and no running maximum.  Products are transposed: 256 keys of
// a request (two M tiles of 128) against 128 queries of one head,
//   S^T_t [128 keys x 128 queries] = K_t . Q^T,   t = 0, 1,
// so a key's weight is a sum along its own TMEM lane and stays in a thread over its
// queries.  The work of one head is the walk over (request, key block, query tile), tiles
// before the block's first key left out; workers (one CTA an SM) take equal parts of
// it.  Head by head (long prompts, by_heads()): each worker goes through its part once for
// every kv head (its keys once, its queries head by head), so that all workers are at the
// same head and the L2 holds its queries; every block's sums grow over the kv heads.
// Otherwise the walk has the heads inside the key block and is cut between
// heads, too.  A block's sums end in a row of their own, or in
// one of two part rows of each worker that shares the block with others, and a last
// kernel adds the parts in the order of the workers: no atomics, the same order every time.
//   warps 0-15  sums: warp w takes keys [32 (w % 4), +32) of M tile (w / 4) % 2 and
//               the half w / 8 of the query columns
//   warp 16     TMA producer (K blocks, Q tiles, the LSE of a tile)
//   warp 17     MMA issuer and TMEM owner
//   warps 18-19 relays: one more arrival on the barrier that frees a score buffer once
//               the step's queries and keys have landed, and one on the barrier of its
//               scores once the LSE has: the issuer waits twice a step, the sums once
//               (a wait costs some 140 clk even on a phase that is over)
// A sum warp has half of its columns on their way from TMEM while it works on the
// other half, across steps, too: the loads' latency is as long as the work.
// TMEM (512 columns): S^T of tile t in columns [256 t, +256), two buffers of 128.
// What bounds it: a step's products need 1,024 clk of the tensor cores, and 1,280 of
// shared memory at 128 B a clk, as both operands come from there; its 32,768 exponentials
// take the special function units as long as the products.  16,384 queries x 32 heads over 20,480 keys:
// 1.44 ms, 1,140 TFLOP/s (1.28 ms with the sums' work left out); the last 64 queries of
// nine prompts of up to 30,000 tokens: 138-147 us, a chain of short steps.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstring>

#include "early_launch.cuh"
#include "internal.h"
#include "plan_rows.cuh"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {
using namespace tc;

constexpr int kBlock = 256;  // keys of a block
constexpr int kBuf = 128;    // TMEM columns of a score buffer
constexpr int kSumWarps = 16, kThreads = 32 * (kSumWarps + 4);
constexpr int kWarpTma = kSumWarps, kWarpMma = kSumWarps + 1, kWarpRelay = kSumWarps + 2;  // and the one after it
constexpr int kLseSlots = 4;
constexpr float kLog2e = 1.4426950408889634f;

// KB buffers of a key block: two where a block meets few query tiles, one where it
// meets many (the ring of queries is then deeper).
// BQ queries a tile: 128, or 64 where no request has more (a window of its last queries).
template <int D, int KB, int BQ>
struct Cfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kTileBytes = 128 * D * 2;     // 128 keys
  static constexpr int kQBytes = BQ * D * 2;
  static constexpr int kQSlots = ((D == 128 ? 7 : 10) - 2 * KB) * 128 / BQ;
  static constexpr int kSmem = 2 * KB * kTileBytes + kQSlots * kQBytes + kLseSlots * BQ * 4;
};

// One request's share of the walk.
struct Req {
  int n, pre, q_base, kv_base;
  int w, off, nq;   // observed queries, the position of the first one, their tiles
  int m, c, m0, nb; // blocks 0 .. m0 - 1 are read by every tile, block k >= m0 from tile m k - c on
};
__host__ __device__ inline Req make_req(const cp_req_desc& d, int window, int bq) {
  Req r;
  r.n = d.new_len;
  r.pre = d.prefix_len;
  r.q_base = d.q_base;
  r.kv_base = d.kv_base;
  r.w = window > 0 && window < d.new_len ? window : d.new_len;
  r.off = d.prefix_len + d.new_len - r.w;
  r.nq = (int)(((long long)r.w + bq - 1) / bq);
  r.c = (int)(((long long)r.off + bq - 1) / bq);
  r.m = kBlock / bq;
  r.m0 = r.c / r.m + 1;
  r.nb = r.nq ? (int)(((long long)d.prefix_len + d.new_len + kBlock - 1) / kBlock) : 0;
  return r;
}
// The first tile that reads block k (its last query is at or behind the block's first key).
__host__ __device__ inline int first_tile(const Req& r, int k) { return k < r.m0 ? 0 : r.m * k - r.c; }
// Tiles of blocks 0 .. k - 1 (of one head).
__host__ __device__ inline long long tiles_before(const Req& r, long long k) {
  long long f = k * r.nq;
  if (k > r.m0) f -= r.m * (k * (k - 1) - (long long)r.m0 * (r.m0 - 1)) / 2 - (long long)r.c * (k - r.m0);
  return f;
}

struct Params {
  PrefillWeightsArgs a;
  int workers;
  int inner;             // heads inside the walk's blocks: Hq, or 1 where each worker takes its part for every head
  long long total;       // steps of the walk
  int bq;                // queries of a tile
  int n_tiles;           // query tiles of all requests
  long long* base;       // [R + 1] first step of every request
  int32_t* tile_base;    // [R + 1] first query tile
  int32_t* block_base;   // [R + 1] first key block (a request without queries has its blocks, too)
  float* lse;            // [Hq][n_tiles][bq] minus the LSE in log2 units, -inf where there is no query
  float* full;           // [2][KV] sums of blocks of one worker, by half of the columns
  float* part;           // [workers][2][2][kBlock]
  float scale_log2;
  unsigned* status;
  unsigned long long wait_ns;
  int stall_test;
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
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ float4 lds4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ void report_timeout(unsigned* status, unsigned site, volatile int* abort) {
  *abort = 1;
  if (atomicCAS(status, 0u, 1u) == 0u) {
    status[1] = kKernPrefillWeights;
    status[2] = site;
    status[3] = blockIdx.x;
    __threadfence();
  }
}

__device__ __forceinline__ cp_req_desc req_desc(const Params& p, int j) {
  return reinterpret_cast<const cp_req_desc*>(p.a.rows.plan + p.a.rows.off_req)[j];
}
// The last j of [0, R) with first(j) <= x.
template <typename F>
__device__ __forceinline__ int find(int R, F first, long long x) {
  int lo = 0, hi = R - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first(mid) <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}
__device__ __forceinline__ long long worker_start(const Params& p, long long w) { return p.total / p.workers * w + p.total % p.workers * w / p.workers; }

// ------------------------------------------------------------------ tables and LSE tiles

// Running sums over the requests: one block, a thread for consecutive requests.
__global__ void __launch_bounds__(256) weights_table_kernel(const Params p) {
  __shared__ long long s_step[256];
  __shared__ int s_tile[256], s_block[256];
  const int R = p.a.rows.R, per = (R + 255) / 256;
  const int j0 = min(R, (int)threadIdx.x * per), j1 = min(R, j0 + per);
  long long step = 0;
  int tile = 0, block = 0;
  auto each = [&](int j) {
    const Req r = make_req(req_desc(p, j), p.a.window, p.bq);
    step += p.inner * tiles_before(r, r.nb);
    tile += r.nq;
    block += (int)(((long long)r.pre + r.n + kBlock - 1) / kBlock);
  };
  for (int j = j0; j < j1; ++j) each(j);
  s_step[threadIdx.x] = step;
  s_tile[threadIdx.x] = tile;
  s_block[threadIdx.x] = block;
  wait_for_earlier_kernels();
  __syncthreads();
  step = tile = block = 0;
  for (int t = 0; t < (int)threadIdx.x; ++t) {
    step += s_step[t];
    tile += s_tile[t];
    block += s_block[t];
  }
  for (int j = j0; j < j1; ++j) {
    p.base[j] = step;
    p.tile_base[j] = tile;
    p.block_base[j] = block;
    each(j);
    if (j + 1 == R) {
      p.base[R] = step;
      p.tile_base[R] = tile;
      p.block_base[R] = block;
    }
  }
}

// A tile's LSE of every head: rank-major rows in, [head][tile][query] out.
__global__ void __launch_bounds__(256) weights_lse_kernel(const Params p) {
  wait_for_earlier_kernels();
  const int tile = blockIdx.x, R = p.a.rows.R, Hq = p.a.Hq;
  const int j = find(R, [&](int x) -> long long { return p.tile_base[x]; }, tile);
  const cp_req_desc d = req_desc(p, j);
  const Req r = make_req(d, p.a.window, p.bq);
  const int i0 = r.n - r.w + (tile - p.tile_base[j]) * p.bq;  // the tile's first query
  __shared__ int s_row[128];
  for (int x = threadIdx.x; x < p.bq; x += 256) s_row[x] = i0 + x < r.n ? plan_row(p.a.rows, j, d, i0 + x) : -1;
  __syncthreads();
  for (int h0 = 0; h0 < Hq; h0 += 8) {
    // eight heads of a row side by side, so that whole sectors are read
    for (int e = threadIdx.x; e < p.bq * 8; e += 256) {
      const int x = e >> 3, h = h0 + (e & 7);
      if (h >= Hq) continue;
      float v = -INFINITY;
      if (s_row[x] >= 0) {
        const float l = __ldcg(p.a.lse + (long long)s_row[x] * Hq + h);
        if (l != -INFINITY) v = -l * kLog2e;  // a query without keys weighs nothing
      }
      p.lse[((long long)h * p.n_tiles + tile) * p.bq + x] = v;
    }
  }
}

// ------------------------------------------------------------------ sums

// A run of steps for one sum warp: the sum of the weights of its 32 keys and half of the
// query columns; *ok = false if a wait ran out.  MASK: some columns do not read a key, or are
// no query of the request.  Functions of their own, so that the loops have the registers
// that the walk's state would take, and the common one no masks (with both in one loop
// 1.50 ms for 16,384 queries x 32 heads over 20,480 keys, else 1.44).
struct SumArgs {
  uint32_t tmem;             // this warp's lanes, its tile's first buffer, its columns
  uint32_t s, go, lfree;     // barriers: scores, free buffers (of the tile's first buffer), LSE slots
  uint32_t lse;              // ring of LSE, from this warp's columns on
  float scale;
  int nq, steps, tile;       // first step, number of steps, query tile of the first one
  int first, last;           // tiles go round [first, last), head after head
  int lo, cols;              // keys are read from column lo - BQ tile on (of this half), columns end at cols - BQ tile
  unsigned long long wait_ns;
  volatile int* abort;
};
template <bool MASK, int BQ>
__device__ __noinline__ float sum_steps(const SumArgs a, bool* ok) {
  const int lane = threadIdx.x & 31;
  uint32_t ra[32], rb[32];
  float sum = 0.f;
  int nq = a.nq, tile = a.tile;
  auto wait_s = [&](int n) {
    const bool got = __all_sync(0xffffffffu, mbar_wait(a.s + 8 * (n & 1), (n >> 1) & 1, a.wait_ns, a.abort));
    if (got) tc_fence_after();
    else *ok = false;
    return got;
  };
  if (!wait_s(nq)) return sum;
  tmem_ld32(a.tmem + (nq & 1) * kBuf, ra);
  for (const int end = nq + a.steps; nq < end; ++nq) {
    const uint32_t lse = a.lse + (nq % kLseSlots) * (BQ * 4);
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    auto add = [&](uint32_t (&sr)[32], int c0) {
      uint32_t keep = 0xffffffffu;
      if constexpr (MASK) {  // bits [from, to) stay
        const int from = min(max(a.lo - tile * BQ - c0, 0), 32), to = min(max(a.cols - tile * BQ - c0, 0), 32);
        keep = __funnelshift_lc(0xffffffffu, 0u, to) & ~__funnelshift_lc(0xffffffffu, 0u, from);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float4 v = lds4(lse + (c0 + 4 * e) * 4);
        float u0, u1, u2, u3;
        fma2(u0, u1, __uint_as_float(sr[4 * e]), __uint_as_float(sr[4 * e + 1]), a.scale, a.scale, v.x, v.y);
        fma2(u2, u3, __uint_as_float(sr[4 * e + 2]), __uint_as_float(sr[4 * e + 3]), a.scale, a.scale, v.z, v.w);
        if constexpr (MASK) {  // behind the LSE, which may be NaN
          if (!(keep >> (4 * e) & 1)) u0 = -INFINITY;
          if (!(keep >> (4 * e + 1) & 1)) u1 = -INFINITY;
          if (!(keep >> (4 * e + 2) & 1)) u2 = -INFINITY;
          if (!(keep >> (4 * e + 3) & 1)) u3 = -INFINITY;
        }
        add2(s0, s1, s0, s1, ex2(u0), ex2(u1));
        add2(s2, s3, s2, s3, ex2(u2), ex2(u3));
      }
    };
    tmem_ld_wait();
    if constexpr (BQ == 128) {
      tmem_ld32(a.tmem + (nq & 1) * kBuf + 32, rb);
      add(ra, 0);
      tmem_ld_wait();
    } else {  // 32 columns: the other array takes the next step's
#pragma unroll
      for (int e = 0; e < 32; ++e) rb[e] = ra[e];
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(a.go + 8 * (nq & 1));
    if (nq + 1 < end) {
      if (!wait_s(nq + 1)) return sum;
      tmem_ld32(a.tmem + ((nq + 1) & 1) * kBuf, ra);
    }
    add(rb, BQ / 2 - 32);
    __syncwarp();
    if (lane == 0) mbar_arrive(a.lfree + 8 * (nq % kLseSlots));
    sum += (s0 + s1) + (s2 + s3);
    if (++tile == a.last) tile = a.first;
  }
  return sum;
}

template <int D, int KB, int BQ>
__global__ void __launch_bounds__(kThreads, 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap qmap,
                      const __grid_constant__ Params p) {
  using C = Cfg<D, KB, BQ>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sK = smem;                                 // [KB buffers][2 tiles]
  uint8_t* sQ = smem + 2 * KB * C::kTileBytes;             // ring of query tiles
  float* sL = reinterpret_cast<float*>(sQ + C::kQSlots * C::kQBytes);  // ring of their LSE
  __shared__ __align__(8) uint64_t bar_k[KB], bar_kfree[KB], bar_q[C::kQSlots], bar_qfree[C::kQSlots], bar_l[kLseSlots],
      bar_lfree[kLseSlots], bar_s[4], bar_go[4], bar_drain, bar_never;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ volatile int zero_flag;
  const PrefillWeightsArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < KB; ++i) {
      mbar_init(smem_u32(&bar_k[i]), 1);
      mbar_init(smem_u32(&bar_kfree[i]), 1);
    }
    for (int i = 0; i < C::kQSlots; ++i) {
      mbar_init(smem_u32(&bar_q[i]), 1);
      mbar_init(smem_u32(&bar_qfree[i]), 1);
    }
    for (int i = 0; i < kLseSlots; ++i) {
      mbar_init(smem_u32(&bar_l[i]), 1);
      mbar_init(smem_u32(&bar_lfree[i]), kSumWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(smem_u32(&bar_s[i]), 2);  // the products' commit and the relay
      mbar_init(smem_u32(&bar_go[i]), kSumWarps / 2 + 1);  // a tile's sum warps and the relay
    }
    mbar_init(smem_u32(&bar_drain), 1);
    mbar_init(smem_u32(&bar_never), 1);
    abort_flag = 0;
    zero_flag = 0;
    mbar_init_fence();
  }
  if (warp == kWarpMma) tmem_alloc(smem_u32(&tmem_slot), 512);
  if (warp == kWarpTma && lane == 0) {
    prefetch_tmap(&kmap);
    prefetch_tmap(&qmap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  wait_for_earlier_kernels();
  const long long begin = worker_start(p, blockIdx.x), end = worker_start(p, blockIdx.x + 1);

  // The spans of this worker, in order: each(request, block, first tile, tiles, heads
  // [h0, h1) of one kv head or of all, first step x0 and last x1 of them (head by head over
  // the tiles), whether the span begins and ends the block's work of this pass, pass).
  // With inner == 1 a pass is a kv head and the tiles are the worker's own.
  struct Span {
    int j, kb, first, cnt, h0, x0, x1, pass;
    bool whole;    // the block is this worker's alone
    bool begins;   // the block's first step is this worker's
  };
  // Heads of a span's first kv head from its first step on.
  auto heads_left = [&](const Span& sp) { return a.G - (sp.h0 + sp.x0 / sp.cnt) % a.G; };
  auto walk = [&](auto&& each) {
    if (begin >= end) return;
    const int passes = p.inner == 1 ? a.Hkv : 1;
    for (int pass = 0; pass < passes; ++pass) {
      int j = find(a.rows.R, [&](int x) { return p.base[x]; }, begin);
      Req r = make_req(req_desc(p, j), a.window, BQ);
      long long base = p.base[j], pos = begin;
      int kb;  // the block of step `begin`: binary search of the sums
      {
        const long long t = (begin - base) / p.inner;
        int lo = 0, hi = r.nb - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (tiles_before(r, mid) <= t) lo = mid; else hi = mid - 1;
        }
        kb = lo;
      }
      while (pos < end) {
        while (kb >= r.nb) {  // the next request with steps
          ++j;
          r = make_req(req_desc(p, j), a.window, BQ);
          base = p.base[j];
          kb = 0;
        }
        const long long s0 = base + p.inner * tiles_before(r, kb);
        const int first = first_tile(r, kb), tiles = r.nq - first;
        const int a0 = (int)(pos - s0), a1 = (int)min((long long)p.inner * tiles, end - s0);
        Span sp = {j, kb, first, tiles, 0, a0, a1, pass, a0 == 0 && a1 == p.inner * tiles, a0 == 0};
        if (p.inner == 1) {  // tiles [a0, a1) for each head of the pass
          sp.first = first + a0;
          sp.cnt = a1 - a0;
          sp.h0 = pass * a.G;
          sp.x0 = 0;
          sp.x1 = a.G * sp.cnt;
        }
        if (!each(r, sp)) return;
        pos = s0 + a1;
        ++kb;
      }
    }
  };

  if (warp == kWarpTma) {
    // ------------------------------------------------------------ TMA
    bool ok = true;
    int nk = 0, nq = 0;  // K blocks and query tiles loaded so far
    auto wait_all = [&](uint64_t* bar, uint32_t parity, unsigned site) {
      if (__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.wait_ns, &abort_flag))) return true;
      if (lane == 0) report_timeout(p.status, site, &abort_flag);
      return ok = false;
    };
    walk([&](const Req& r, const Span& sp) {
      int h = sp.x0 / sp.cnt, q = sp.x0 - h * sp.cnt, g_in = -1;
      h += sp.h0;
      int g = h / a.G, hg = h - g * a.G;
      const int tile0 = p.tile_base[sp.j];
      for (int x = sp.x0; x < sp.x1; ++x) {
        const int s = nq % C::kQSlots, l = nq % kLseSlots;
        if (nq >= C::kQSlots && !wait_all(&bar_qfree[s], (nq / C::kQSlots - 1) & 1, 2)) return false;
        if (nq >= kLseSlots && !wait_all(&bar_lfree[l], (nq / kLseSlots - 1) & 1, 3)) return false;
        if (elect_one()) {
          const uint32_t full = smem_u32(&bar_q[s]), dst = smem_u32(sQ + s * C::kQBytes);
          mbar_expect_tx(full, C::kQBytes);
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_3d(dst + c * (BQ * 128), &qmap, c * 64, h, r.q_base + r.n - r.w + (sp.first + q) * BQ, full);
          const uint32_t lf = smem_u32(&bar_l[l]);
          mbar_expect_tx(lf, BQ * 4);
          bulk_load(smem_u32(sL + l * BQ), p.lse + ((long long)h * p.n_tiles + tile0 + sp.first + q) * BQ, BQ * 4, lf);
        }
        __syncwarp();
        ++nq;
        if (g != g_in) {  // behind the first query tile that meets the block: that is on its way meanwhile
          g_in = g;
          const int b = nk % KB;
          if (nk >= KB && !wait_all(&bar_kfree[b], (nk / KB - 1) & 1, 1)) return false;
          if (elect_one()) {
            const uint32_t full = smem_u32(&bar_k[b]), dst = smem_u32(sK + b * 2 * C::kTileBytes);
            mbar_expect_tx(full, 2 * C::kTileBytes);
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_3d(dst + t * C::kTileBytes + c * (128 * 128), &kmap, c * 64, g, r.kv_base + sp.kb * kBlock + t * 128, full);
          }
          __syncwarp();
          ++nk;
        }
        if (++q == sp.cnt) {
          q = 0;
          ++h;
          if (++hg == a.G) {
            hg = 0;
            ++g;
          }
        }
      }
      return true;
    });
    if (!ok) {
      // never leave with a copy in flight: the last fill of every place
      auto drain = [&](uint64_t* bar, int n, int slots) {
        for (int x = 0; x < slots; ++x) {
          const int fills = n / slots + (x < n % slots);
          if (fills > 0) mbar_wait(smem_u32(bar + x), (fills - 1) & 1, 1000000000ull, &zero_flag);
        }
      };
      drain(bar_k, nk, KB);
      drain(bar_q, nq, C::kQSlots);
      drain(bar_l, nq, kLseSlots);
      __syncwarp();
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issue
    const uint32_t id = idesc_bf16_f32(128, BQ, 0, 0);
    const uint64_t dK = smem_desc(smem_u32(sK), 16, 1024), dQ = smem_desc(smem_u32(sQ), 16, 1024);
    int nk = 0, nq = 0;
    auto wait_all = [&](uint64_t* bar, uint32_t parity, unsigned site) {
      if (__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.wait_ns, &abort_flag))) return true;
      if (lane == 0) report_timeout(p.status, site, &abort_flag);
      return false;
    };
    if (!p.stall_test || wait_all(&bar_never, 0, 10))
      walk([&](const Req&, const Span& sp) {
        // steps until the kv head changes
        int left = heads_left(sp) * sp.cnt - sp.x0 % sp.cnt;
        ++nk;
        for (int x = sp.x0; x < sp.x1; ++x, ++nq) {
          if (left == 0) {
            left = a.G * sp.cnt;
            ++nk;
          }
          --left;
          const bool last = x + 1 == sp.x1 || left == 0;  // of this K block
          const int s = nq % C::kQSlots, buf = nq & 1;
          for (int t = 0; t < 2; ++t) {
            // the buffer's scores of two steps ago are read, this step's queries and keys have landed
            if (!wait_all(&bar_go[2 * t + buf], (nq >> 1) & 1, 6)) return false;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t k = dK + ((uint32_t)((((nk - 1) % KB) * 2 + t) * C::kTileBytes) >> 4);
              const uint64_t b = dQ + ((uint32_t)(s * C::kQBytes) >> 4);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t ko = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4, qo = ((kk >> 2) * (BQ * 128) + (kk & 3) * 32) >> 4;
                mma_ss(tmem + t * 256 + buf * kBuf, k + ko, b + qo, id, kk > 0);
              }
              mma_commit(smem_u32(&bar_s[2 * t + buf]));
              if (t == 1) {
                mma_commit(smem_u32(&bar_qfree[s]));
                if (last) mma_commit(smem_u32(&bar_kfree[(nk - 1) % KB]));
              }
            }
            __syncwarp();
          }
        }
        return true;
      });
    // never free TMEM under a running product
    if (elect_one()) mma_commit(smem_u32(&bar_drain));
    __syncwarp();
    mbar_wait(smem_u32(&bar_drain), 0, 1000000000ull, &zero_flag);
  } else if (warp >= kWarpRelay) {
    // ------------------------------------------------------------ relays
    // The arrival for step n comes after the barrier's phase of step n - 2 is over, so
    // no phase takes an arrival that is the next one's.
    const bool operands = warp == kWarpRelay;  // else the LSE
    int nq = 0, nk = 0;
    walk([&](const Req&, const Span& sp) {
      int left = heads_left(sp) * sp.cnt - sp.x0 % sp.cnt;
      bool keys = true;  // the step's K block is a new one
      for (int x = sp.x0; x < sp.x1; ++x, ++nq) {
        bool got;
        if (operands) {
          got = mbar_wait(smem_u32(&bar_q[nq % C::kQSlots]), (nq / C::kQSlots) & 1, p.wait_ns, &abort_flag);
          if (left == 0) {
            left = a.G * sp.cnt;
            keys = true;
          }
          --left;
          if (keys) {
            got = got && mbar_wait(smem_u32(&bar_k[nk % KB]), (nk / KB) & 1, p.wait_ns, &abort_flag);
            ++nk;
            keys = false;
          }
        } else {
          got = mbar_wait(smem_u32(&bar_l[nq % kLseSlots]), (nq / kLseSlots) & 1, p.wait_ns, &abort_flag);
        }
        for (int t = 0; t < 2 && got; ++t) {
          const uint32_t bar = smem_u32(operands ? &bar_go[2 * t + (nq & 1)] : &bar_s[2 * t + (nq & 1)]);
          if (nq >= 2) got = mbar_wait(bar, (nq / 2 - 1) & 1, p.wait_ns, &abort_flag);
          got = __all_sync(0xffffffffu, got);
          if (got && lane == 0) mbar_arrive(bar);
        }
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) report_timeout(p.status, 8, &abort_flag);
          return false;
        }
      }
      return true;
    });
  } else {
    // ------------------------------------------------------------ sums
    const int quarter = warp & 3, t = (warp >> 2) & 1, half = warp >> 3;
    const int i = t * 128 + quarter * 32 + lane;  // key of the block
    SumArgs sa;
    sa.tmem = tmem + ((uint32_t)(quarter * 32) << 16) + t * 256 + BQ / 2 * half;
    sa.s = smem_u32(&bar_s[2 * t]);
    sa.go = smem_u32(&bar_go[2 * t]);
    sa.lfree = smem_u32(&bar_lfree[0]);
    sa.lse = smem_u32(sL + BQ / 2 * half);
    sa.scale = p.scale_log2;
    sa.nq = 0;
    sa.wait_ns = p.wait_ns;
    sa.abort = &abort_flag;
    if (lane == 0) {  // both buffers are free
      mbar_arrive(smem_u32(&bar_go[2 * t]));
      mbar_arrive(smem_u32(&bar_go[2 * t + 1]));
    }
    walk([&](const Req& r, const Span& sp) {
      // column c of tile q stands at position off + BQ q + c: it reads this key from c = lo - BQ q on
      sa.lo = sp.kb * kBlock + i - r.off - BQ / 2 * half;
      sa.cols = r.w - BQ / 2 * half;
      // tiles [mask0, mask1) have all of this warp's columns for all of its keys
      const int warp_lo = max(0, sa.lo - lane + 31), last = sp.first + sp.cnt;
      const int mask0 = (warp_lo + BQ - 1) / BQ, mask1 = sa.cols < BQ / 2 ? 0 : (sa.cols - BQ / 2) / BQ + 1;
      sa.tile = sp.first + sp.x0 % sp.cnt;
      sa.first = sp.first;
      sa.last = last;
      const bool none = max(mask0, sp.first) >= min(mask1, last);  // no such tile here
      float sum = 0.f;
      bool ok = true;
      for (int left = sp.x1 - sp.x0; left > 0 && ok; left -= sa.steps) {
        const bool whole = sa.tile >= mask0 && sa.tile < mask1;
        sa.steps = none ? left : min(left, (whole ? min(mask1, last) : sa.tile < mask0 ? min(mask0, last) : last) - sa.tile);
        sum += whole ? sum_steps<false, BQ>(sa, &ok) : sum_steps<true, BQ>(sa, &ok);
        sa.nq += sa.steps;
        sa.tile += sa.steps;
        if (sa.tile == last) sa.tile = sp.first;
      }
      if (!ok) {
        if (lane == 0) report_timeout(p.status, 7, &abort_flag);
        return false;
      }
      // the whole block: its own row; else this worker's first part (the block began
      // with another worker) or its second.  Later kv heads add to what this thread wrote.
      float* to = nullptr;
      if (!sp.whole) {
        to = p.part + (((long long)blockIdx.x * 2 + sp.begins) * 2 + half) * kBlock + i;
      } else {
        const long long row = (long long)sp.kb * kBlock + i;
        if (row < (long long)r.pre + r.n) to = p.full + (long long)half * a.rows.KV + r.kv_base + row;
      }
      if (to) *to = sp.pass ? *to + sum : sum;
      return true;
    });
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ parts

// A block of keys: its row, or its workers' parts in order.
__global__ void __launch_bounds__(kBlock) weights_join_kernel(const Params p) {
  wait_for_earlier_kernels();
  const int R = p.a.rows.R;
  const int j = find(R, [&](int x) -> long long { return p.block_base[x]; }, blockIdx.x);
  const Req r = make_req(req_desc(p, j), p.a.window, p.bq);
  const int kb = blockIdx.x - p.block_base[j];
  const long long row = (long long)kb * kBlock + threadIdx.x;
  if (row >= (long long)r.pre + r.n) return;
  float sum = 0.f;
  if (kb < r.nb) {
    const long long s0 = p.base[j] + p.inner * tiles_before(r, kb), s1 = p.base[j] + p.inner * tiles_before(r, kb + 1);
    // the last worker that starts at or before a step
    auto worker = [&](long long s) { return find(p.workers, [&](int w) { return worker_start(p, w); }, s); };
    const int w0 = worker(s0), w1 = worker(s1 - 1);
    if (w0 == w1) {
      const long long at = r.kv_base + row;
      sum = __ldcg(p.full + at) + __ldcg(p.full + p.a.rows.KV + at);
    } else {
      for (int w = w0; w <= w1; ++w) {
        if (worker_start(p, w) == worker_start(p, w + 1)) continue;  // a worker without steps
        const float* x = p.part + (((long long)w * 2 + (worker_start(p, w) <= s0)) * 2) * kBlock + threadIdx.x;
        sum += __ldcg(x) + __ldcg(x + kBlock);
      }
    }
  }
  p.a.out[r.kv_base + row] = sum;
}

struct Layout {
  long long total = 0;  // tiles of one head
  int n_tiles = 0, n_blocks = 0, bq = 64;
  size_t base, tile_base, block_base, lse, full, part, bytes;
};
Layout layout(const cp_req_desc* reqs, int R, int KV, int Hq, int window, int workers) {
  Layout l;
  for (int j = 0; j < R && l.bq == 64; ++j)
    if ((window > 0 && window < reqs[j].new_len ? window : reqs[j].new_len) > 64) l.bq = 128;
  for (int j = 0; j < R; ++j) {
    const Req r = make_req(reqs[j], window, l.bq);
    l.total += tiles_before(r, r.nb);
    l.n_tiles += r.nq;
    l.n_blocks += (int)(((long long)r.pre + r.n + kBlock - 1) / kBlock);
  }
  size_t at = 0;
  auto place = [&](size_t n) {
    const size_t here = at;
    at = (at + n + 511) / 512 * 512;
    return here;
  };
  l.base = place(8 * ((size_t)R + 1));
  l.tile_base = place(4 * ((size_t)R + 1));
  l.block_base = place(4 * ((size_t)R + 1));
  l.lse = place((size_t)Hq * l.n_tiles * l.bq * 4);
  l.full = place((size_t)2 * KV * 4);
  l.part = place((size_t)workers * 4 * kBlock * 4);
  l.bytes = at;
  return l;
}

constexpr int kWorkers = 152;  // one an SM

// Whether the workers go head by head.  A pass over a kv head costs them some 9 us (64 kv heads of
// one, 12,288 queries: 1,734 us head by head, 1,134 with the heads inside), and saves up to
// 10 % where all heads' queries pass the L2's 129 MB: what a pass saves grows with its
// steps, tiles of a worker x heads of a kv head.  At D = 128 on changing inputs, head by
// head and heads inside, us (steps of a pass, MB of queries):
//   32 heads / 8: 12,288 queries 639 and 580 (62, 101); 16,384: 1,022 and 1,000 (109, 134), behind
//   4,096 more keys 1,452 and 1,473 (163, 134); 20,480: 1,538 and 1,540 (170, 168); 24,576:
//   2,145 and 2,207 (245, 201); 28,672: 2,842 and 2,994 (333, 235)
//   64 / 8: 12,288: 1,169 and 1,171 (124, 201); 16,384: 1,944 and 2,030 (219, 268)
// At D = 64 a step's queries are half as long, and the heads inside were faster throughout
// (32 / 8, 24,576 queries of 101 MB 1,816 and 1,738; 64 / 8, 49,152 of 403 MB 13,130 and 13,034).
bool by_heads(const Layout& l, int T, int Hq, int G, int D, int workers) {
  return l.bq == 128 && D == 128 && l.total * G >= 130ll * workers && (long long)T * Hq * D * 2 >= 128ll << 20;
}

template <int D, int KB, int BQ>
cudaError_t launch_d(const CUtensorMap& km, const CUtensorMap& qm, const Params& p, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(weights_tc_kernel<D, KB, BQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, KB, BQ>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(weights_tc_kernel<D, KB, BQ>, (unsigned)p.workers, kThreads, Cfg<D, KB, BQ>::kSmem, s, 1, km, qm, p);
}

}  // namespace

size_t prefill_weights_tc_bytes(const int32_t* host_plan, const cp_plan_header& h, int Hq, int window) {
  return layout(reinterpret_cast<const cp_req_desc*>(host_plan + h.off_req), h.R, h.KV, Hq, window, kWorkers).bytes;
}

cudaError_t launch_prefill_weights_tc(const PrefillWeightsArgs& a, const int32_t* host_plan, const cp_plan_header& h, int D,
                                      void* ws, bool stall_test, cudaStream_t s) {
  const Layout l = layout(reinterpret_cast<const cp_req_desc*>(host_plan + h.off_req), h.R, h.KV, a.Hq, a.window, kWorkers);
  uint8_t* w = static_cast<uint8_t*>(ws);
  Params p;
  p.a = a;
  p.workers = kWorkers;
  const bool heads = by_heads(l, h.T, a.Hq, a.G, D, kWorkers);
  p.inner = heads ? 1 : a.Hq;
  p.total = l.total * p.inner;
  p.bq = l.bq;
  p.n_tiles = l.n_tiles;
  p.base = reinterpret_cast<long long*>(w + l.base);
  p.tile_base = reinterpret_cast<int32_t*>(w + l.tile_base);
  p.block_base = reinterpret_cast<int32_t*>(w + l.block_base);
  p.lse = reinterpret_cast<float*>(w + l.lse);
  p.full = reinterpret_cast<float*>(w + l.full);
  p.part = reinterpret_cast<float*>(w + l.part);
  p.scale_log2 = a.sm_scale * kLog2e;
  p.status = device_status_ptr();
  if (!p.status) return cudaErrorInvalidDevice;
  p.wait_ns = stall_test ? 50000000ull : wait_limit_ns();
  p.stall_test = stall_test ? 1 : 0;
  cudaError_t e = launch_early(weights_table_kernel, 1, 256, 0, s, 1, p);
  if (e == cudaSuccess && l.n_tiles > 0) {
    CUtensorMap km, qm;
    const uint32_t box[3] = {64, 1, 128}, qbox[3] = {64, 1, (uint32_t)l.bq};
    const uint64_t kd[3] = {(uint64_t)D, (uint64_t)a.Hkv, (uint64_t)a.rows.KV}, ks[2] = {(uint64_t)D * 2, (uint64_t)a.Hkv * D * 2};
    const uint64_t qd[3] = {(uint64_t)D, (uint64_t)a.Hq, (uint64_t)a.rows.T}, qs[2] = {(uint64_t)D * 2, (uint64_t)a.Hq * D * 2};
    if (!encode_tensor_map_bf16(&km, a.k, 3, kd, ks, box) || !encode_tensor_map_bf16(&qm, a.q, 3, qd, qs, qbox))
      return cudaErrorInvalidValue;
    e = launch_early(weights_lse_kernel, (unsigned)l.n_tiles, 256, 0, s, 1, p);
    if (e == cudaSuccess) {
      if (D == 128)
        e = heads ? launch_d<128, 1, 128>(km, qm, p, s) : l.bq == 64 ? launch_d<128, 2, 64>(km, qm, p, s) : launch_d<128, 2, 128>(km, qm, p, s);
      else
        e = l.bq == 64 ? launch_d<64, 2, 64>(km, qm, p, s) : launch_d<64, 2, 128>(km, qm, p, s);
    }
  }
  if (e == cudaSuccess) e = launch_early(weights_join_kernel, (unsigned)l.n_blocks, kBlock, 0, s, 1, p);
  return e;
}

}  // namespace cpattn

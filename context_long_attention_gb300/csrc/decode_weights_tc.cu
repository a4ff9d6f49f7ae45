// The attention weights of a decode step over a paged cache on the tcgen05
// tensor cores: GQA (bf16 at head dim 64 or 128, E4M3 at 128) and the latent entries of
// MLA (576, bf16 or E4M3).
//
// The step reads every key once more (no value), so memory bounds it.  Products
// are transposed: a tile's 128 cache rows are the MMA's M, the columns the query
// rows x heads of one kv head,
//   S^T [128 rows x NP] = K_g tile . Q_g^T,
// so a row's weight is a sum over the columns of its own TMEM lane, over all kv
// heads in turn, and stays in one thread: no atomics, the same order every time.
// A tile's kv heads and their dims come as 16 KB chunks (128 rows x 128 bytes) through
// a ring, rows whole and in order as far as the memory sees them.
//   warps 0-3  sums (thread = cache row); at a new request its queries and LSE to
//              shared memory
//   warp 4     TMA producer    warp 5  MMA issuer and TMEM owner
// E4M3: the codes are multiplied as they are stored.  A bf16 query row enters as two
// E4M3 numbers, hi + lo / 16 of the row times a power of two that brings its largest
// element to [128, 256): 4 + 4 significant bits hold bf16's 8 down to 2^-13 of the largest,
// and smaller elements are off by up to 2^-21 of it; the columns of hi and lo lie side by
// side in one product.
// Measured: 16 requests of up to 32,768 tokens, 8 kv heads of 128 (470 MB of keys) 94 us,
// 0.75 of HBM, over E4M3 64 us of 235 MB; 64 of up to 20,000 latent E4M3 entries 90 us, 0.6: a
// worker meets 1.4 requests there, whose 64 query rows take some 5 us each; over bf16 126 us, 0.85.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstring>

#include "early_launch.cuh"
#include "internal.h"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {
using namespace tc;

constexpr int kRows = 128, kChunkBytes = kRows * 128;
constexpr int kThreads = 192, kSum = 128, kWarpTma = 4, kWarpMma = 5;
constexpr int kMaxStages = 12, kBufs = 4;
constexpr int kMaxQBytes = 96 * 1024;
constexpr int kSmemLimit = 226 * 1024;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  DecodeWeightsArgs a;
  int D, chunks, stages;  // chunks of a kv head's dims
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
__device__ __forceinline__ void report_timeout(unsigned* status, unsigned site, volatile int* abort) {
  *abort = 1;
  if (atomicCAS(status, 0u, 1u) == 0u) {
    status[1] = kKernDecodeWeights;
    status[2] = site;
    status[3] = blockIdx.x;
    __threadfence();
  }
}
// Two floats to two E4M3 codes, `a` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ void e4m3x2_value(uint32_t codes, float& a, float& b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  asm("{\n .reg .f16 l, u;\n mov.b32 {l, u}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, u;\n}" : "=f"(a), "=f"(b) : "r"(h));
}

template <int NC>
__device__ __forceinline__ void tmem_ld_cols(uint32_t addr, uint32_t (&r)[NC]) {
  if constexpr (NC == 16) {
    tmem_ld16(addr, r);
  } else {
#pragma unroll
    for (int c = 0; c < NC / 32; ++c) tmem_ld32(addr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&r[32 * c]));
  }
}

struct Item {
  int pair, b, row_begin, nrows, ntiles;
  cp_pair_desc pd;
};
__device__ __forceinline__ Item read_item(const DecodeWeightsArgs& a, int wi) {
  const cp_work_desc wd = reinterpret_cast<const cp_work_desc*>(a.plan + a.off_work)[wi];
  Item it;
  it.pair = wd.pair;
  it.b = wd.pair % a.B;
  it.pd = reinterpret_cast<const cp_pair_desc*>(a.plan + a.off_pair)[wd.pair];
  it.row_begin = wd.row_begin;
  it.nrows = wd.row_end - wd.row_begin;
  it.ntiles = (it.nrows + kRows - 1) / kRows;
  return it;
}

// NP columns a kv head (16, 32 or 64).
template <int NP, bool F8>
__global__ void __launch_bounds__(kThreads, 1)
    decode_weights_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ Params p) {
  constexpr int NT = F8 ? 2 * NP : NP;              // columns of a product
  constexpr int kCols = kBufs * NT < 32 ? 32 : kBufs * NT;
  constexpr int kElems = F8 ? 128 : 64;             // of a chunk's row
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const DecodeWeightsArgs& a = p.a;
  uint8_t* sK = smem;                               // [stages][128 rows x 128 B]
  uint8_t* sQ = smem + p.stages * kChunkBytes;      // [Hkv][chunks][NT rows x 128 B]
  const int q_bytes = a.Hkv * p.chunks * NT * 128;
  float* sL = reinterpret_cast<float*>(sQ + q_bytes);  // [Hkv][NP] LSE in log2 units, +inf: no weight
  float* sF = sL + a.Hkv * NP;                         // [Hkv][NP] E4M3: what undoes the row's power of two
  __shared__ __align__(8) uint64_t bar_full[kMaxStages], bar_empty[kMaxStages], bar_s[kBufs], bar_free[kBufs], bar_q,
      bar_drain, bar_never;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ volatile int zero_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&bar_full[s]), 1);
      mbar_init(smem_u32(&bar_empty[s]), 1);
    }
    for (int s = 0; s < kBufs; ++s) {
      mbar_init(smem_u32(&bar_s[s]), 1);
      mbar_init(smem_u32(&bar_free[s]), 4);
    }
    mbar_init(smem_u32(&bar_q), 1);
    mbar_init(smem_u32(&bar_drain), 1);
    mbar_init(smem_u32(&bar_never), 1);
    abort_flag = 0;
    zero_flag = 0;
    mbar_init_fence();
  }
  // query rows past the columns in use and dims past D stay zero
  for (int i = threadIdx.x; i < q_bytes / 16; i += kThreads) reinterpret_cast<uint4*>(sQ)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (warp == kWarpMma) tmem_alloc(smem_u32(&tmem_slot), kCols);
  if (warp == kWarpTma && lane == 0) prefetch_tmap(&kmap);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  wait_for_earlier_kernels();
  const int w0 = a.plan[a.off_worker + blockIdx.x], w1 = a.plan[a.off_worker + blockIdx.x + 1];

  if (warp == kWarpTma) {
    // ------------------------------------------------------------ TMA
    bool ok = true;
    int s = 0, use = 0;  // the stage of the next chunk and how often it was filled before
    int filled = 0;
    for (int wi = w0; wi < w1 && ok; ++wi) {
      const Item it = read_item(a, wi);
      // pool rows of a tile's two 64-row halves (each inside one page; a half behind the
      // pair's rows lies past the pool and reads zeros), found one tile ahead
      auto locate = [&](int j, int half) {
        const int i = it.row_begin + j * kRows + 64 * half;
        return (int)(i < it.pd.rows ? map_row_early(a.rm, it.pair, 0, i) : a.rm.pool_rows);
      };
      int y0 = 0, y1 = 0;
      if (it.ntiles > 0) {
        y0 = locate(0, 0);
        y1 = locate(0, 1);
      }
      for (int j = 0; j < it.ntiles && ok; ++j) {
        int n0 = 0, n1 = 0;
        if (j + 1 < it.ntiles) {
          n0 = locate(j + 1, 0);
          n1 = locate(j + 1, 1);
        }
        for (int kh = 0; kh < a.Hkv && ok; ++kh)
          for (int c = 0; c < p.chunks; ++c) {
            if (use > 0 &&
                !__all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_empty[s]), (use - 1) & 1, p.wait_ns, &abort_flag))) {
              if (lane == 0) report_timeout(p.status, 1, &abort_flag);
              ok = false;
              break;
            }
            if (elect_one()) {
              const uint32_t full = smem_u32(&bar_full[s]), dst = smem_u32(sK + s * kChunkBytes);
              mbar_expect_tx(full, kChunkBytes);
              tma_load_3d(dst, &kmap, c * kElems, kh, y0, full);
              tma_load_3d(dst + kChunkBytes / 2, &kmap, c * kElems, kh, y1, full);
            }
            __syncwarp();
            ++filled;
            if (++s == p.stages) {
              s = 0;
              ++use;
            }
          }
        y0 = n0;
        y1 = n1;
      }
    }
    if (!ok) {
      // never leave with a copy in flight: each stage's last fill
      for (int x = 0; x < p.stages; ++x) {
        const int fills = filled / p.stages + (x < filled % p.stages);
        if (fills > 0) mbar_wait(smem_u32(&bar_full[x]), (fills - 1) & 1, 1000000000ull, &zero_flag);
      }
      __syncwarp();
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA issue
    const uint32_t id = F8 ? idesc_e4m3_f32(kRows, NT, 0, 0) : idesc_bf16_f32(kRows, NT, 0, 0);
    const uint64_t dK = smem_desc(smem_u32(sK), 16, 1024), dQ = smem_desc(smem_u32(sQ), 16, 1024);
    bool ok = true;
    int s = 0, phase = 0, u = 0, nq = 0, q_b = -1;
    auto wait_all = [&](uint64_t* bar, uint32_t parity, unsigned site) {
      if (__all_sync(0xffffffffu, mbar_wait(smem_u32(bar), parity, p.wait_ns, &abort_flag))) return true;
      if (lane == 0) report_timeout(p.status, site, &abort_flag);
      return false;
    };
    if (p.stall_test) ok = wait_all(&bar_never, 0, 10);
    for (int wi = w0; wi < w1 && ok; ++wi) {
      const Item it = read_item(a, wi);
      if (it.ntiles == 0) continue;
      if (it.b != q_b) {
        q_b = it.b;
        ok = wait_all(&bar_q, nq & 1, 2);
        ++nq;
      }
      for (int j = 0; j < it.ntiles && ok; ++j)
        for (int kh = 0; kh < a.Hkv && ok; ++kh, ++u) {
          const int buf = u % kBufs;
          if (u >= kBufs) ok = wait_all(&bar_free[buf], (u / kBufs - 1) & 1, 3);
          for (int c = 0; c < p.chunks && ok; ++c) {
            ok = wait_all(&bar_full[s], phase, 4);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t k = dK + ((uint32_t)(s * kChunkBytes) >> 4);
              const uint64_t q = dQ + ((uint32_t)((kh * p.chunks + c) * NT * 128) >> 4);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                if constexpr (F8) mma_ss_f8(tmem + buf * NT, k + ((kk * 32) >> 4), q + ((kk * 32) >> 4), id, c > 0 || kk > 0);
                else mma_ss(tmem + buf * NT, k + ((kk * 32) >> 4), q + ((kk * 32) >> 4), id, c > 0 || kk > 0);
              }
              mma_commit(smem_u32(&bar_empty[s]));
              if (c + 1 == p.chunks) mma_commit(smem_u32(&bar_s[buf]));
            }
            __syncwarp();
            if (++s == p.stages) {
              s = 0;
              phase ^= 1;
            }
          }
        }
    }
    // never free TMEM under a running product
    if (elect_one()) mma_commit(smem_u32(&bar_drain));
    __syncwarp();
    mbar_wait(smem_u32(&bar_drain), 0, 1000000000ull, &zero_flag);
  } else {
    // ------------------------------------------------------------ sums (warps 0-3)
    const int t = threadIdx.x, ncols = a.G * a.s_q;
    const uint32_t lane_addr = tmem + ((uint32_t)(warp * 32) << 16);
    // A warp that gave up walks on without waiting, so that it meets the others at the barriers.
    bool ok = true;
    int u = 0, q_b = -1;
    for (int wi = w0; wi < w1; ++wi) {
      const Item it = read_item(a, wi);
      if (it.ntiles == 0) continue;
      if (it.b != q_b) {
        q_b = it.b;
        // every product of the request before has completed: this warp saw its scores, and
        // past this barrier all four did
        named_bar_sync(1, kSum);
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (long long)it.b * a.s_q * a.Hq * p.D;
        const float* lse = a.lse + (long long)it.b * a.s_q * a.Hq;
        for (int i = t; i < a.Hkv * NP; i += kSum) {
          const int kh = i / NP, n = i % NP;
          float l = INFINITY;
          if (n < ncols) {
            const float x = lse[(n / a.G) * a.Hq + kh * a.G + n % a.G];
            if (x != -INFINITY) l = x * kLog2e;
          }
          sL[i] = l;
        }
        // a warp kBatch query rows (kv head, column) at a time: their loads overlap
        constexpr int kBatch = 8, kPer = 5;  // E4M3: pieces of 4 dims a lane, up to 576
        const int rows = a.Hkv * ncols;
        for (int i0 = warp * kBatch; i0 < rows; i0 += 4 * kBatch) {
          if constexpr (!F8) {
            const int vec = p.D / 8;
            uint4 x[kBatch][3];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int i = min(i0 + k, rows - 1), kh = i / ncols, n = i - kh * ncols;
              const uint4* src = reinterpret_cast<const uint4*>(q + ((long long)(n / a.G) * a.Hq + kh * a.G + n % a.G) * p.D);
#pragma unroll
              for (int c = 0; c < 3; ++c)
                if (lane + 32 * c < vec) x[k][c] = __ldcg(src + lane + 32 * c);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int i = min(i0 + k, rows - 1), kh = i / ncols, n = i - kh * ncols;
              uint8_t* base = sQ + kh * p.chunks * NT * 128 + n * 128;
#pragma unroll
              for (int c = 0; c < 3; ++c) {
                const int e = lane + 32 * c;
                if (e < vec) *reinterpret_cast<uint4*>(base + (e >> 3) * NT * 128 + (((e & 7) ^ (n & 7)) << 4)) = x[k][c];
              }
            }
          } else {
            uint2 x[kBatch][kPer];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int i = min(i0 + k, rows - 1), kh = i / ncols, n = i - kh * ncols;
              const uint2* src = reinterpret_cast<const uint2*>(q + ((long long)(n / a.G) * a.Hq + kh * a.G + n % a.G) * p.D);
#pragma unroll
              for (int c = 0; c < kPer; ++c) x[k][c] = 4 * lane + 128 * c < p.D ? __ldcg(src + lane + 32 * c) : make_uint2(0, 0);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const int i = min(i0 + k, rows - 1), kh = i / ncols, n = i - kh * ncols;
              // magnitudes are ordered like their bits, two bf16 at a time
              uint32_t m = 0;
#pragma unroll
              for (int c = 0; c < kPer; ++c) m = __vmaxu2(m, __vmaxu2(x[k][c].x & 0x7fff7fffu, x[k][c].y & 0x7fff7fffu));
              const uint32_t top = __reduce_max_sync(0xffffffffu, max(m & 0xffff0000u, m << 16));
              // 2^(7 - e) brings a largest element of [2^e, 2^(e+1)) to [128, 256)
              const int e = max(-100, (int)(top >> 23) - 127);
              const float f = __uint_as_float((uint32_t)(7 - e + 127) << 23);
              // an infinite element would become 448: the row's scores are NaN instead
              if (lane == 0) sF[kh * NP + n] = __uint_as_float(e < 128 ? (uint32_t)(e - 7 + 127) << 23 : 0x7fffffffu);
              uint8_t* base = sQ + kh * p.chunks * NT * 128 + 4 * (lane & 3);
#pragma unroll
              for (int c = 0; c < kPer; ++c) {
                if (c >= p.chunks) break;
                uint32_t hi = 0, lo = 0;
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                  const uint32_t b = w ? x[k][c].y : x[k][c].x;
                  const float v0 = __uint_as_float(b << 16) * f, v1 = __uint_as_float(b & 0xffff0000u) * f;
                  const uint32_t h = e4m3x2(v0, v1);
                  float h0, h1;
                  e4m3x2_value(h, h0, h1);
                  hi |= h << (16 * w);
                  lo |= e4m3x2((v0 - h0) * 16.f, (v1 - h1) * 16.f) << (16 * w);
                }
                uint8_t* row = base + c * NT * 128 + (((lane >> 2) ^ (n & 7)) << 4);
                *reinterpret_cast<uint32_t*>(row + n * 128) = hi;
                *reinterpret_cast<uint32_t*>(row + (NP + n) * 128) = lo;
              }
            }
          }
        }
        fence_proxy_async_smem();
        named_bar_sync(1, kSum);
        if (t == 0) mbar_arrive(smem_u32(&bar_q));
      }
      const int lim = it.pd.ctx_len - a.s_q;
      // A tile's pool rows, weights and scales are loaded one tile ahead, their pages two:
      // the chain of the three must not stand between the products and the sums.
      auto page_of = [&](int j) {
        const int i = min(it.row_begin + j * kRows + t, it.pd.rows - 1);
        return j < it.ntiles ? __ldcg(a.rm.table + (long long)it.pair * a.rm.max_pages + i / a.rm.page_size) : 0;
      };
      int page = page_of(0), next_page = page_of(1);
      long long row = 0;
      float before = 0.f, scale = 0.f;
      auto fetch = [&](int j, int pg) {
        const int i = j * kRows + t;
        if (i >= it.nrows) return;
        row = (long long)pg * a.rm.page_size + (it.row_begin + i) % a.rm.page_size;
        before = a.weights[row];
        if (F8) scale = __ldcg(a.scale + row);
      };
      fetch(0, page);
      for (int j = 0; j < it.ntiles; ++j) {
        const int i = j * kRows + t;
        const bool valid = i < it.nrows;
        const long long row_j = row;
        const float before_j = before, c = F8 ? p.scale_log2 * scale : p.scale_log2;
        fetch(j + 1, next_page);
        next_page = page_of(j + 2);
        // several query rows: row qi reads tokens up to L - s_q + qi, so this cache row
        // weighs nothing for the columns n = qi G + i of qi < tok - lim
        const int first = max(0, it.pd.tok0 + (it.row_begin + i) * it.pd.tok_step - lim) * a.G;
        float w = 0.f;
        for (int kh = 0; kh < a.Hkv; ++kh, ++u) {
          const int buf = u % kBufs;
          if (ok) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bar_s[buf]), (u / kBufs) & 1, p.wait_ns, &abort_flag));
            if (!ok) report_timeout(p.status, 5, &abort_flag);
          }
          if (!ok) continue;
          tc_fence_after();
          uint32_t sr[NT];
          tmem_ld_cols<NT>(lane_addr + buf * NT, sr);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bar_free[buf]));
          float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int n0 = 0; n0 < NP; n0 += 4) {
            if (n0 >= ncols) break;
            const float4 l = *reinterpret_cast<const float4*>(sL + kh * NP + n0);
            const float lv[4] = {l.x, l.y, l.z, l.w};
            float fv[4] = {1.f, 1.f, 1.f, 1.f};
            if constexpr (F8) {
              const float4 f = *reinterpret_cast<const float4*>(sF + kh * NP + n0);
              fv[0] = f.x; fv[1] = f.y; fv[2] = f.z; fv[3] = f.w;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int n = n0 + k;
              float x = __uint_as_float(sr[n]);
              if constexpr (F8) x = fmaf(__uint_as_float(sr[NP + n]), 0.0625f, x) * fv[k];
              const float e = ex2(fmaf(x, c, -lv[k]));
              part[k] += n >= first && n < ncols ? e : 0.f;
            }
          }
          w += (part[0] + part[1]) + (part[2] + part[3]);
        }
        if (valid && ok) a.weights[row_j] = before_j + w;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarpMma) tmem_dealloc(tmem, kCols);
}

int padded_cols(int ncols) { return ncols <= 16 ? 16 : ncols <= 32 ? 32 : 64; }

template <int NP, bool F8>
cudaError_t launch_np(const CUtensorMap& map, Params p, int workers, cudaStream_t s) {
  const int q_bytes = p.a.Hkv * p.chunks * (F8 ? 2 * NP : NP) * 128, cols = p.a.Hkv * NP * 8;
  int stages = (kSmemLimit - 1024 - q_bytes - cols) / kChunkBytes;
  p.stages = stages > kMaxStages ? kMaxStages : stages;
  auto kern = decode_weights_tc_kernel<NP, F8>;
  // one limit for all calls: another thread's call may set it at the same time
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e != cudaSuccess) return e;
  return launch_early(kern, (unsigned)workers, kThreads, (size_t)p.stages * kChunkBytes + q_bytes + cols + 1024, s, 1, map, p);
}

}  // namespace

bool decode_weights_tc_supported(cp_dtype kv, int Hkv, int G, int s_q, int D) {
  if (kv == CP_BF16 ? (D != 64 && D != 128 && D != 576) : (kv != CP_FP8_E4M3 || (D != 128 && D != 576))) return false;
  if (G * s_q > 64) return false;
  const bool f8 = kv == CP_FP8_E4M3;
  const int chunks = f8 ? (D + 127) / 128 : D / 64;
  return Hkv * chunks * padded_cols(G * s_q) * (f8 ? 2 : 1) * 128 <= kMaxQBytes;
}

cudaError_t launch_decode_weights_tc(const DecodeWeightsArgs& a, cp_dtype kv, int D, int workers, bool stall_test, cudaStream_t s) {
  const bool f8 = kv == CP_FP8_E4M3;
  Params p = {a, D, f8 ? (D + 127) / 128 : D / 64, 0, a.sm_scale * kLog2e, device_status_ptr(),
              stall_test ? 50000000ull : wait_limit_ns(), stall_test ? 1 : 0};
  if (!p.status) return cudaErrorInvalidDevice;
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.Hkv, (uint64_t)a.rm.pool_rows};
  const uint64_t es = f8 ? 1 : 2, strides[2] = {D * es, (uint64_t)a.Hkv * D * es};
  const uint32_t box[3] = {f8 ? 128u : 64u, 1, 64};
  if (!(f8 ? encode_tensor_map_u8_3d(&map, a.k, dims, strides, box) : encode_tensor_map_bf16(&map, a.k, 3, dims, strides, box)))
    return cudaErrorInvalidValue;
  switch (padded_cols(a.G * a.s_q)) {
    case 16: return f8 ? launch_np<16, true>(map, p, workers, s) : launch_np<16, false>(map, p, workers, s);
    case 32: return f8 ? launch_np<32, true>(map, p, workers, s) : launch_np<32, false>(map, p, workers, s);
    default: return f8 ? launch_np<64, true>(map, p, workers, s) : launch_np<64, false>(map, p, workers, s);
  }
}

}  // namespace cpattn

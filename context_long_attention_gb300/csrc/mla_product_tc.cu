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
//   warp 0     TMA producer: stages of the tokens' [128 x 64] and the
//              weight's [NB x 64] pieces (absorb: the whole K = 128 in one
//              stage; its weight is read as an MN-major operand, so one
//              layout of W serves all three)
//   warp 1     MMA issuer and TMEM owner, two accumulators of NB columns
//   warps 4-7  epilogue: a thread per token row
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "tc_ptx.cuh"

namespace cpattn {
namespace {
using namespace tc;

constexpr int BM = 128;  // tokens per item
constexpr int kLatent = 512;
constexpr int kHeadRows = 256;  // W rows per head
constexpr int kKeyDims = 128;   // W rows of the key part; the value part follows
constexpr int kRope = 64;
constexpr int kThreads = 256;

enum Mode { kExpand = 0, kAbsorb = 1, kProject = 2 };

template <int MODE, int NB>
struct Cfg {
  static constexpr int kN = MODE == kExpand ? kHeadRows : MODE == kAbsorb ? kLatent : kKeyDims;  // columns per head
  static constexpr int kK = MODE == kAbsorb ? kKeyDims : kLatent;
  static constexpr int kNBlocks = kN / NB;
  static constexpr int kStageK = MODE == kAbsorb ? kKeyDims : 64;
  static constexpr int kIters = kK / kStageK;
  static constexpr int kABytes = BM * kStageK * 2;
  static constexpr int kBBytes = NB * kStageK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStageBytes > 6 ? 6 : 196608 / kStageBytes;
  static constexpr int kSmem = kStages * kStageBytes + 1024;
  static constexpr int kTmemCols = 2 * NB < 32 ? 32 : 2 * NB;
};

struct Params {
  int H;
  int n_items;  // token tiles x heads x column blocks
  int n_tokens;
  __nv_bfloat16* out;
  const __nv_bfloat16* q;  // absorb: the rotated part's source
  unsigned* status;
  unsigned long long wait_ns;
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

template <int MODE, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    mla_product_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap wmap,
                       const Params p) {
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
      mbar_init(smem_u32(&bar_empty[s]), 1);
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
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  auto wait_all = [&](uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, p.wait_ns, &abort_flag));
  };

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    int g = 0;  // stages filled so far
    bool ok = true;
    for (int i = blockIdx.x; i < p.n_items && ok; i += gridDim.x) {
      const Item it = item_of<C>(i, p.H);
      for (int k = 0; k < C::kIters && ok; ++k, ++g) {
        const int s = g % C::kStages;
        if (g >= C::kStages) ok = wait_all(smem_u32(&bar_empty[s]), (g / C::kStages - 1) & 1);
        if (!ok) break;
        if (elect_one()) {
          const uint32_t full = smem_u32(&bar_full[s]);
          const uint32_t a = smem_u32(smem + s * C::kStageBytes), b = a + C::kABytes;
          mbar_expect_tx(full, C::kStageBytes);
          if (MODE == kExpand) {
            tma_load_2d(a, &amap, k * 64, it.tile * BM, full);
          } else {
#pragma unroll
            for (int c = 0; c < C::kStageK / 64; ++c)
              tma_load_3d(a + c * (BM * 128), &amap, k * C::kStageK + c * 64, it.h, it.tile * BM, full);
          }
          if (MODE == kAbsorb) {  // [128 key dims x 64 latent columns] pieces
#pragma unroll
            for (int c = 0; c < NB / 64; ++c)
              tma_load_2d(b + c * (kKeyDims * 128), &wmap, it.nb * NB + c * 64, it.h * kHeadRows, full);
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
        const uint64_t db = MODE == kAbsorb ? smem_desc(b, kKeyDims * 128, 1024) : smem_desc(b, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < C::kStageK / 16; ++kk) {
            const uint32_t oa = ((kk >> 2) * (BM * 128) + (kk & 3) * 32) >> 4;
            const uint32_t ob = MODE == kAbsorb ? (kk * 16 * 128) >> 4 : ((kk & 3) * 32) >> 4;
            mma_ss(tmem + acc * NB, da + oa, db + ob, id, (k > 0 || kk > 0) ? 1u : 0u);
          }
          mma_commit(smem_u32(&bar_empty[s]));
          if (k == C::kIters - 1) mma_commit(smem_u32(&bar_acc[acc]));
        }
        __syncwarp();
      }
    }
    if (bad && lane == 0) report_timeout(p.status, bad, &abort_flag);
    if (elect_one()) mma_commit(smem_u32(&bar_drain));
    __syncwarp();
    mbar_wait(smem_u32(&bar_drain), 0, 1000000000ull, &zero_flag);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_addr = tmem + ((uint32_t)(quarter * 32) << 16);
    int n = 0;
    for (int i = blockIdx.x; i < p.n_items; i += gridDim.x, ++n) {
      const Item it = item_of<C>(i, p.H);
      const int acc = n & 1;
      const long long tok = (long long)it.tile * BM + row;
      const bool valid = tok < p.n_tokens;
      constexpr int ld = MODE == kExpand ? kHeadRows : MODE == kAbsorb ? kLatent + kRope : kKeyDims;
      __nv_bfloat16* dst = p.out + (tok * p.H + it.h) * ld + it.nb * NB;
      if (MODE == kAbsorb && it.nb == 0 && valid) {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (tok * p.H + it.h) * (kKeyDims + kRope) + kKeyDims);
        uint4* d = reinterpret_cast<uint4*>(dst + kLatent);
#pragma unroll
        for (int c = 0; c < kRope / 8; ++c) d[c] = __ldg(src + c);
      }
      if (!wait_all(smem_u32(&bar_acc[acc]), (n / 2) & 1)) {
        if (lane == 0) report_timeout(p.status, 4, &abort_flag);
        break;
      }
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < NB / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(lane_addr + acc * NB + c * 32, r);
        tmem_ld_wait();
        if (valid) {
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(r[8 * v4 + 0]), __uint_as_float(r[8 * v4 + 1]));
            w.y = pack_bf16x2(__uint_as_float(r[8 * v4 + 2]), __uint_as_float(r[8 * v4 + 3]));
            w.z = pack_bf16x2(__uint_as_float(r[8 * v4 + 4]), __uint_as_float(r[8 * v4 + 5]));
            w.w = pack_bf16x2(__uint_as_float(r[8 * v4 + 6]), __uint_as_float(r[8 * v4 + 7]));
            reinterpret_cast<uint4*>(dst + c * 32)[v4] = w;
          }
        }
      }
      tc_fence_before();
      mbar_arrive(smem_u32(&bar_free[acc]));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <int MODE, int NB>
cudaError_t launch(const CUtensorMap& am, const CUtensorMap& wm, Params p, int sms, cudaStream_t s) {
  using C = Cfg<MODE, NB>;
  const long long items = (long long)((p.n_tokens + BM - 1) / BM) * p.H * C::kNBlocks;
  if (items > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  p.n_items = (int)items;
  cudaError_t e = cudaFuncSetAttribute(mla_product_kernel<MODE, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = (int)(items < sms ? items : sms);
  mla_product_kernel<MODE, NB><<<grid, kThreads, C::kSmem, s>>>(am, wm, p);
  return cudaGetLastError();
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

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  return n;
}

}  // namespace

cudaError_t launch_mla_expand(const void* latent, long long stride, const void* w, int T, int H, void* kv,
                              cudaStream_t s) {
  Params p = {H, 0, T, static_cast<__nv_bfloat16*>(kv), nullptr, device_status_ptr(), wait_limit_ns()};
  const int sms = sm_count();
  if (!p.status || !sms) return cudaErrorInvalidDevice;
  CUtensorMap am, wm;
  const uint64_t dims[2] = {kLatent, (uint64_t)T};
  const uint64_t strides[1] = {(uint64_t)stride * 2};
  const uint32_t box[2] = {64, BM};
  if (!encode_tensor_map_bf16(&am, latent, 2, dims, strides, box)) return cudaErrorInvalidValue;
  if (!weight_map(&wm, w, H, 256)) return cudaErrorInvalidValue;
  return launch<kExpand, 256>(am, wm, p, sms, s);
}

cudaError_t launch_mla_absorb(const void* q, const void* w, int n, int H, void* ql, cudaStream_t s) {
  Params p = {H, 0, n, static_cast<__nv_bfloat16*>(ql), static_cast<const __nv_bfloat16*>(q), device_status_ptr(),
              wait_limit_ns()};
  const int sms = sm_count();
  if (!p.status || !sms) return cudaErrorInvalidDevice;
  CUtensorMap am, wm;
  if (!token_map(&am, q, n, H, kKeyDims + kRope) || !weight_map(&wm, w, H, kKeyDims)) return cudaErrorInvalidValue;
  return launch<kAbsorb, 256>(am, wm, p, sms, s);
}

cudaError_t launch_mla_project(const void* ol, const void* w, int n, int H, void* o, cudaStream_t s) {
  Params p = {H, 0, n, static_cast<__nv_bfloat16*>(o), nullptr, device_status_ptr(), wait_limit_ns()};
  const int sms = sm_count();
  if (!p.status || !sms) return cudaErrorInvalidDevice;
  CUtensorMap am, wm;
  if (!token_map(&am, ol, n, H, kLatent) || !weight_map(&wm, w, H, 128)) return cudaErrorInvalidValue;
  return launch<kProject, 128>(am, wm, p, sms, s);
}

}  // namespace cpattn

// The per-head products of latent attention for a handful of tokens, on the
// CUDA cores (bf16 in, fp32 products and sums, one rounding to bf16).
//
//   absorb   ql[n, h, 0:512] = W[h, 0:128]^T q[n, h, 0:128];  ql[n, h, 512:576] = q[n, h, 128:192]
//   project  o[n, h, :]      = W[h, 128:256] ol[n, h, :]
//
// With one to four tokens the call is its weight's read (131 KB a head) behind
// a chain of latencies, which these kernels keep short: no tensor maps, no
// tensor memory, every weight load in flight at once, one barrier.  In a
// replayed graph, against the tensor-core kernels (us, absorb / project):
//   64 heads   1 token 2.2 / 1.9 and 5.1 / 4.7   4 tokens 4.9 / 3.3 and 4.5 / 4.8   8 tokens 7.3 / 4.6 and 3.9 / 4.8
//   8 heads    1 token 1.5 / 1.5 and 3.1 / 4.5   4 tokens 2.6 / 2.2 and 3.1 / 4.5   8 tokens 3.9 / 2.9 and 3.1 / 4.5
// so they take up to four (one token over 64 heads reads its 8.4 MB of weight at 3.8 TB/s, launch included).
#include <cuda_bf16.h>

#include "early_launch.cuh"
#include "internal.h"

namespace cpattn {
namespace {

constexpr int kLatent = 512, kHeadRows = 256, kKeyDims = 128, kRope = 64;
constexpr int kThreads = 256;
constexpr int kCols = 128;  // absorb: latent columns a block
constexpr int kRows = 32;   // project: value dims a block

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
  x[0] = lo(w.x), x[1] = hi(w.x), x[2] = lo(w.y), x[3] = hi(w.y);
  x[4] = lo(w.z), x[5] = hi(w.z), x[6] = lo(w.w), x[7] = hi(w.w);
}

// A block: one head's 128 key dims x 128 latent columns.  Sixteen threads take
// a row's 128 columns (8 each), so a thread has 8 columns of 8 rows; the rows
// are summed over the two halves of a warp and then over the warps.
template <int NT>
__global__ void __launch_bounds__(kThreads) absorb_small_kernel(const __nv_bfloat16* q, const __nv_bfloat16* w,
                                                                __nv_bfloat16* out, int n, int H) {
  __shared__ float sq[NT][kKeyDims];
  __shared__ float red[kThreads / 32][NT][kCols];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x / (kLatent / kCols), col0 = blockIdx.x % (kLatent / kCols) * kCols;
  const int cl = tid & 15, row0 = (tid >> 4) * 8;
  const __nv_bfloat16* src = w + ((long long)h * kHeadRows + row0) * kLatent + col0 + cl * 8;
  wait_for_earlier_kernels();
  uint4 wv[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) wv[j] = __ldcg(reinterpret_cast<const uint4*>(src + j * kLatent));
  for (int i = tid; i < NT * kKeyDims; i += kThreads) {
    const int t = i / kKeyDims, d = i % kKeyDims;
    sq[t][d] = t < n ? __bfloat162float(q[((long long)t * H + h) * (kKeyDims + kRope) + d]) : 0.f;
  }
  if (col0 == 0 && tid < n * (kRope / 8)) {  // the rotated part
    const int t = tid / (kRope / 8), c = tid % (kRope / 8);
    reinterpret_cast<uint4*>(out + ((long long)t * H + h) * (kLatent + kRope) + kLatent)[c] =
        __ldcg(reinterpret_cast<const uint4*>(q + ((long long)t * H + h) * (kKeyDims + kRope) + kKeyDims) + c);
  }
  __syncthreads();
  float acc[NT][8];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[t][e] = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float x[8];
    unpack(wv[j], x);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const float qv = sq[t][row0 + j];
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[t][e] = fmaf(qv, x[e], acc[t][e]);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      acc[t][e] += __shfl_xor_sync(0xffffffffu, acc[t][e], 16);
      if (lane < 16) red[warp][t][cl * 8 + e] = acc[t][e];
    }
  __syncthreads();
  for (int i = tid; i < NT * kCols / 2; i += kThreads) {
    const int t = i / (kCols / 2), c = 2 * (i % (kCols / 2));
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
      a += red[k][t][c];
      b += red[k][t][c + 1];
    }
    if (t < n)
      *reinterpret_cast<__nv_bfloat162*>(out + ((long long)t * H + h) * (kLatent + kRope) + col0 + c) =
          __floats2bfloat162_rn(a, b);
  }
}

// A block: one head's 32 value dims, four a warp; a lane has 16 of a row's 512
// latent columns.
template <int NT>
__global__ void __launch_bounds__(kThreads) project_small_kernel(const __nv_bfloat16* ol, const __nv_bfloat16* w,
                                                                 __nv_bfloat16* out, int n, int H) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x / (kKeyDims / kRows), row0 = blockIdx.x % (kKeyDims / kRows) * kRows + warp * 4;
  const __nv_bfloat16* src = w + ((long long)h * kHeadRows + kKeyDims + row0) * kLatent + lane * 8;
  wait_for_earlier_kernels();
  uint4 wv[4][2];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) wv[j][k] = __ldcg(reinterpret_cast<const uint4*>(src + j * kLatent + k * 256));
  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    uint4 xv[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      xv[k] = t < n ? __ldcg(reinterpret_cast<const uint4*>(ol + ((long long)t * H + h) * kLatent + lane * 8 + k * 256))
                    : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[t][j] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float x[8];
      unpack(xv[k], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float y[8];
        unpack(wv[j][k], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[t][j] = fmaf(x[e], y[e], acc[t][j]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) acc[t][j] += __shfl_xor_sync(0xffffffffu, acc[t][j], d);
    if (lane == t && t < n) {
      __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(out + ((long long)t * H + h) * kKeyDims + row0);
      dst[0] = __floats2bfloat162_rn(acc[t][0], acc[t][1]);
      dst[1] = __floats2bfloat162_rn(acc[t][2], acc[t][3]);
    }
  }
}

}  // namespace

cudaError_t launch_mla_absorb_small(const void* q, const void* w, int n, int H, void* ql, cudaStream_t s) {
  const unsigned grid = (unsigned)H * (kLatent / kCols);
  auto kern = n == 1 ? absorb_small_kernel<1> : n == 2 ? absorb_small_kernel<2> : absorb_small_kernel<kMlaSmall>;
  return launch_early(kern, grid, kThreads, 0, s, 1, static_cast<const __nv_bfloat16*>(q),
                      static_cast<const __nv_bfloat16*>(w), static_cast<__nv_bfloat16*>(ql), n, H);
}

cudaError_t launch_mla_project_small(const void* ol, const void* w, int n, int H, void* o, cudaStream_t s) {
  const unsigned grid = (unsigned)H * (kKeyDims / kRows);
  auto kern = n == 1 ? project_small_kernel<1> : n == 2 ? project_small_kernel<2> : project_small_kernel<kMlaSmall>;
  return launch_early(kern, grid, kThreads, 0, s, 1, static_cast<const __nv_bfloat16*>(ol),
                      static_cast<const __nv_bfloat16*>(w), static_cast<__nv_bfloat16*>(o), n, H);
}

}  // namespace cpattn

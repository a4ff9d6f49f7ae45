// The attention weight that cached tokens received: for key j
//   w_j = sum over queries i that read j and heads h of exp(sm_scale q_ih . k_jg - LSE_ih)
// (CUDA-core forms: every shape that the tensor-core kernels do not take).
//
// The LSE is the attention's own, so a weight is the softmax probability itself
// and no second pass over the keys is needed; keys are the rows of the work and
// a key's sum stays with one thread or warp, so no sum is made by atomics.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "internal.h"
#include "plan_rows.cuh"

namespace cpattn {
namespace {

__device__ __forceinline__ float ld_elem(const float* p, long long i) { return p[i]; }
__device__ __forceinline__ float ld_elem(const __nv_bfloat16* p, long long i) { return __bfloat162float(p[i]); }
__device__ __forceinline__ float ld_elem(const __nv_fp8_e4m3* p, long long i) { return float(p[i]); }

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
// exp(s - LSE); a query without keys (LSE = -inf) weighs nothing
__device__ __forceinline__ float weight(float s, float lse) { return lse == -INFINITY ? 0.f : expf(s - lse); }

constexpr int kWarps = 4;

// A warp a key row of the prompt; lane l holds its dims l, l + 32, ...
template <typename T, int ND>
__global__ void __launch_bounds__(kWarps * 32) prefill_weights_simt_kernel(const PrefillWeightsArgs a) {
  constexpr int D = ND * 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= a.rows.KV) return;
  const cp_req_desc* reqs = reinterpret_cast<const cp_req_desc*>(a.rows.plan + a.rows.off_req);
  int lo = 0, hi = a.rows.R - 1;  // the last request whose first row is at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (reqs[mid].kv_base <= row) lo = mid; else hi = mid - 1;
  }
  const cp_req_desc rq = reqs[lo];
  const int key = (int)(row - rq.kv_base);
  const int first = max(a.window ? max(0, rq.new_len - a.window) : 0, key - rq.prefix_len);
  float w = 0.f;
  for (int g = 0; g < a.Hkv; ++g) {
    float kv[ND];
#pragma unroll
    for (int e = 0; e < ND; ++e) kv[e] = ld_elem(static_cast<const T*>(a.k), (row * a.Hkv + g) * D + lane + 32 * e);
    // sums of 128 queries each: a sum of all of them one after another would lose
    // bits of a heavy key's weight
    for (int i0 = first; i0 < rq.new_len; i0 += 128) {
      float sum = 0.f;
      for (int i = i0; i < min(i0 + 128, rq.new_len); ++i) {
        const long long f = rq.q_base + i, out = plan_row(a.rows, lo, rq, i);
        for (int h = g * a.G; h < (g + 1) * a.G; ++h) {
          float part = 0.f;
#pragma unroll
          for (int e = 0; e < ND; ++e) part += kv[e] * ld_elem(static_cast<const T*>(a.q), (f * a.Hq + h) * D + lane + 32 * e);
          sum += weight(a.sm_scale * warp_sum(part), a.lse[out * a.Hq + h]);
        }
      }
      w += sum;
    }
  }
  if (lane == 0) a.out[row] = w;
}

// A warp a row of a decode work item.
template <typename TQ, typename T, int ND>
__global__ void __launch_bounds__(kWarps * 32) decode_weights_simt_kernel(const DecodeWeightsArgs a) {
  constexpr int D = ND * 32;
  const int lane = threadIdx.x & 31;
  const cp_pair_desc* pairs = reinterpret_cast<const cp_pair_desc*>(a.plan + a.off_pair);
  const cp_work_desc* work = reinterpret_cast<const cp_work_desc*>(a.plan + a.off_work);
  for (int wi = a.plan[a.off_worker + blockIdx.x]; wi < a.plan[a.off_worker + blockIdx.x + 1]; ++wi) {
    const cp_work_desc wd = work[wi];
    const cp_pair_desc pd = pairs[wd.pair];
    const int b = wd.pair % a.B;
    for (int i = wd.row_begin + blockIdx.y * kWarps + (threadIdx.x >> 5); i < wd.row_end; i += gridDim.y * kWarps) {
      const long long row = map_row(a.rm, wd.pair, 0, i);
      const int tok = pd.tok0 + i * pd.tok_step;
      const float rs = a.scale ? a.scale[row] : 1.f;
      float w = 0.f;
      for (int g = 0; g < a.Hkv; ++g) {
        float kv[ND];
#pragma unroll
        for (int e = 0; e < ND; ++e) kv[e] = ld_elem(static_cast<const T*>(a.k), (row * a.Hkv + g) * D + lane + 32 * e);
        // query row qi reads the tokens up to L - s_q + qi
        for (int qi = max(0, tok - (pd.ctx_len - a.s_q)); qi < a.s_q; ++qi)
          for (int h = g * a.G; h < (g + 1) * a.G; ++h) {
            const long long n = ((long long)b * a.s_q + qi) * a.Hq + h;
            float part = 0.f;
#pragma unroll
            for (int e = 0; e < ND; ++e) part += kv[e] * ld_elem(static_cast<const TQ*>(a.q), n * D + lane + 32 * e);
            w += weight(a.sm_scale * rs * warp_sum(part), a.lse[n]);
          }
      }
      if (lane == 0) a.weights[row] += w;
    }
  }
}

template <typename TQ, typename T>
cudaError_t decode_t(const DecodeWeightsArgs& a, int D, int workers, cudaStream_t s) {
  auto run = [&](auto kern) {
    kern<<<dim3(workers, 16), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
  };
  switch (D / 32) {
    case 1: return run(decode_weights_simt_kernel<TQ, T, 1>);
    case 2: return run(decode_weights_simt_kernel<TQ, T, 2>);
    case 3: return run(decode_weights_simt_kernel<TQ, T, 3>);
    case 4: return run(decode_weights_simt_kernel<TQ, T, 4>);
    case 5: return run(decode_weights_simt_kernel<TQ, T, 5>);
    case 6: return run(decode_weights_simt_kernel<TQ, T, 6>);
    case 7: return run(decode_weights_simt_kernel<TQ, T, 7>);
    case 8: return run(decode_weights_simt_kernel<TQ, T, 8>);
    case 18: return run(decode_weights_simt_kernel<TQ, T, 18>);
    default: return cudaErrorInvalidValue;
  }
}

template <typename T>
cudaError_t prefill_t(const PrefillWeightsArgs& a, int D, cudaStream_t s) {
  auto run = [&](auto kern) {
    kern<<<(unsigned)(((long long)a.rows.KV + kWarps - 1) / kWarps), kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
  };
  switch (D / 32) {
    case 1: return run(prefill_weights_simt_kernel<T, 1>);
    case 2: return run(prefill_weights_simt_kernel<T, 2>);
    case 3: return run(prefill_weights_simt_kernel<T, 3>);
    case 4: return run(prefill_weights_simt_kernel<T, 4>);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_prefill_weights_simt(const PrefillWeightsArgs& a, int D, cudaStream_t s) { return prefill_t<float>(a, D, s); }

cudaError_t launch_decode_weights_simt(const DecodeWeightsArgs& a, cp_dtype kv, int D, int workers, cudaStream_t s) {
  switch (kv) {
    case CP_BF16: return decode_t<__nv_bfloat16, __nv_bfloat16>(a, D, workers, s);
    case CP_FP32: return decode_t<float, float>(a, D, workers, s);
    default: return decode_t<__nv_bfloat16, __nv_fp8_e4m3>(a, D, workers, s);
  }
}

}  // namespace cpattn

// Attention of groups of queries over the prefix that each group shares: the
// CUDA-core form and the merge of the parts.  (bf16 and FP8 caches at the usual
// head dims run on the tensor cores, prefix_tc.cu.)
//
// The query rows of a group and the G = Hq / Hkv heads of a kv head are the rows
// m = n G + i of one attention over the group's keys, in blocks of 256.  The plan
// cuts the (block, key tile) walk evenly over the workers; a block cut between
// workers, or joined with the partial results of the queries' own tokens, goes
// through parts in the workspace, combined exactly by log-sum-exp ("How GPUs
// Share a Long Context During LLM Inference" §3.3).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "early_launch.cuh"
#include "internal.h"

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

// A warp a row m, lane l holding dims l, l + 32, ...: every shape that the tensor
// cores do not take (fp32, other head dims).
constexpr int kSimtWarps = 4;
template <typename TQ, typename T, int ND>
__global__ void __launch_bounds__(kSimtWarps * 32) prefix_simt_kernel(const PrefixArgs a) {
  constexpr int D = ND * 32;
  const int lane = threadIdx.x & 31, dm = blockIdx.y * kSimtWarps + (threadIdx.x >> 5);
  const TQ* q = static_cast<const TQ*>(a.q);
  for (int wi = a.plan[a.off_worker + blockIdx.x]; wi < a.plan[a.off_worker + blockIdx.x + 1]; ++wi) {
    const cp_prefix_item it = reinterpret_cast<const cp_prefix_item*>(a.plan + a.off_item)[wi];
    if (dm >= it.m_rows) continue;
    const int m = it.m0 + dm, head = it.kv_head * a.G + m % a.G;
    const long long n = it.row0 + m / a.G;
    float qv[ND], acc[ND], mx = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < ND; ++e) {
      qv[e] = ld_elem(q, (n * a.Hq + head) * D + lane + 32 * e);
      acc[e] = 0.f;
    }
    const int32_t* tile_off = a.plan + a.off_tiles + it.group * (a.C + 1);
    for (int r = 0; r < a.C; ++r) {
      const int t0 = max(it.tile_begin, tile_off[r]) - tile_off[r], t1 = min(it.tile_end, tile_off[r + 1]) - tile_off[r];
      const int pair = r * a.R + it.group;
      const cp_pair_desc pd = reinterpret_cast<const cp_pair_desc*>(a.plan + a.off_pair)[pair];
      const T* kb = static_cast<const T*>(a.k.p[r]);
      const T* vb = static_cast<const T*>(a.v.p[r]);
      const float* scr = a.sc.p[r];
      for (int row = t0 * kDecodeTileRows; row < min(pd.rows, t1 * kDecodeTileRows); ++row) {
        const long long cr = map_row(a.rm, pair, pd.row_off, row);
        const long long kr = (cr * a.Hkv + it.kv_head) * D + lane;
        const float rs = scr ? scr[cr] : 1.f;
        float part = 0.f, vv[ND];
#pragma unroll
        for (int e = 0; e < ND; ++e) {
          part += qv[e] * ld_elem(kb, kr + 32 * e);
          vv[e] = ld_elem(vb, kr + 32 * e) * rs;
        }
        const float s = a.sm_scale * rs * warp_sum(part);
        const float mn = fmaxf(mx, s), corr = expf(mx - mn), p = expf(s - mn);
        l = l * corr + p;
#pragma unroll
        for (int e = 0; e < ND; ++e) acc[e] = acc[e] * corr + p * vv[e];
        mx = mn;
      }
    }
    const float inv = 1.f / l, lse = mx + logf(l);
    if (it.alone && !a.P) {
      const long long at = n * a.Hq + head;
#pragma unroll
      for (int e = 0; e < ND; ++e) {
        const long long i = at * D + lane + 32 * e;
        if (a.o_bf16) static_cast<__nv_bfloat16*>(a.o)[i] = __float2bfloat16_rn(acc[e] * inv);
        else static_cast<float*>(a.o)[i] = acc[e] * inv;
      }
      if (lane == 0) a.lse[at] = lse;
    } else {
      const long long at = (long long)it.part * kPrefixRows + dm;
#pragma unroll
      for (int e = 0; e < ND; ++e) a.ws_o[at * D + lane + 32 * e] = acc[e] * inv;
      if (lane == 0) a.ws_lse[at] = lse;
    }
  }
}

// ------------------------------------------------------------------ merge

// A warp an output row: the weights of its parts, one to a lane, then its dims over
// the lanes, NV pieces of four to a lane; kBatch parts' rows are loaded together.
constexpr int kMergeWarps = 8;
template <int NV, int kBatch>
__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const PrefixArgs a) {
  constexpr int kPer = kPrefixRows / kMergeWarps;
  const int lane = threadIdx.x & 31, dm = (blockIdx.x % kPer) * kMergeWarps + (threadIdx.x >> 5);
  // the plan comes by copies, never from a kernel: it is there before the kernel before this one ends
  const cp_prefix_block bl = reinterpret_cast<const cp_prefix_block*>(a.plan + a.off_block)[blockIdx.x / kPer];
  wait_for_earlier_kernels();
  if (dm >= bl.m_rows) return;
  const int m = bl.m0 + dm, head = bl.kv_head * a.G + m % a.G;
  const long long at = (long long)(bl.row0 + m / a.G) * a.Hq + head, NH = (long long)a.N * a.Hq;
  const int parts = bl.n_parts + a.P;
  // part i: the block's own parts, then the caller's
  auto lse_at = [&](int i) {
    return i < bl.n_parts ? __ldcg(a.ws_lse + (long long)(bl.first_part + i) * kPrefixRows + dm) : __ldcg(a.own_lse + (i - bl.n_parts) * NH + at);
  };
  float g = -INFINITY;
  for (int i = lane; i < parts; i += 32) g = fmaxf(g, lse_at(i));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, d));
  const float g0 = g == -INFINITY ? 0.f : g;
  float4 acc[NV];
#pragma unroll
  for (int c = 0; c < NV; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
  const int vec = a.D / 4;
  for (int i0 = 0; i0 < parts; i0 += 32) {
    const float w = i0 + lane < parts ? expf(lse_at(i0 + lane) - g0) : 0.f;
    const int n = min(32, parts - i0);
    for (int k0 = 0; k0 < n; k0 += kBatch) {
      float wk[kBatch];
      float4 x[kBatch][NV];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        wk[k] = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
        if (k0 + k >= n) wk[k] = 0.f;
        const int i = i0 + k0 + k;
        const float4* row = reinterpret_cast<const float4*>(
            i < bl.n_parts ? a.ws_o + ((long long)(bl.first_part + i) * kPrefixRows + dm) * a.D : a.own_o + ((i - bl.n_parts) * NH + at) * a.D);
#pragma unroll
        for (int c = 0; c < NV; ++c)  // an empty part's row is not read
          x[k][c] = wk[k] != 0.f && lane + 32 * c < vec ? __ldcg(row + lane + 32 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        z += wk[k];
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          acc[c].x += wk[k] * x[k][c].x;
          acc[c].y += wk[k] * x[k][c].y;
          acc[c].z += wk[k] * x[k][c].z;
          acc[c].w += wk[k] * x[k][c].w;
        }
      }
    }
  }
  const float inv = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int d = 4 * (lane + 32 * c);
    if (d >= a.D) continue;
    const float x = acc[c].x * inv, y = acc[c].y * inv, u = acc[c].z * inv, v = acc[c].w * inv;
    if (a.o_bf16) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(x, y), hi = __floats2bfloat162_rn(u, v);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.o) + at * a.D + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(a.o) + at * a.D + d) = make_float4(x, y, u, v);
    }
  }
  if (lane == 0) a.lse[at] = z == 0.f ? -INFINITY : g + logf(z);  // NaN stays NaN
}

template <typename TQ, typename T>
cudaError_t simt_t(const PrefixArgs& a, int workers, cudaStream_t s) {
  const dim3 grid(workers, kPrefixRows / kSimtWarps);
  auto run = [&](auto kern) {
    kern<<<grid, kSimtWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
  };
  switch (a.D / 32) {
    case 1: return run(prefix_simt_kernel<TQ, T, 1>);
    case 2: return run(prefix_simt_kernel<TQ, T, 2>);
    case 3: return run(prefix_simt_kernel<TQ, T, 3>);
    case 4: return run(prefix_simt_kernel<TQ, T, 4>);
    case 5: return run(prefix_simt_kernel<TQ, T, 5>);
    case 6: return run(prefix_simt_kernel<TQ, T, 6>);
    case 7: return run(prefix_simt_kernel<TQ, T, 7>);
    case 8: return run(prefix_simt_kernel<TQ, T, 8>);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_prefix_simt(const PrefixArgs& a, cp_dtype kv, int workers, cudaStream_t s) {
  switch (kv) {
    case CP_BF16: return simt_t<__nv_bfloat16, __nv_bfloat16>(a, workers, s);
    case CP_FP32: return simt_t<float, float>(a, workers, s);
    default: return simt_t<__nv_bfloat16, __nv_fp8_e4m3>(a, workers, s);
  }
}

cudaError_t launch_prefix_merge(const PrefixArgs& a, int blocks, cudaStream_t s) {
  if (blocks == 0) return cudaSuccess;
  const unsigned grid = (unsigned)blocks * (kPrefixRows / kMergeWarps);
  // Few blocks: all the parts that a block of 152 workers usually has at once (4 requests
  // behind 4,096 tokens 20.1 -> 18.5 us, 64 behind 32,768 53.1 -> 51.4); in several waves
  // the registers of 20 would cost the warps that hide the latency (124 -> 130 us for 300 x 64 heads).
  auto kern = a.D > 128 ? prefix_merge_kernel<2, 8> : grid <= 2 * 152 ? prefix_merge_kernel<1, 20> : prefix_merge_kernel<1, 12>;
  return launch_early(kern, grid, kMergeWarps * 32, 0, s, 1, a);
}

}  // namespace cpattn

// The rank-major output row of a prompt's query, from a prefill plan's segments.
#pragma once

#include "internal.h"

namespace cpattn {

// What plan_row needs of a prefill plan.
struct PlanRows {
  const int32_t* plan;
  int off_req, off_seg;
  int C, R, T, KV;
  int zigzag;
};

struct PrefillWeightsArgs {
  PlanRows rows;
  const void *q, *k;      // [T][Hq][D], [KV][Hkv][D]
  const float* lse;       // [T][Hq], rank-major
  float* out;             // [KV]
  int Hq, Hkv, G, window;
  float sm_scale;
};

// On the tensor cores (prefill_weights_tc.cu): bf16, head dim 64 or 128.
size_t prefill_weights_tc_bytes(const int32_t* host_plan, const cp_plan_header& h, int Hq, int window);
cudaError_t launch_prefill_weights_tc(const PrefillWeightsArgs& a, const int32_t* host_plan, const cp_plan_header& h, int D,
                                      void* ws, bool stall_test, cudaStream_t s);

#ifdef __CUDACC__
// Row of query i (of rq.new_len) of request j.  Segments go by rank, then
// request; a zigzag rank has two blocks of every request (early, late).
__device__ __forceinline__ int plan_row(const PlanRows& p, int j, const cp_req_desc& rq, int i) {
  const cp_seg_desc* seg = reinterpret_cast<const cp_seg_desc*>(p.plan + p.off_seg);
  if (p.zigzag) {
    const int nb = 2 * p.C, size = rq.new_len / nb, extra = rq.new_len - size * nb;
    const int split = extra * (size + 1);  // queries in the blocks that are one longer
    const int b = i < split ? i / (size + 1) : extra + (i - split) / size;
    const int start = b * size + min(b, extra);
    const int rank = min(b, nb - 1 - b), which = b < p.C ? 0 : 1;
    return seg[((long long)rank * p.R + j) * 2 + which].local_start + i - start;
  }
  const int f = rq.q_base + i, rank = f % p.C;
  const cp_seg_desc& s = seg[(long long)rank * p.R + j];
  return s.local_start + (f - s.first_f) / p.C;
}
#endif

}  // namespace cpattn

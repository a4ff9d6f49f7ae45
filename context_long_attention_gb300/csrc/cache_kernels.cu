// Pages, slots and new tokens of a paged token-sharded decode cache.
//
// * page_slots_kernel: from request lengths on the GPU, the pages that a
//   step's new tokens need (into the page table) and every new token's pool
//   row ("How GPUs Share a Long Context During LLM Inference" §3.1, "Storing
//   each token once": token p on shard p mod C at row p / C; serving caches keep
//   those rows in pages, "DeepSeek-V4 Attention Inference Systems" §9.2).
// * append kernels: the new tokens' rows into those pool rows, as they are or
//   as E4M3 codes with one fp32 scale a token.
#include <cuda_bf16.h>

#include "early_launch.cuh"
#include "internal.h"

namespace cpattn {
namespace {

// ------------------------------------------------------------------ slots
//
// L tokens over C shards: with q = L / C and m = L mod C, shards r < m hold
// q + 1 rows and the others q.  So the pages of shards 0..r-1 have a closed
// form, and only the requests need a running sum:
//   F(L, r) = min(r, m) ceil((q + 1) / page) + max(0, r - m) ceil(q / page)
// New pages are taken in the order of requests, then shards, then pages.
// Every block runs the sum over the requests for itself (a few loads a
// thread) and writes its own part, so the step is one launch without a barrier
// between blocks; the first blocks write slots, the others table entries, so
// neither waits for the other's loads.  The step of a decode batch is a chain of
// latencies (launch, lengths, sum, page id, store): lengths are divided by C
// and the page size with a multiplication.
constexpr int kSlotThreads = 256;
constexpr int kSlotWarps = kSlotThreads / 32;

// n / d for 0 <= n < 2^31: with 2^s >= d > 2^(s-1) and m = ceil(2^(31+s) / d),
// m d - 2^(31+s) < d <= 2^s, so n m / 2^(31+s) passes n / d by less than 1 / d.
struct FastDiv {
  uint32_t m;
  int shift, d;
  explicit FastDiv(int div) : d(div) {
    int s = 0;
    while ((1ll << s) < div) ++s;
    shift = 31 + s;
    m = (uint32_t)(((1ull << shift) + div - 1) / div);
  }
  __device__ __forceinline__ int operator()(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> shift); }
};

struct SlotsParams {
  PageSlotsArgs a;
  FastDiv by_c, by_page;
  int tok_blocks;  // blocks that write slots; the others write table entries
  int wide;        // a warp a pair (many pages each) instead of a thread
};

struct PageCount {
  int m, small, big;  // the first m shards hold `big` pages, the others `small`
};
__device__ __forceinline__ PageCount page_count(const SlotsParams& p, int L) {
  PageCount c;
  const int q = p.by_c(L), qp = p.by_page(q);
  c.m = L - q * p.by_c.d;
  c.small = qp + (q != qp * p.by_page.d);
  c.big = qp + 1;
  return c;
}
__device__ __forceinline__ int pages_before(const PageCount& c, int r) {
  return min(r, c.m) * c.big + max(0, r - c.m) * c.small;
}
__device__ __forceinline__ int pages_of(const PageCount& c, int r) { return r < c.m ? c.big : c.small; }
// Sums that stop at 2^32 - 1, past every limit that they are compared with
// (limits are at most 2^31 - 1).
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) {
  const uint32_t sum = a + b;
  return sum < a ? 0xFFFFFFFFu : sum;
}

// VEC consecutive tokens a thread.
template <int VEC>
__global__ void __launch_bounds__(kSlotThreads) page_slots_kernel(const SlotsParams p) {
  extern __shared__ int32_t sm[];
  const PageSlotsArgs& a = p.a;
  int32_t* s_cu = sm;              // [B + 1] new tokens before request b
  int32_t* s_take = sm + a.B + 1;  // [B] pages taken before request b
  __shared__ uint32_t w_tok[kSlotWarps], w_take[kSlotWarps];
  __shared__ int w_bad[kSlotWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.B, C = a.C, page = a.page_size;
  wait_for_earlier_kernels();
  const int pos = *a.free_pos;

  // running sums over the requests: a thread takes `per` consecutive ones
  const int per = (B + kSlotThreads - 1) / kSlotThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  uint32_t tok = 0, take = 0;
  int bad = 0;
  for (int b = b0; b < b1; ++b) {
    const int L = a.ctx_len[b], n = a.new_len[b];
    if (L < 0 || n < 0 || L > 0x7FFFFFFF - n) {
      bad |= CP_SLOTS_BAD_LENGTH;
      continue;
    }
    const PageCount want = page_count(p, L + n), have = page_count(p, L);
    if (pages_of(want, 0) > a.max_pages) bad |= CP_SLOTS_TABLE_FULL;
    tok = sat_add(tok, n);
    take = sat_add(take, pages_before(want, C) - pages_before(have, C));  // at most C + 2^31 / 64 pages each
  }
  uint32_t tok_in = tok, take_in = take;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, tok_in, d), y = __shfl_up_sync(0xffffffffu, take_in, d);
    if (lane >= d) {
      tok_in = sat_add(tok_in, x);
      take_in = sat_add(take_in, y);
    }
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (lane == 31) {
    w_tok[warp] = tok_in;
    w_take[warp] = take_in;
    w_bad[warp] = bad;
  }
  __syncthreads();
  uint32_t before_tok = 0, before_take = 0, total = 0, taken = 0;
#pragma unroll
  for (int w = 0; w < kSlotWarps; ++w) {
    if (w == warp) {
      before_tok = total;
      before_take = taken;
    }
    total = sat_add(total, w_tok[w]);
    taken = sat_add(taken, w_take[w]);
    bad |= w_bad[w];
  }
  if (pos < 0 || pos > a.n_free || taken > (uint32_t)(a.n_free - pos)) bad |= CP_SLOTS_NO_PAGES;
  if (total > (uint32_t)a.max_tokens) bad |= CP_SLOTS_TOO_MANY;
  if (blockIdx.x == 0 && tid == 0)
    *reinterpret_cast<int4*>(a.info) =
        bad ? make_int4(bad, pos, 0, 0) : make_int4(0, pos + (int)taken, (int)taken, (int)total);
  const bool tokens = blockIdx.x < (unsigned)p.tok_blocks;
  if (bad) {  // nothing is taken: no table entry changes, no token has a slot
    for (int b = tid; b <= B && blockIdx.x == 0; b += kSlotThreads) a.cu_new[b] = 0;
    for (long long t = (long long)blockIdx.x * kSlotThreads + tid; tokens && t < a.max_tokens;
         t += (long long)p.tok_blocks * kSlotThreads)
      a.slots[t] = -1;
    return;
  }
  // nothing saturated: every sum is at most n_free or max_tokens
  int tok0 = (int)(before_tok + tok_in - tok), take0 = (int)(before_take + take_in - take);
  for (int b = b0; b < b1; ++b) {
    const int L = a.ctx_len[b], n = a.new_len[b];
    s_cu[b] = tok0;
    s_take[b] = take0;
    if (blockIdx.x == 0) a.cu_new[b] = tok0;
    if (b + 1 == b1) break;
    tok0 += n;
    take0 += pages_before(page_count(p, L + n), C) - pages_before(page_count(p, L), C);
  }
  if (tid == 0) {
    s_cu[B] = (int)total;
    if (blockIdx.x == 0) a.cu_new[B] = (int)total;
  }
  __syncthreads();

  auto id_of = [&](int i) {  // a page id of the free list, -1 if it names no page
    const int id = a.free_ids[i];
    return id >= 0 && id < a.num_pages ? id : -1;
  };
  if (!tokens) {
    // new table entries of the (request, shard) pairs
    const int pairs = B * C, block = blockIdx.x - p.tok_blocks, blocks = gridDim.x - p.tok_blocks;
    const int step = p.wide ? 32 : 1, off = p.wide ? lane : 0;
    const int first = p.wide ? warp * blocks + block : block * kSlotThreads + tid;
    const int stride = p.wide ? blocks * kSlotWarps : blocks * kSlotThreads;
    for (int u = first; u < pairs; u += stride) {
      const int b = p.by_c(u), r = u - b * C;
      const int L = a.ctx_len[b], n = a.new_len[b];
      if (n == 0) continue;
      const PageCount want = page_count(p, L + n), have = page_count(p, L);
      const int h0 = pages_of(have, r), h1 = pages_of(want, r);
      const int src = pos + s_take[b] + pages_before(want, r) - pages_before(have, r) - h0;
      int32_t* row = a.table + ((long long)r * B + b) * a.max_pages;
      for (int i = h0 + off; i < h1; i += step) row[i] = id_of(src + i);
    }
    return;
  }
  const long long stride = (long long)p.tok_blocks * kSlotThreads * VEC;
  for (long long t0 = ((long long)blockIdx.x * kSlotThreads + tid) * VEC; t0 < a.max_tokens; t0 += stride) {
    int out[VEC];
    int lo = 0, hi = B - 1;  // the last request starting at or before t0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_cu[mid] <= t0) lo = mid; else hi = mid - 1;
    }
    int b = lo, L = 0;
    PageCount want, have;
    bool fresh = true;
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const long long t = t0 + k;
      out[k] = -1;
      if (t >= total) continue;
      while (t >= s_cu[b + 1]) {  // requests without new tokens are passed over
        ++b;
        fresh = true;
      }
      if (fresh) {
        L = a.ctx_len[b];
        want = page_count(p, s_cu[b + 1] - s_cu[b] + L);
        have = page_count(p, L);
        fresh = false;
      }
      const int q = L + (int)(t - s_cu[b]);
      const int i = p.by_c(q), r = q - i * C, pg = p.by_page(i);
      const int h0 = pages_of(have, r);
      int id;
      if (pg < h0) {
        id = a.table[((long long)r * B + b) * a.max_pages + pg];
        if (id < 0 || id >= a.num_pages) id = -1;
      } else {
        id = id_of(pos + s_take[b] + pages_before(want, r) - pages_before(have, r) + pg - h0);
      }
      if (id >= 0) out[k] = id * page + (i - pg * page);
    }
    if (VEC == 4 && t0 + VEC <= a.max_tokens) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(out[0], out[VEC > 1 ? 1 : 0], out[VEC > 2 ? 2 : 0], out[VEC > 3 ? 3 : 0]);
    } else {
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (t0 + k < a.max_tokens) a.slots[t0 + k] = out[k];
    }
  }
}

// ------------------------------------------------------------------ append

constexpr int kAppendThreads = 128;

// Rows as they are: LPR lanes a row, 16-byte pieces of K and V, loaded before
// the first store (which may alias the next load for all the compiler knows):
// both rows' one piece a lane where they are short, else four of K, then of V.
template <int LPR>
__global__ void __launch_bounds__(kAppendThreads) append_copy_kernel(const AppendArgs a, int elem) {
  const int per_block = kAppendThreads / LPR;
  const long long row = (long long)blockIdx.x * per_block + threadIdx.x / LPR;
  const int lane = threadIdx.x % LPR;
  wait_for_earlier_kernels();
  if (row >= a.n) return;
  const int slot = a.slots[row];
  if (slot < 0 || slot >= a.pool_rows) return;
  const int vec = a.row_elems * elem / 16;
  const uint4* k = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.k) + row * a.k_stride * elem);
  const uint4* v = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.v) + (a.v ? row * a.v_stride * elem : 0));
  uint4* kd = static_cast<uint4*>(a.k_pool) + (long long)slot * vec;
  uint4* vd = static_cast<uint4*>(a.v_pool) + (a.v ? (long long)slot * vec : 0);
  const float scale = a.scale_pool && lane == 0 ? a.new_scale[row] : 0.f;
  if constexpr (LPR < 32) {
    if (lane < vec) {
      const uint4 x = __ldcg(k + lane), y = a.v ? __ldcg(v + lane) : make_uint4(0, 0, 0, 0);
      kd[lane] = x;
      if (a.v) vd[lane] = y;
    }
  } else {
    auto copy = [&](const uint4* src, uint4* dst) {
      for (int c0 = lane; c0 < vec; c0 += 4 * LPR) {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + i * LPR < vec) x[i] = __ldcg(src + c0 + i * LPR);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + i * LPR < vec) dst[c0 + i * LPR] = x[i];
      }
    };
    copy(k, kd);
    if (a.v) copy(v, vd);
  }
  if (a.scale_pool && lane == 0) a.scale_pool[slot] = scale;
}

// Eight elements of a row as floats.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  uint4 x;
  __device__ void load(const void* p) { x = __ldcg(static_cast<const uint4*>(p)); }
  __device__ void zero() { x = make_uint4(0, 0, 0, 0); }
  __device__ float at(int i) const {
    const uint32_t w = i < 2 ? x.x : i < 4 ? x.y : i < 6 ? x.z : x.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  // The largest magnitude, as fp32 bits, of this and `top`: magnitudes are
  // ordered like their bits, two bf16 at a time here.
  __device__ uint32_t top_of(uint32_t top) const {
    const uint32_t k = 0x7fff7fffu;
    const uint32_t m = __vmaxu2(__vmaxu2(x.x & k, x.y & k), __vmaxu2(x.z & k, x.w & k));
    return max(top, max(m & 0xffff0000u, m << 16));
  }
};
template <>
struct Piece<float> {
  uint4 x, y;
  __device__ void load(const void* p) {
    x = __ldcg(static_cast<const uint4*>(p));
    y = __ldcg(static_cast<const uint4*>(p) + 1);
  }
  __device__ void zero() { x = y = make_uint4(0, 0, 0, 0); }
  __device__ float at(int i) const {
    const uint4& w = i < 4 ? x : y;
    const int k = i & 3;
    return __uint_as_float(k == 0 ? w.x : k == 1 ? w.y : k == 2 ? w.z : w.w);
  }
  __device__ uint32_t top_of(uint32_t top) const {
    const uint32_t k = 0x7fffffffu;
    return max(top, max(max(max(x.x & k, x.y & k), max(x.z & k, x.w & k)), max(max(y.x & k, y.y & k), max(y.z & k, y.w & k))));
  }
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// Codes of eight elements: rn_E4M3(x / scale), the quotient rounded to fp32
// first as a division gives it.  With y = 1 / scale rounded once, q = x y is
// within two units of the quotient, x - q scale is exact in one FMA, and adding
// it times y rounds to the quotient (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): three operations
// where a division is some ten (37.5 us instead of 31.1 for 32,768 tokens of 2,048 elements).
// `plain` for scales whose products could leave the normal range.
template <typename T>
__device__ __forceinline__ uint2 codes_of(const Piece<T>& x, float scale, float inv, bool plain) {
  float q[8];
  if (plain) {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(x.at(i), scale);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = x.at(i), q0 = v * inv;
      q[i] = __fmaf_rn(-__fmaf_rn(q0, scale, -v), inv, q0);  // these signs keep that of a zero
    }
  }
  return make_uint2(e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
}

// Rows to E4M3 codes with one scale a token, amax / 448 (at least 2^-149; 1 for
// a row of zeros) over its K row and, where there is one, its V row: a warp a token,
// PIECES pieces of eight elements of each row a lane, kept in registers between
// the maximum and the codes (PIECES = 0: any row length, read twice).
template <typename T, int PIECES, bool HAS_V>
__global__ void __launch_bounds__(kAppendThreads) append_e4m3_kernel(const AppendArgs a) {
  const long long row = (long long)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  wait_for_earlier_kernels();
  if (row >= a.n) return;
  const int slot = a.slots[row];
  if (slot < 0 || slot >= a.pool_rows) return;
  constexpr int N = PIECES ? PIECES : 1, R = HAS_V ? 2 : 1;
  const int vec = a.row_elems / 8;
  const T* src[R];
  uint2* dst[R];
  src[0] = static_cast<const T*>(a.k) + row * a.k_stride + 8 * lane;
  dst[0] = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.k_pool) + (long long)slot * a.row_elems) + lane;
  if (HAS_V) {
    src[R - 1] = static_cast<const T*>(a.v) + row * a.v_stride + 8 * lane;
    dst[R - 1] = reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.v_pool) + (long long)slot * a.row_elems) + lane;
  }
  uint32_t top = 0;
  Piece<T> x[R][N];
  if (PIECES) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane + 32 * i < vec) x[r][i].load(src[r] + 256 * i); else x[r][i].zero();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < N; ++i) top = x[r][i].top_of(top);
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
      for (int c = 0; c < vec - lane; c += 32) {
        x[r][0].load(src[r] + 8 * c);
        top = x[r][0].top_of(top);
      }
  }
  const float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, top));
  // the quotient of an fp32 row up to 224 x 2^-149 is 0, which would make codes
  // of NaN out of its zeros: the least positive scale stands for such rows
  const float scale = amax > 0.f ? fmaxf(__fdiv_rn(amax, 448.f), 0x1p-149f) : 1.f;
  if (lane == 0) a.scale_pool[slot] = scale;
  const float inv = __frcp_rn(scale);
  const bool plain = !(scale >= 0x1p-80f && scale <= 0x1p100f);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (PIECES) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (lane + 32 * i < vec) dst[r][32 * i] = codes_of(x[r][i], scale, inv, plain);
    } else {
      for (int c = 0; c < vec - lane; c += 32) {
        x[r][0].load(src[r] + 8 * c);
        dst[r][c] = codes_of(x[r][0], scale, inv, plain);
      }
    }
  }
}

template <typename T, bool HAS_V>
cudaError_t append_e4m3(const AppendArgs& a, cudaStream_t s) {
  const int per_lane = (a.row_elems / 8 + 31) / 32;
  const unsigned grid = (unsigned)(((long long)a.n + kAppendThreads / 32 - 1) / (kAppendThreads / 32));
  auto kern = append_e4m3_kernel<T, 0, HAS_V>;
  if (per_lane == 1) kern = append_e4m3_kernel<T, 1, HAS_V>;
  else if (per_lane == 2) kern = append_e4m3_kernel<T, 2, HAS_V>;
  else if (per_lane == 3) kern = append_e4m3_kernel<T, 3, HAS_V>;
  else if (per_lane == 4) kern = append_e4m3_kernel<T, 4, HAS_V>;
  else if (per_lane <= 8 && sizeof(T) == 2) kern = append_e4m3_kernel<T, sizeof(T) == 2 ? 8 : 0, HAS_V>;
  return launch_early(kern, grid, kAppendThreads, 0, s, 1, a);
}

template <int LPR>
cudaError_t append_copy(const AppendArgs& a, int elem, cudaStream_t s) {
  const int per_block = kAppendThreads / LPR;
  return launch_early(append_copy_kernel<LPR>, (unsigned)(((long long)a.n + per_block - 1) / per_block), kAppendThreads, 0, s, 1, a,
                      elem);
}

}  // namespace

cudaError_t launch_page_slots(const PageSlotsArgs& a, cudaStream_t s) {
  SlotsParams p = {a, FastDiv(a.C), FastDiv(a.page_size), 0, 0};
  // one token a thread until the blocks fill the SMs twice, then four
  const bool vec = a.max_tokens > 304 * kSlotThreads;
  const long long per_block = (long long)kSlotThreads * (vec ? 4 : 1);
  const long long tok = (a.max_tokens + per_block - 1) / per_block;
  p.tok_blocks = (int)(tok < 1 ? 1 : tok > 608 ? 608 : tok);
  const long long pairs = (long long)a.B * a.C;
  p.wide = a.max_tokens > 4 * pairs * a.page_size;  // some four new pages a pair or more
  const long long pb = p.wide ? (pairs + kSlotWarps - 1) / kSlotWarps : (pairs + kSlotThreads - 1) / kSlotThreads;
  const unsigned grid = (unsigned)(p.tok_blocks + (pb > 152 ? 152 : pb));
  const size_t smem = (size_t)(2 * a.B + 1) * sizeof(int32_t);
  auto kern = vec ? page_slots_kernel<4> : page_slots_kernel<1>;
  if (smem > 40 * 1024) {
    // the most that any call needs: a limit of this call's own would be another
    // thread's for a moment, and refuse its launch
    constexpr int kMost = (2 * CP_SLOTS_MAX_B + 1) * (int)sizeof(int32_t);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  return launch_early(kern, grid, kSlotThreads, smem, s, 1, p);
}

cudaError_t launch_cache_append(const AppendArgs& a, cp_dtype src, cp_dtype pool, cudaStream_t s) {
  if (src == pool) {
    const int elem = src == CP_FP32 ? 4 : src == CP_BF16 ? 2 : 1;
    const int vec = a.row_elems * elem / 16;
    return vec <= 8 ? append_copy<8>(a, elem, s) : vec <= 16 ? append_copy<16>(a, elem, s) : append_copy<32>(a, elem, s);
  }
  if (src == CP_BF16) return a.v ? append_e4m3<__nv_bfloat16, true>(a, s) : append_e4m3<__nv_bfloat16, false>(a, s);
  return a.v ? append_e4m3<float, true>(a, s) : append_e4m3<float, false>(a, s);
}

}  // namespace cpattn

// Eviction from a paged token-sharded cache by accumulated attention weight.
//
// A request of L cached tokens that shall keep K of them holds, on shard r,
// n = ceil((L - r) / C) rows before and m = ceil((K - r) / C) after ("How GPUs
// Share a Long Context During LLM Inference" §3.1, the round-robin rows of K
// tokens), so plans and slots of K tokens fit the thinned cache.  Each pair
// (shard, request) keeps the m heaviest of its own rows: no shard needs another's.
//
// * evict_select_kernel: which rows those are, and the moves that bring them
//   together.  Attention does not depend on the order of the rows (keys carry their
//   rotation), so only kept rows behind the m-th move, into the places of evicted
//   ones before it: a step that evicts a few tokens moves a few rows.
// * cache_move_kernel: the moves (180 MB of 2 KB rows read and written in 28 us).
// * page_release_kernel: the pages that the shorter pairs no longer need, back
//   to the free list that page_slots_kernel takes them from.
#include "early_launch.cuh"
#include "internal.h"
#include "page_count.cuh"

namespace cpattn {
namespace {

// ------------------------------------------------------------------ select

// A pair's rows are ranked by a 32-bit key with the order of their weights: the
// m-th largest key is found, and a scan in row order tells the rows equal to it
// apart and numbers the moves.  A block a pair.
constexpr uint32_t kProtected = 0xFFFFFFFFu;  // above +inf's key

// Larger weight, larger key; equal weights (-0 and 0 too), equal keys; NaN below all.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  if (w != w) return 0;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Protected by its position: below keep_below, or from `start`, its request's keep_from, on.  A negative
// position, which nobody has written, protects nothing.
__device__ __forceinline__ bool protects(const EvictArgs& a, int pos, int start) {
  return pos >= 0 && (pos < a.keep_below || (a.keep_from && pos >= start));
}

// Pairs of up to R x 1,024 rows: the keys stay in registers, R of a thread (rows
// tid, tid + NT, ...), and the m-th largest one is found bit by bit: it is the largest T
// that at least m keys reach.  A bit is one count over the block and one barrier (512
// pairs of 264 rows with their moves 22.7 -> 16.3 us against a radix select).
constexpr int kBitThreads = 1024;
template <int R>
__global__ void __launch_bounds__(kBitThreads) evict_bits_kernel(const EvictArgs a, const FastDiv by_page) {
  __shared__ int s_count[2][32], s_equal[R][32], s_holes[R][32], s_movers[R][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, warps = nt >> 5;
  const int pair = blockIdx.x, b = pair % a.B, r = pair / a.B;
  wait_for_earlier_kernels();
  // a row behind the pair's last reads its page's entry as far as the table goes, too
  int id[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int page = by_page(tid + k * nt);
    id[k] = page < a.max_pages ? __ldcg(a.table + (long long)pair * a.max_pages + page) : -1;
  }
  const int L = a.ctx_len[b], K = a.keep_len[b], start = a.keep_from ? a.keep_from[b] : 0;
  auto rows_of = [&](int len) { return len > r ? (len - r - 1) / a.C + 1 : 0; };
  const bool bad_len = L < 0 || K < 0 || rows_of(L) > (long long)a.max_pages * a.page_size;
  const int n = bad_len ? 0 : rows_of(L), m = bad_len ? 0 : min(n, rows_of(K));
  uint32_t key[R];
  int row[R];
  bool outside = false;
  {
    float w[R];
    int pos[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int i = tid + k * nt;
      const bool in = id[k] >= 0 && id[k] < a.num_pages;
      outside |= i < n && !in;
      row[k] = id[k] * a.page_size + (i - by_page(i) * a.page_size);
      pos[k] = in && i < n && a.pos ? __ldcg(a.pos + row[k]) : i * a.C + r;
      w[k] = in && i < n ? __ldcg(a.weights + row[k]) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < R; ++k) key[k] = protects(a, pos[k], start) ? kProtected : weight_key(w[k]);
  }
  const bool bad = __syncthreads_or(outside);
  int32_t* src = a.src + (long long)pair * a.max_moves;
  int32_t* dst = a.dst + (long long)pair * a.max_moves;
  int moves = bad_len || bad ? -1 : 0;
  if (m > 0 && m < n && !bad) {
    // keys that are at least t, of the whole block
    int turn = 0;
    auto reach = [&](uint32_t t) {
      int c = 0;
#pragma unroll
      for (int k = 0; k < R; ++k) c += tid + k * nt < n && key[k] >= t;
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) s_count[turn][warp] = c;
      __syncthreads();
      c = __reduce_add_sync(0xffffffffu, lane < warps ? s_count[turn][lane] : 0);
      turn ^= 1;  // the next count writes where nobody reads any more after its barrier
      return c;
    };
    uint32_t mth = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t t = mth | (1u << bit);
      if (reach(t) >= m) mth = t;
    }
    // of the rows equal to the m-th, the first `need` stay
    const int need = m - (mth == 0xFFFFFFFFu ? 0 : reach(mth + 1));
    const unsigned below = (1u << lane) - 1;
    unsigned eq[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      eq[k] = __ballot_sync(0xffffffffu, tid + k * nt < n && key[k] == mth);
      if (lane == 0) s_equal[k][warp] = __popc(eq[k]);
    }
    __syncthreads();
    // a count's running sum over the rows before this warp's of slice k, and its total
    auto before = [&](int (&count)[R][32], int (&first)[R]) {
      int total = 0;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int c = lane < warps ? count[k][lane] : 0;
        first[k] = total + __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
        total += __reduce_add_sync(0xffffffffu, c);
      }
      return total;
    };
    int first[R];
    before(s_equal, first);
    unsigned holes[R], movers[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int i = tid + k * nt;
      const bool equal = i < n && key[k] == mth;
      const bool stay = i < n && (equal ? first[k] + __popc(eq[k] & below) < need : key[k] > mth);
      holes[k] = __ballot_sync(0xffffffffu, i < n && !stay && i < m);
      movers[k] = __ballot_sync(0xffffffffu, stay && i >= m);
      if (lane == 0) {
        s_holes[k][warp] = __popc(holes[k]);
        s_movers[k][warp] = __popc(movers[k]);
      }
    }
    __syncthreads();
    int hole[R], mover[R];
    moves = before(s_holes, hole);
    before(s_movers, mover);
    if (moves > a.max_moves) {
      moves = -1;
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (holes[k] >> lane & 1) dst[hole[k] + __popc(holes[k] & below)] = row[k];
        if (movers[k] >> lane & 1) src[mover[k] + __popc(movers[k] & below)] = row[k];
      }
    }
  }
  for (long long x = max(moves, 0) + tid; x < a.max_moves; x += nt) src[x] = dst[x] = -1;
  if (tid == 0) a.count[pair] = moves;
}

// Longer pairs: a radix select over the key's four bytes, the keys in shared memory (read
// from the pool again where they do not fit).
struct SelectParams {
  EvictArgs a;
  FastDiv by_page;
  int cached;  // keys that fit shared memory
};

template <int NT>
__global__ void __launch_bounds__(NT) evict_select_kernel(const SelectParams p) {
  constexpr int kWarps = NT / 32;
  extern __shared__ uint32_t s_key[];
  __shared__ int s_hist[256], s_count[kWarps], s_count2[kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need, s_equal, s_bad;
  const EvictArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = blockIdx.x, b = pair % a.B, r = pair / a.B;
  wait_for_earlier_kernels();
  const int L = a.ctx_len[b], K = a.keep_len[b], start = a.keep_from ? a.keep_from[b] : 0;
  auto rows_of = [&](int len) { return len > r ? (len - r - 1) / a.C + 1 : 0; };
  int32_t* src = a.src + (long long)pair * a.max_moves;
  int32_t* dst = a.dst + (long long)pair * a.max_moves;
  const bool bad_len = L < 0 || K < 0 || rows_of(L) > (long long)a.max_pages * a.page_size;
  const int n = bad_len ? 0 : rows_of(L), m = bad_len ? 0 : min(n, rows_of(K));
  const int32_t* table = a.table + (long long)pair * a.max_pages;
  auto pool_row = [&](int i) -> int {  // -1: its page is outside the pool
    const int pg = p.by_page(i), id = table[pg];
    return id >= 0 && id < a.num_pages ? id * a.page_size + (i - pg * a.page_size) : -1;
  };
  auto read_key = [&](int i) -> uint32_t {
    const int row = pool_row(i);
    if (row < 0) return 0;
    const int pos = a.pos ? a.pos[row] : i * a.C + r;
    if (protects(a, pos, start)) return kProtected;
    return weight_key(a.weights[row]);
  };
  auto key_of = [&](int i) { return i < p.cached ? s_key[i] : read_key(i); };
  // Keys of kBatch rows a thread: pages, then weights and positions are loaded together.
  // False where a page is outside the pool.
  constexpr int kBatch = 4;
  auto load_keys = [&](int i0) {
    int id[kBatch], pos[kBatch];
    float w[kBatch];
    bool good = true;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) id[k] = i0 + k * NT < n ? __ldcg(table + p.by_page(i0 + k * NT)) : 0;
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * NT;
      const bool in = id[k] >= 0 && id[k] < a.num_pages;
      const int row = id[k] * a.page_size + (i - p.by_page(i) * a.page_size);
      good &= in || i >= n;
      pos[k] = in && i < n && a.pos ? __ldcg(a.pos + row) : i * a.C + r;
      w[k] = in && i < n ? __ldcg(a.weights + row) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * NT;
      if (i < n && i < p.cached) s_key[i] = protects(a, pos[k], start) ? kProtected : weight_key(w[k]);
    }
    return good;
  };
  int moves = bad_len ? -1 : 0;
  if (n > 0 && !(m > 0 && m < n)) {  // all rows stay or none: of the pages nothing is asked but that they are there
    bool bad = false;
    for (int pg = tid; pg <= p.by_page(n - 1); pg += NT) {
      const int id = __ldcg(table + pg);
      bad |= id < 0 || id >= a.num_pages;
    }
    if (__syncthreads_or(bad)) moves = -1;
  }
  if (m > 0 && m < n) {
    if (tid == 0) {
      s_prefix = 0;
      s_need = m;
      s_bad = 0;
    }
    for (int i = tid; i < 256; i += NT) s_hist[i] = 0;
    __syncthreads();
    bool bad = false;
    for (int i = tid; i < n; i += kBatch * NT) bad |= !load_keys(i);
    if (bad) s_bad = 1;
    __syncthreads();
    for (int shift = 24; shift >= 0; shift -= 8) {
      const uint32_t prefix = s_prefix;
      for (int i0 = 0; i0 < n; i0 += NT) {
        const int i = i0 + tid;
        const uint32_t key = i < n ? key_of(i) : 0;
        // bytes above this one equal to the m-th key's
        const bool in = i < n && (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)));
        const int digit = (key >> shift) & 255;
        // rows of a warp with one digit count as one addition: weights share their first bytes
        const unsigned who = __match_any_sync(0xffffffffu, in ? digit : 256 + lane);
        if (in && lane == __ffs(who) - 1) atomicAdd(&s_hist[digit], __popc(who));
      }
      __syncthreads();
      if (warp == 0) {
        // from the largest digit down: lane l holds digits 255 - 8 l .. 248 - 8 l
        int mine = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) mine += s_hist[255 - 8 * lane - k];
        int before = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, before, d);
          if (lane >= d) before += y;
        }
        before -= mine;
        const int need = s_need;
        __syncwarp();
        if (before < need && need <= before + mine) {
          for (int k = 0; k < 8; ++k) {
            const int digit = 255 - 8 * lane - k, c = s_hist[digit];
            if (need <= before + c) {
              s_prefix = prefix | ((uint32_t)digit << shift);
              s_need = need - before;
              s_equal = c;
              break;
            }
            before += c;
          }
        }
        __syncwarp();
        for (int i = lane; i < 256; i += 32) s_hist[i] = 0;
      }
      __syncthreads();
    }
    const uint32_t mth = s_prefix;
    const int need = s_need;              // rows with the m-th key that stay: the first ones
    const bool all_equal = need == s_equal;
    // a warp takes consecutive rows, so that ballots number them in order
    const int per = ((n + kWarps - 1) / kWarps + 31) & ~31;
    const int w0 = min(n, warp * per), w1 = min(n, w0 + per);
    int equal0 = 0;
    if (!all_equal) {
      int c = 0;
      for (int i0 = w0; i0 < w1; i0 += 32) c += __popc(__ballot_sync(0xffffffffu, i0 + lane < w1 && key_of(i0 + lane) == mth));
      if (lane == 0) s_count[warp] = c;
      __syncthreads();
      for (int w = 0; w < warp; ++w) equal0 += s_count[w];
      __syncthreads();
    }
    const unsigned below = (1u << lane) - 1;
    // holes (evicted rows before m) and movers (kept rows from m on) of this warp's rows
    auto walk = [&](auto&& each) {
      int equal = equal0;
      for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const bool there = i < w1;
        const uint32_t key = there ? key_of(i) : 0;
        bool stay = there && key >= mth;
        if (!all_equal) {
          const unsigned eq = __ballot_sync(0xffffffffu, there && key == mth);
          if (there && key == mth) stay = equal + __popc(eq & below) < need;
          equal += __popc(eq);
        }
        each(i, __ballot_sync(0xffffffffu, there && !stay && i < m), __ballot_sync(0xffffffffu, stay && i >= m));
      }
    };
    int holes = 0, movers = 0;
    walk([&](int, unsigned h, unsigned v) {
      holes += __popc(h);
      movers += __popc(v);
    });
    if (lane == 0) {
      s_count[warp] = holes;
      s_count2[warp] = movers;
    }
    __syncthreads();
    int hole0 = 0, mover0 = 0;
    moves = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
        hole0 = moves;
        for (int x = 0; x < w; ++x) mover0 += s_count2[x];
      }
      moves += s_count[w];
    }
    if (s_bad || moves > a.max_moves) {
      moves = -1;
    } else {
      walk([&](int i, unsigned h, unsigned v) {
        if (h >> lane & 1) dst[hole0 + __popc(h & below)] = pool_row(i);
        if (v >> lane & 1) src[mover0 + __popc(v & below)] = pool_row(i);
        hole0 += __popc(h);
        mover0 += __popc(v);
      });
    }
  }
  for (long long i = max(moves, 0) + tid; i < a.max_moves; i += NT) src[i] = dst[i] = -1;
  if (tid == 0) a.count[pair] = moves;
}

// ------------------------------------------------------------------ move

constexpr int kMoveThreads = 256;

struct MoveParams {
  MoveArgs a;
  int splits;  // blocks that share a pair
};

// A warp a move: both rows' pieces are loaded before the first store, and the rows
// of its next moves are known before (a lane reads those of one).  Sources are rows behind
// the new length and destinations before it, so no move reads what another writes.
__global__ void __launch_bounds__(kMoveThreads) cache_move_kernel(const MoveParams p) {
  const MoveArgs& a = p.a;
  const int pair = blockIdx.x / p.splits, part = blockIdx.x - pair * p.splits;
  const int lane = threadIdx.x & 31, warp = part * (kMoveThreads / 32) + (threadIdx.x >> 5);
  const int step = p.splits * (kMoveThreads / 32);
  wait_for_earlier_kernels();
  int n = min(__ldcg(a.count + pair), a.max_moves);
  if (a.B) {  // a request whole: none of it moves where a shard's choice did not fit
    bool unfit = false;
    for (int r = lane; r < a.C; r += 32) unfit |= __ldcg(a.count + r * a.B + pair % a.B) < 0;
    if (__any_sync(0xffffffffu, unfit)) n = 0;
  }
  const int vec = a.row_bytes / 16;
  for (long long j0 = warp; j0 < n; j0 += 32 * step) {
    const long long mine = j0 + lane * step;
    const long long at = (long long)pair * a.max_moves + mine;
    const int src = mine < n ? __ldcg(a.src + at) : -1, dst = mine < n ? __ldcg(a.dst + at) : -1;
    const bool good = src >= 0 && dst >= 0 && src < a.pool_rows && dst < a.pool_rows;
    if (good) {  // the words a row has beside its pieces
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (a.words[k]) a.words[k][dst] = __ldcg(a.words[k] + src);
    }
    for (unsigned left = __ballot_sync(0xffffffffu, good); left; left &= left - 1) {
      const int k = __ffs(left) - 1;
      const long long from = __shfl_sync(0xffffffffu, src, k), to = __shfl_sync(0xffffffffu, dst, k);
      const uint4* k0 = static_cast<const uint4*>(a.k) + from * vec;
      uint4* k1 = static_cast<uint4*>(a.k) + to * vec;
      const uint4* v0 = a.v ? static_cast<const uint4*>(a.v) + from * vec : nullptr;
      uint4* v1 = a.v ? static_cast<uint4*>(a.v) + to * vec : nullptr;
      for (int c0 = lane; c0 < vec; c0 += 128) {
        uint4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 32 * i < vec) {
            x[i] = __ldcg(k0 + c0 + 32 * i);
            if (v0) y[i] = __ldcg(v0 + c0 + 32 * i);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + 32 * i < vec) {
            k1[c0 + 32 * i] = x[i];
            if (v0) v1[c0 + 32 * i] = y[i];
          }
      }
    }
  }
}

// ------------------------------------------------------------------ release

constexpr int kReleaseThreads = 256;
constexpr int kReleaseWarps = kReleaseThreads / 32;

struct ReleaseParams {
  ReleaseArgs a;
  FastDiv by_c, by_page;
};

// Every block sums over the requests for itself, as page_slots_kernel does;
// then a warp a pair hands back its pages and clears the rows that it leaves.  With the
// choice's counts a request with a pair of -1 stays as it is.  512 pairs that hand back a
// page each 2.2 us; 1,396 pages of 64 pairs with their weights and positions 18.5, a warp's
// walk over its pages.
__global__ void __launch_bounds__(kReleaseThreads) page_release_kernel(const ReleaseParams p) {
  extern __shared__ int32_t s_before[];  // [B] pages released before request b; -1: it stays as it is
  __shared__ uint32_t w_sum[kReleaseWarps];
  __shared__ int w_bad[kReleaseWarps], w_stay[kReleaseWarps];
  const ReleaseArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.B, C = a.C;
  wait_for_earlier_kernels();
  const int pos = *a.free_pos;
  const int per = (B + kReleaseThreads - 1) / kReleaseThreads;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  auto released = [&](int b, int* bad) -> uint32_t {
    const int L = a.ctx_len[b], K = a.keep_len[b];
    if (L < 0 || K < 0) {
      *bad |= CP_SLOTS_BAD_LENGTH;
      return 0;
    }
    const PageCount have = page_count(p.by_c, p.by_page, L);
    if (pages_of(have, 0) > a.max_pages) *bad |= CP_SLOTS_TABLE_FULL;
    return K < L ? pages_before(have, C) - pages_before(page_count(p.by_c, p.by_page, K), C) : 0;
  };
  uint32_t sum = 0;
  int bad = 0, stay = 0;
  for (int b = b0; b < b1; ++b) {
    bool unfit = false;  // a shard's choice did not fit
    if (a.count)
      for (int r = 0; r < C; ++r) unfit |= __ldcg(a.count + r * B + b) < 0;
    s_before[b] = unfit ? -1 : 0;
    if (unfit) ++stay;
    else sum = sat_add(sum, released(b, &bad));
  }
  uint32_t in = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, in, d);
    if (lane >= d) in = sat_add(in, x);
  }
  bad = __reduce_or_sync(0xffffffffu, bad);
  stay = __reduce_add_sync(0xffffffffu, stay);
  if (lane == 31) {
    w_sum[warp] = in;
    w_bad[warp] = bad;
    w_stay[warp] = stay;
  }
  __syncthreads();
  uint32_t before = 0, total = 0;
  stay = 0;
#pragma unroll
  for (int w = 0; w < kReleaseWarps; ++w) {
    if (w == warp) before = total;
    total = sat_add(total, w_sum[w]);
    bad |= w_bad[w];
    stay += w_stay[w];
  }
  if (pos < 0 || pos > a.n_free || total > (uint32_t)pos) bad |= CP_SLOTS_NO_PAGES;
  if (blockIdx.x == 0 && tid == 0)
    *reinterpret_cast<int4*>(a.info) = bad ? make_int4(bad, pos, 0, 0) : make_int4(0, pos - (int)total, (int)total, stay);
  if (bad) return;
  // nothing saturated: the sum is at most *free_pos
  int at = (int)(before + in - sum);
  for (int b = b0; b < b1; ++b) {
    if (s_before[b] < 0) continue;
    s_before[b] = at;
    int ignored = 0;
    at += released(b, &ignored);
  }
  __syncthreads();
  const int first = pos - (int)total;
  for (int u = blockIdx.x * kReleaseWarps + warp; u < B * C; u += gridDim.x * kReleaseWarps) {
    const int b = p.by_c(u), r = u - b * C;
    const int L = a.ctx_len[b], K = a.keep_len[b];
    if (K >= L || s_before[b] < 0) continue;
    const PageCount have = page_count(p.by_c, p.by_page, L), want = page_count(p.by_c, p.by_page, K);
    const int q = p.by_c(K), rows = q + (r < K - q * C);  // the pair's new length
    const int h = pages_of(have, r), w = pages_of(want, r);
    int32_t* row = a.table + ((long long)r * B + b) * a.max_pages;
    const int to = first + s_before[b] + pages_before(have, r) - pages_before(want, r) - w;
    for (int i = p.by_page(rows); i < h; ++i) {
      const int id = row[i];
      if (id >= 0 && id < a.num_pages)
        for (int k = (i * a.page_size < rows ? rows - i * a.page_size : 0) + lane; k < a.page_size; k += 32) {
          const long long x = (long long)id * a.page_size + k;
          if (a.weights) a.weights[x] = 0.f;
          if (a.pos) a.pos[x] = -1;
        }
      __syncwarp();
      if (lane == 0 && i >= w) {
        a.free_ids[to + i] = id;
        row[i] = -1;
      }
    }
  }
}

template <int NT>
cudaError_t select_nt(const SelectParams& p, cudaStream_t s) {
  // the most that any call needs: another thread's call may set it at the same time
  constexpr int kMost = 48 * 1024 * 4;
  const size_t smem = (size_t)p.cached * 4;
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  return launch_early(evict_select_kernel<NT>, (unsigned)(p.a.B * p.a.C), NT, smem, s, 1, p);
}

}  // namespace

cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t s) {
  const long long most = (long long)a.max_pages * a.page_size;  // rows of a pair
  const unsigned pairs = (unsigned)(a.B * a.C);
  const FastDiv by_page(a.page_size);
  if (most <= kBitThreads) return launch_early(evict_bits_kernel<1>, pairs, (unsigned)(most + 31) / 32 * 32, 0, s, 1, a, by_page);
  if (most <= 4 * kBitThreads) return launch_early(evict_bits_kernel<4>, pairs, kBitThreads, 0, s, 1, a, by_page);
  // longer ones: a radix select over shared memory (at 4,096 rows the bits are faster: eight
  // prompts with their moves 44 us against 58)
  const SelectParams p = {a, by_page, (int)(most < 48 * 1024 ? most : 48 * 1024)};
  return select_nt<1024>(p, s);
}

cudaError_t launch_cache_move(const MoveArgs& a, cudaStream_t s) {
  // some eight blocks an SM, as many as a pair has work for (four: the same within 2 %)
  const int useful = (a.max_moves - 1) / (kMoveThreads / 32) + 1;
  int splits = (152 * 8 - 1) / a.pairs + 1;
  if (splits > useful) splits = useful;
  return launch_early(cache_move_kernel, (unsigned)a.pairs * splits, kMoveThreads, 0, s, 1, MoveParams{a, splits});
}

cudaError_t launch_page_release(const ReleaseArgs& a, cudaStream_t s) {
  const long long pairs = (long long)a.B * a.C, blocks = (pairs + kReleaseWarps - 1) / kReleaseWarps;
  // requests' sums: at most CP_SLOTS_MAX_B words, within every block's static limit
  return launch_early(page_release_kernel, (unsigned)(blocks < 304 ? blocks : 304), kReleaseThreads, (size_t)a.B * 4, s, 1,
                      ReleaseParams{a, FastDiv(a.C), FastDiv(a.page_size)});
}

}  // namespace cpattn

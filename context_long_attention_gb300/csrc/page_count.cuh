// Pages of the shards of a token-sharded cache.  L tokens over C shards: with
// q = L / C and m = L mod C, shards r < m hold q + 1 rows and the others q.  So
// the pages of shards 0..r-1 have a closed form:
//   F(L, r) = min(r, m) ceil((q + 1) / page) + max(0, r - m) ceil(q / page)
#pragma once

#include <stdint.h>

namespace cpattn {

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

struct PageCount {
  int m, small, big;  // the first m shards hold `big` pages, the others `small`
};
__device__ __forceinline__ PageCount page_count(const FastDiv& by_c, const FastDiv& by_page, int L) {
  PageCount c;
  const int q = by_c(L), qp = by_page(q);
  c.m = L - q * by_c.d;
  c.small = qp + (q != qp * by_page.d);
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

}  // namespace cpattn

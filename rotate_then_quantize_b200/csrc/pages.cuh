// Pages of the quantised cache: rows of a pool, page_size consecutive rows to
// a page. Token t of a sequence lies in row table[t / page_size] * page_size
// + t % page_size of the pool.
#pragma once

#include <cstdint>

namespace srftq {

// n / d for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 d) and
// m = floor(2^32 (2^l - d) / d) + 1, n / d = (hi(m n) + (n - hi(m n)) / 2) >> (l - 1)
// (Granlund and Montgomery, "Division by Invariant Integers using
// Multiplication", 1994). d = 1 is the identity.
struct FastDiv {
  uint32_t d, m, shift;
  static FastDiv make(uint32_t d) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1;
    return {d, uint32_t(m), l == 0 ? 0u : l - 1};
  }
  __host__ __device__ __forceinline__ uint32_t div(uint32_t n) const {
    if (d == 1) return n;
#ifdef __CUDA_ARCH__
    const uint32_t hi = __umulhi(m, n);
#else
    const uint32_t hi = uint32_t((uint64_t(m) * n) >> 32);
#endif
    return (hi + ((n - hi) >> 1)) >> shift;
  }
};

struct PageMap {
  FastDiv page;       // page_size
  int32_t n_pages;    // pages of the pool

  // Pool row of token t, or -1 when the table's entry is no page of the pool
  // (the entry of a page that was never given out, for instance).
  __device__ __forceinline__ int64_t row(const int32_t* table, uint32_t t) const {
    const uint32_t i = page.div(t);
    const int32_t p = __ldg(table + i);
    return uint32_t(p) < uint32_t(n_pages) ? int64_t(p) * page.d + (t - i * page.d) : -1;
  }
};

}  // namespace srftq

// Block tables and slot maps of a step, built from the request lengths.
//
// Sequence b holds cached_b tokens and gets new_b more. It needs the pages
// first_b .. last_b - 1, first_b = ceil(cached_b / page), last_b =
// ceil((cached_b + new_b) / page), taken from the free list in order of the
// sequences, so its pages start at entry sum_{a < b} (last_a - first_a) of that
// list. Its new tokens are the batch rows sum_{a < b} new_a onwards, and row
// r's slot is page * page_size + offset.
//
// One launch. Every block scans all lengths (8 bytes a sequence, from L2
// after the first block) in chunks of kTabThreads with a carry, so no block
// waits for another, and writes the rows and pages that fall to it: blocks of
// kTabThreads consecutive ones in turn. A row finds its sequence by bisection
// in the chunk's scan in shared memory; the row's page is either fresh (its
// free-list entry, which the block knows without reading the table back) or
// the partly filled last page, whose table entry this call does not write. So
// no access depends on another block's. What bounds it is the chain of
// dependent steps, lengths -> scan -> page -> slot: 7 us at 32 sequences, where a
// call of the public entry takes 17 us, most of it the host's; and for large
// batches the search, 11 steps in shared memory for each row at 2047 sequences:
// 18 us for 921000 rows of 8 bytes, 72 % of the issue slots.
#include <climits>

#include "launch_impl.cuh"
#include "pages.cuh"

namespace srftq {

constexpr int kTabThreads = 1024;

struct TableArgs {
  int32_t n_seq;
  const int32_t* cached;
  const int32_t* fresh;
  FastDiv page;
  const int32_t* free_pages;
  int64_t n_free;
  int32_t* table;
  int32_t max_pages;
  int64_t* slots;
  int64_t n_slots;
  int32_t* seq_lens;
  int32_t* row_start;
  int32_t* counts;
  unsigned* guard;
  // Index check of the debug build: the entry of page pg of sequence b.
  __device__ __forceinline__ bool dbg_entry(int64_t b, int64_t pg) const {
    return dbg_ok(b >= 0 && b < n_seq && pg >= 0 && pg < max_pages, guard);
  }
};

__device__ __forceinline__ int64_t warp_inclusive(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__device__ __forceinline__ int32_t saturate32(int64_t v) {
  return v > INT_MAX ? INT_MAX : int32_t(v);
}

// Largest i < n with start[i] <= x (start ascending, start[0] <= x).
__device__ __forceinline__ int last_at_most(const int64_t* start, int n, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kTabThreads) block_tables_kernel(const TableArgs a) {
  __shared__ int64_t rows[kTabThreads + 1], pages[kTabThreads + 1];   // exclusive sums, whole batch
  __shared__ int32_t held[kTabThreads];                               // cached tokens
  __shared__ int64_t part[2][32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t step = int64_t(gridDim.x) * kTabThreads;
  int64_t row0 = 0, page0 = 0;   // sums over the chunks before this one
  for (int b0 = 0; b0 < a.n_seq; b0 += kTabThreads) {
    const int n = a.n_seq - b0 < kTabThreads ? a.n_seq - b0 : kTabThreads;
    int32_t c = 0, f = 0;
    if (tid < n) {
      c = max(a.cached[b0 + tid], 0);
      f = min(max(a.fresh[b0 + tid], 0), INT_MAX - c);   // lengths stay below 2^31
    }
    // ceil(x / page) as 0 for 0 and (x - 1) / page + 1 above
    const int32_t first = c ? int32_t(a.page.div(uint32_t(c - 1))) + 1 : 0;
    const int32_t last = c + f ? int32_t(a.page.div(uint32_t(c + f - 1))) + 1 : 0;
    const int32_t need = max(min(last, a.max_pages) - first, 0);
    const int64_t ri = warp_inclusive(f, lane), pi = warp_inclusive(need, lane);
    if (lane == 31) {
      part[0][warp] = ri;
      part[1][warp] = pi;
    }
    __syncthreads();
    if (warp == 0) {
      const int64_t x = part[0][lane], y = part[1][lane];
      const int64_t xs = warp_inclusive(x, lane) - x, ys = warp_inclusive(y, lane) - y;
      part[0][lane] = xs;
      part[1][lane] = ys;
    }
    __syncthreads();
    rows[tid] = row0 + part[0][warp] + ri - f;
    pages[tid] = page0 + part[1][warp] + pi - need;
    held[tid] = c;
    if (tid == kTabThreads - 1) {
      rows[kTabThreads] = row0 + part[0][warp] + ri;
      pages[kTabThreads] = page0 + part[1][warp] + pi;
    }
    __syncthreads();
    if ((b0 / kTabThreads) % int(gridDim.x) == int(blockIdx.x) && tid < n) {
      a.seq_lens[b0 + tid] = c + f;
      a.row_start[b0 + tid] = saturate32(rows[tid]);
    }
    const int64_t row1 = rows[kTabThreads], page1 = pages[kTabThreads];
    // this block's rows of [row0, row1), those below n_slots
    const int64_t row_end = row1 < a.n_slots ? row1 : a.n_slots;
    for (int64_t base = row0 / step * step + int64_t(blockIdx.x) * kTabThreads; base < row_end;
         base += step) {
      const int64_t r = base + tid;
      if (r < row0 || r >= row_end) continue;
      const int i = last_at_most(rows, n, r);
      const int64_t pos = held[i] + (r - rows[i]);
      const int32_t pg = int32_t(a.page.div(uint32_t(pos)));
      const int32_t at = held[i] ? int32_t(a.page.div(uint32_t(held[i] - 1))) + 1 : 0;
      int32_t id = -1;
      if (pg < a.max_pages) {
        if (pg < at) {
          if (a.dbg_entry(int64_t(b0) + i, pg)) id = a.table[(int64_t(b0) + i) * a.max_pages + pg];
        } else {
          const int64_t k = pages[i] + (pg - at);
          id = k < a.n_free ? a.free_pages[k] : -1;
        }
      }
      if (!dbg_ok(r >= 0 && r < a.n_slots, a.guard)) continue;
      a.slots[r] = id >= 0 ? int64_t(id) * a.page.d + (pos - int64_t(pg) * a.page.d) : -1;
    }
    // this block's pages of [page0, page1)
    for (int64_t base = page0 / step * step + int64_t(blockIdx.x) * kTabThreads; base < page1;
         base += step) {
      const int64_t k = base + tid;
      if (k < page0 || k >= page1) continue;
      const int i = last_at_most(pages, n, k);
      const int32_t at = held[i] ? int32_t(a.page.div(uint32_t(held[i] - 1))) + 1 : 0;
      if (!a.dbg_entry(int64_t(b0) + i, at + (k - pages[i]))) continue;
      a.table[(int64_t(b0) + i) * a.max_pages + at + (k - pages[i])] =
          k < a.n_free ? a.free_pages[k] : -1;
    }
    row0 = row1;
    page0 = page1;
    __syncthreads();   // the scan is read before the next chunk overwrites it
  }
  // rows behind the last sequence's, and the totals
  for (int64_t base = row0 / step * step + int64_t(blockIdx.x) * kTabThreads; base < a.n_slots;
       base += step)
    if (base + tid >= row0 && base + tid < a.n_slots) a.slots[base + tid] = -1;
  if (blockIdx.x == 0 && tid == 0) {
    a.row_start[a.n_seq] = saturate32(row0);
    a.counts[0] = saturate32(page0 < a.n_free ? page0 : a.n_free);
    a.counts[1] = saturate32(page0);
    a.counts[2] = saturate32(row0);
  }
}

int launch_block_tables(const BlockTablesCall& c) {
  TableArgs a{int32_t(c.n_seq), c.cached_lens, c.new_lens, FastDiv::make(uint32_t(c.page_size)),
              c.free_pages,     c.n_free,      c.block_table, int32_t(c.max_pages), c.slots,
              c.n_slots,        c.seq_lens,    c.row_start,   c.counts,
              kDebugChecks ? Runtime::guard_word() : nullptr};
  if (kDebugChecks && !a.guard) return SRFTQ_ERR_CUDA;
  // a block for each 1024 slots, up to two per SM (each scans all lengths)
  const int64_t want = (c.n_slots + kTabThreads - 1) / kTabThreads;
  const int64_t cap = 2 * int64_t(Runtime::num_sms());
  const int grid = int(want < 1 ? 1 : want < cap ? want : cap);
  block_tables_kernel<<<grid, kTabThreads, 0, c.stream>>>(a);
  return finish_launch();
}

}  // namespace srftq

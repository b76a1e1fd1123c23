// The paged cache as the kernels see it, and the rows a query of
// csa2_attend_paged sees in it.
//
// Row p of sequence b lies in page table[b][p >> page_shift], at row
// p & (page_size - 1) of that page. A table entry outside [0, n_pages) holds
// no rows: a query that should see one records CSA2_FLAG_BAD_PAGE and skips it.
#pragma once
#include "common.cuh"

namespace csa2 {

struct PagedView {
  uint8_t* pages;        // codes of page 0
  uint8_t* scales;       // scales of page 0 (fp8 / fp4)
  int64_t page_stride;   // bytes from one page's codes to the next page's
  int64_t scale_stride;  // the same for the scales
  const int32_t* table;  // [n_seq][table_ld], the first max_pages entries of a row in use
  int64_t table_ld;
  int32_t max_pages;
  int32_t n_pages;
  int32_t page_shift;
  int32_t n_seq;
};

// Page of position p >= 0 of sequence b, -1 where the table has none.
__device__ __forceinline__ int32_t page_of(const PagedView& v, int b, int64_t p) {
  const int64_t j = p >> v.page_shift;
  if (j >= v.max_pages) return -1;
  const int32_t g = v.table[(int64_t)b * v.table_ld + j];
  return (uint32_t)g < (uint32_t)v.n_pages ? g : -1;
}

// What one query sees: the first tokens [lo, lo + head) and [tail, t]. Its
// rows are taken in chunks, aligned runs of 2^shift positions that lie in one
// page (chunk_shift): first the chunks that the first tokens touch, then those
// of [tail, t] that are left. Rows of a chunk that the query does not see are
// masked. Positions are 32 bits: a table holds at most 2^30 rows, and what lies
// past them is cut to that first (64-bit ones cost 2% of a window's decode).
struct Visible {
  int32_t lo, tail, end;  // end: one past the last position (t + 1, or the table's end)
  int32_t head;           // first tokens seen
  int32_t head_chunk, n_head, tail_chunk, n_chunks;
  bool past_table;  // t lies beyond the table's last column: those rows are not there
};

// rows of a chunk: a page, or 64 rows of a larger one
__host__ __device__ __forceinline__ int chunk_shift(int page_shift) { return page_shift < 6 ? page_shift : 6; }

// t >= -1; cap: rows of the table, at most 2^30
__host__ __device__ __forceinline__ Visible visible_rows(int64_t t, int64_t lo_in, int64_t window, int64_t n_first,
                                                         int32_t cap, int shift) {
  Visible s;
  s.lo = lo_in > 0 ? (lo_in < cap ? (int32_t)lo_in : cap) : 0;
  s.past_table = t >= cap;
  s.end = s.past_table ? cap : (int32_t)t + 1;
  s.head = 0;
  s.tail = s.lo;
  s.head_chunk = s.n_head = s.tail_chunk = s.n_chunks = 0;
  if (s.end <= s.lo) return s;
  if (window > 0) {
    const int32_t all = s.end - s.lo;
    s.head = n_first < all ? (int32_t)n_first : all;
    // the window counts from t itself; a window that starts inside the first
    // tokens continues after them, so that no row is seen twice
    const int64_t from = t - window + 1;
    s.tail = s.lo + s.head;
    if (from > s.tail) s.tail = from < cap ? (int32_t)from : cap;
  }
  if (s.head > 0) {
    s.head_chunk = s.lo >> shift;
    s.n_head = ((s.lo + s.head - 1) >> shift) - s.head_chunk + 1;
  }
  s.n_chunks = s.n_head;
  if (s.end > s.tail) {
    const int32_t first = s.tail >> shift, after = s.head_chunk + s.n_head;
    s.tail_chunk = s.n_head > 0 && after > first ? after : first;
    s.n_chunks += ((s.end - 1) >> shift) - s.tail_chunk + 1;
  }
  return s;
}

// Position of row r of the query's chunk k < n_chunks, and whether it is seen.
__host__ __device__ __forceinline__ int32_t chunk_pos(const Visible& s, int k, int r, int shift) {
  const int32_t c = k < s.n_head ? s.head_chunk + k : s.tail_chunk + (k - s.n_head);
  return (c << shift) + r;
}
__host__ __device__ __forceinline__ bool is_seen(const Visible& s, int32_t p) {
  return (p >= s.lo && p < s.lo + s.head) || (p >= s.tail && p < s.end);
}

}  // namespace csa2

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

// The rows one query sees, packed: the first tokens [lo, lo + head), then
// [tail, t]. Packed row i < count is position lo + i or tail + i - head.
struct Visible {
  int64_t lo, tail;
  int32_t head, count;
  bool past_table;  // t lies beyond the table's last column: those rows are not there
};

__host__ __device__ __forceinline__ Visible visible_rows(int64_t t, int64_t lo_in, int64_t window, int64_t n_first, int64_t cap) {
  Visible s;
  s.lo = lo_in > 0 ? lo_in : 0;
  s.past_table = t >= cap;
  const int64_t te = s.past_table ? cap - 1 : t;
  s.head = 0;
  s.tail = s.lo;
  s.count = 0;
  if (te < s.lo) return s;
  if (window > 0) {
    const int64_t all = te - s.lo + 1;
    s.head = (int32_t)(n_first < all ? n_first : all);
    // the window counts from t itself; a window that starts inside the first
    // tokens continues after them, so that no row is seen twice
    const int64_t from = t - window + 1;
    s.tail = s.lo + s.head > from ? s.lo + s.head : from;
  }
  if (te >= s.tail) s.count = s.head + (int32_t)(te - s.tail + 1);
  else s.count = s.head;
  return s;
}

__host__ __device__ __forceinline__ int64_t visible_pos(const Visible& s, int i) {
  return i < s.head ? s.lo + i : s.tail + (i - s.head);
}

}  // namespace csa2

// Page pools, plans and the arrays their pages lie in, as the kernels of
// k_pages.cu see them.
#pragma once
#include "common.cuh"

namespace csa2 {

struct PagePool {
  int32_t* table;  // [n_seq][table_ld]; -1: no page
  int64_t table_ld;
  int64_t* seq_len;  // [n_seq] tokens
  int32_t* ref;      // [n_pages] table entries that name the page; 0: free
  int32_t n_seq, max_pages, n_pages, page_shift;
  uint32_t* flags;
};

struct PageArray {
  uint8_t* base;
  int64_t stride;  // bytes from one page to the next
  int32_t row_bytes;
  int32_t wide;  // base, stride and the chunks start on 16 bytes
};

struct PageArrays {
  int32_t n;
  PageArray a[CSA2_PAGE_ARRAYS_MAX];
};

// workspace of one call
struct PagePlan {
  int32_t *owner, *need, *off;         // [n_seq]
  int32_t *fresh, *src, *rows, *map;   // [n_pages]
  int32_t* count;                      // [4]
};

}  // namespace csa2

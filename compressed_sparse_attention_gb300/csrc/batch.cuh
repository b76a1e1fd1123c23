// Arguments of the batch kernels (k_batch.cu).
#pragma once
#include "pages.cuh"

namespace csa2 {

struct BatchParams {
  PagePool pool;
  const int32_t* seqs;   // [n_req]
  const int64_t* n_new;  // [n_req]
  int32_t* table;        // out [n_req][table_ld], the pool's max_pages columns
  int64_t table_ld;
  int64_t* tok_off;      // out [n_req + 1]
  int64_t* first_pos;    // out [n_req]
  int32_t* req_of_tok;   // out [max_tokens]
  int64_t* tok_pos;
  int64_t* tok_slot;
  int64_t max_tokens;
  int n_req;
  int tok_ctas, row_ctas;  // CTAs of the token arrays; of one table row
};

constexpr int kMaxGroupQueries = 4096;
struct GroupParams {
  const int32_t* table;
  int64_t table_ld;
  const int64_t* q_pos;
  const int32_t* seq_of_q;
  int32_t* order;
  int32_t* head;
  int64_t* shared;
  int32_t* n_groups;  // nullable
  uint32_t* flags;
  int n_query, n_seq, max_pages, n_pages, page_shift;
  int columns;  // leading pages that a group's queries share at least
};

}  // namespace csa2

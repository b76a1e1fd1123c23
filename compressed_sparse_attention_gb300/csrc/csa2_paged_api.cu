// Host side of the paged-cache and rotary entry points: argument validation
// and launches.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <string>

#include "ctx.cuh"
#include "launchers.cuh"

namespace {

csa2_status fail(csa2_ctx* c, csa2_status s, const std::string& msg) {
  if (c) c->err = msg;
  return s;
}

csa2_status cuda_fail(csa2_ctx* c, cudaError_t e, const char* where) {
  cudaGetLastError();
  return fail(c, CSA2_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// every pointer a multiple of `size` (a power of two); null ones are
template <class... P>
bool aligned_all(uintptr_t size, const P*... p) {
  return (aligned(p, size) && ...);
}

// A launch goes to the current device: it must be the context's.
csa2_status begin(csa2_ctx* ctx, const char* where) {
  ctx->last_launches = 0;
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(ctx, e, where);
  if (dev != ctx->device)
    return fail(ctx, CSA2_ERR_INVALID_ARG, std::string(where) + ": the context's device must be the current device");
  return CSA2_OK;
}

csa2_status check_ws(csa2_ctx* c, const char* where, const void* ws, size_t have, size_t need) {
  if (ws == nullptr || have < need)
    return fail(c, CSA2_ERR_WORKSPACE,
                std::string(where) + ": workspace too small: need " + std::to_string(need) + " bytes");
  if (!aligned(ws, 256)) return fail(c, CSA2_ERR_INVALID_ARG, std::string(where) + ": workspace must be 256-byte aligned");
  return CSA2_OK;
}

// log2 of a page size that is a power of two in [1, 4096], else -1
int page_shift(int32_t page_size) {
  if (page_size < 1 || page_size > 4096 || (page_size & (page_size - 1)) != 0) return -1;
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

csa2_status check_pages(csa2_ctx* c, const std::string& where, int32_t n_pages, int32_t page_size) {
  if (page_shift(page_size) < 0)
    return fail(c, CSA2_ERR_UNSUPPORTED, where + ": page_size must be a power of two, 1..4096");
  if (n_pages < 1) return fail(c, CSA2_ERR_INVALID_ARG, where + ": n_pages");
  if (n_pages > 1 << 30) return fail(c, CSA2_ERR_UNSUPPORTED, where + ": at most 2^30 pages");
  return CSA2_OK;
}

// the table's shape, common to caches and pools
csa2_status check_table(csa2_ctx* c, const std::string& where, const void* table, int64_t ld, int32_t max_pages,
                        int32_t n_pages, int32_t page_size, int32_t n_seq) {
  if (page_shift(page_size) < 0)
    return fail(c, CSA2_ERR_UNSUPPORTED, where + ": page_size must be a power of two, 1..4096");
  if (n_seq < 1 || n_pages < 1 || max_pages < 1 || ld < max_pages)
    return fail(c, CSA2_ERR_INVALID_ARG, where + ": n_seq, n_pages, max_pages or table_ld");
  // the plans step 32-bit counters past them by up to 4,096 and add one to n_pages
  if (n_seq > 1 << 30 || n_pages > 1 << 30)
    return fail(c, CSA2_ERR_UNSUPPORTED, where + ": at most 2^30 sequences and 2^30 pages");
  if ((int64_t)max_pages * page_size > (int64_t)1 << 30)
    return fail(c, CSA2_ERR_UNSUPPORTED, where + ": a table row may hold at most 2^30 rows");
  if (!table || !aligned(table, 4)) return fail(c, CSA2_ERR_INVALID_ARG, where + ": table");
  return CSA2_OK;
}

// table: whether the call reads it
csa2_status check_kv(csa2_ctx* c, const std::string& where, const csa2_paged_kv* kv, csa2::PagedView* v, bool table = true) {
  if (!kv) return fail(c, CSA2_ERR_INVALID_ARG, where + ": no cache");
  const csa2_status s = table ? check_table(c, where, kv->table, kv->table_ld, kv->max_pages, kv->n_pages, kv->page_size, kv->n_seq)
                              : check_pages(c, where, kv->n_pages, kv->page_size);
  if (s != CSA2_OK) return s;
  const int f = c->cfg.kv_format;
  const int64_t code = f == CSA2_KV_BF16 ? 1024 : (f == CSA2_KV_FP8_E4M3_B32 ? 512 : 256);
  const int64_t scale = f == CSA2_KV_BF16 ? 0 : (f == CSA2_KV_FP8_E4M3_B32 ? 16 : 32);
  if (!kv->pages || !aligned(kv->pages, 16)) return fail(c, CSA2_ERR_INVALID_ARG, where + ": pages must be 16-byte aligned");
  if (kv->page_stride < code * kv->page_size || kv->page_stride % 16 != 0)
    return fail(c, CSA2_ERR_INVALID_ARG, where + ": page_stride must hold a page's codes and be a multiple of 16 bytes");
  if (scale > 0 && (!kv->scales || !aligned(kv->scales, 16) || kv->scale_stride < scale * kv->page_size ||
                    kv->scale_stride % 16 != 0))
    return fail(c, CSA2_ERR_INVALID_ARG,
                where + ": an fp8 / fp4 cache needs 16-byte aligned scales with a scale_stride that holds a page's");
  v->pages = static_cast<uint8_t*>(kv->pages);
  v->scales = kv->scales;
  v->page_stride = kv->page_stride;
  v->scale_stride = kv->scale_stride;
  v->table = kv->table;
  v->table_ld = kv->table_ld;
  v->max_pages = kv->max_pages;
  v->n_pages = kv->n_pages;
  v->page_shift = page_shift(kv->page_size);
  v->n_seq = kv->n_seq;
  return CSA2_OK;
}

csa2_status check_pool(csa2_ctx* c, const std::string& where, const csa2_page_pool* pool, int32_t n, csa2::PagePool* P) {
  if (!pool) return fail(c, CSA2_ERR_INVALID_ARG, where + ": no pool");
  const csa2_status s =
      check_table(c, where, pool->table, pool->table_ld, pool->max_pages, pool->n_pages, pool->page_size, pool->n_seq);
  if (s != CSA2_OK) return s;
  if (!pool->seq_len || !pool->ref || !aligned(pool->seq_len, 8) || !aligned(pool->ref, 4))
    return fail(c, CSA2_ERR_INVALID_ARG, where + ": seq_len or ref");
  if (n < 0 || n > pool->n_seq) return fail(c, CSA2_ERR_INVALID_ARG, where + ": more entries than sequences");
  P->table = pool->table;
  P->table_ld = pool->table_ld;
  P->seq_len = pool->seq_len;
  P->ref = pool->ref;
  P->n_seq = pool->n_seq;
  P->max_pages = pool->max_pages;
  P->n_pages = pool->n_pages;
  P->page_shift = page_shift(pool->page_size);
  P->flags = c->d_flags;
  return CSA2_OK;
}

csa2_status check_arrays(csa2_ctx* c, const std::string& where, int32_t page_size, int32_t n, const csa2_page_array* in,
                         csa2::PageArrays* out) {
  if (n < 0 || (n > 0 && !in)) return fail(c, CSA2_ERR_INVALID_ARG, where + ": arrays");
  if (n > CSA2_PAGE_ARRAYS_MAX)
    return fail(c, CSA2_ERR_UNSUPPORTED, where + ": at most " + std::to_string(CSA2_PAGE_ARRAYS_MAX) + " arrays a call");
  out->n = n;
  for (int i = 0; i < n; ++i) {
    if (!in[i].base || in[i].row_bytes < 1 || in[i].page_stride < (int64_t)in[i].row_bytes * page_size)
      return fail(c, CSA2_ERR_INVALID_ARG, where + ": array " + std::to_string(i));
    out->a[i].base = static_cast<uint8_t*>(in[i].base);
    out->a[i].stride = in[i].page_stride;
    out->a[i].row_bytes = in[i].row_bytes;
    out->a[i].wide = aligned(in[i].base, 16) && in[i].page_stride % 16 == 0 ? 1 : 0;
  }
  return CSA2_OK;
}

// Whether two tensors of the same strides share an element: rows of `width`
// elements at a * outer + b * inner, a < n_outer, b < n_inner, the second
// tensor's `delta` elements on. Rows of one tensor lie apart, inner ones within
// an outer stride; an axis of one has stride 0.
bool share_elements(int64_t delta, int64_t n_outer, int64_t outer, int64_t n_inner, int64_t inner, int64_t width) {
  // the row pairs (difference of a) that can meet leave a rest below a stride,
  // and so do, of those, the ones by b: the two multiples on either side of 0
  auto nearest = [](int64_t rest, int64_t stride, int64_t n, int64_t (&k)[2]) {
    k[0] = k[1] = 0;
    if (stride == 0) return;
    const int64_t down = rest >= 0 ? rest / stride : -((-rest + stride - 1) / stride);
    for (int i = 0; i < 2; ++i) k[i] = std::min(std::max(down + i, 1 - n), n - 1);
  };
  int64_t a[2], b[2];
  nearest(delta, outer, n_outer, a);
  for (const int64_t ka : a) {
    const int64_t rest = delta - ka * outer;
    nearest(rest, inner, n_inner, b);
    for (const int64_t kb : b)
      if (std::abs(rest - kb * inner) < width) return true;
  }
  return false;
}

// Rows of `width` bytes, `stride` apart, that a call reads or writes.
struct Extent {
  uint64_t base, rows, stride, width;
};
template <class T>
Extent extent(const T* p, int64_t n) {
  return Extent{reinterpret_cast<uintptr_t>(p), n > 0 ? 1u : 0u, 0, (uint64_t)std::max<int64_t>(n, 0) * sizeof(T)};
}
Extent extent(const int32_t* table, int64_t rows, int64_t ld, int64_t columns) {
  return Extent{reinterpret_cast<uintptr_t>(table), (uint64_t)rows, 4 * (uint64_t)ld, 4 * (uint64_t)columns};
}
// Whether a and b share a byte; one of them is a single row.
bool meet(const Extent& a, const Extent& b) {
  if (b.rows > 1) return meet(b, a);
  if (a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0 || b.base + b.width <= a.base) return false;
  // the row of a that begins last before b does, and the one behind it
  const uint64_t i = b.base < a.base || a.rows == 1 ? 0 : std::min((b.base - a.base) / a.stride, a.rows - 1);
  const uint64_t at = a.base + i * a.stride;
  if (b.base < at + a.width && at < b.base + b.width) return true;
  return i + 1 < a.rows && b.base < at + a.stride + a.width && at + a.stride < b.base + b.width;
}
// Whether one of the outputs meets another or an input; at most one of the inputs
// and one of the outputs (not compared with each other) have several rows.
template <size_t O, size_t I>
bool any_meet(const Extent (&out)[O], const Extent (&in)[I]) {
  for (size_t i = 0; i < O; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return true;
    for (size_t j = 0; j < I; ++j)
      if (!(out[i].rows > 1 && in[j].rows > 1) && meet(out[i], in[j])) return true;
  }
  return false;
}

}  // namespace

extern "C" {

size_t csa2_attend_paged_workspace_size(const csa2_ctx* ctx, int32_t n_query) {
  return ctx != nullptr && n_query > 0 ? csa2::attend_paged_workspace_bytes(ctx->num_sms) : 0;
}

csa2_status csa2_attend_paged(csa2_ctx* ctx, void* stream, const csa2_paged_kv* kv, int32_t n_query, const uint16_t* q,
                              const int64_t* q_pos, const int32_t* seq_of_q, const int64_t* lo, int64_t window,
                              int64_t n_first, const float* sink, uint16_t* out, float* lse, void* workspace,
                              size_t workspace_bytes) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "attend_paged");
  if (s != CSA2_OK) return s;
  csa2::PagedView v{};
  if ((s = check_kv(ctx, "attend_paged", kv, &v)) != CSA2_OK) return s;
  if (n_query < 0 || window < 0 || n_first < 0)
    return fail(ctx, CSA2_ERR_INVALID_ARG, "attend_paged: n_query, window and n_first must not be negative");
  if (n_query == 0) return CSA2_OK;
  if (!q || !q_pos || !seq_of_q || !out || !aligned_all(16, q, out) || !aligned_all(8, q_pos, lo) || !aligned_all(4, seq_of_q, sink, lse))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "attend_paged: null or misaligned buffer");
  // CTAs that share a query's output dims each read its whole Q: one may store
  // its share of out before another has read q
  const uint64_t qb = reinterpret_cast<uintptr_t>(q), ob = reinterpret_cast<uintptr_t>(out);
  if ((ob > qb ? ob - qb : qb - ob) < (uint64_t)n_query * csa2::kHeads * csa2::kDim * 2)
    return fail(ctx, CSA2_ERR_INVALID_ARG, "attend_paged: out overlaps q");
  s = check_ws(ctx, "attend_paged", workspace, workspace_bytes, csa2::attend_paged_workspace_bytes(ctx->num_sms));
  if (s != CSA2_OK) return s;
  csa2::AttendParams a{};
  a.q = q;
  a.q_pos = q_pos;
  a.seq_of_q = seq_of_q;
  a.sink = sink;
  a.out = out;
  a.lse = lse;
  a.flags = ctx->d_flags;
  a.n_seq = kv->n_seq;
  a.n_query = n_query;
  a.scale_log2 = ctx->cfg.softmax_scale * 1.4426950408889634f;
  a.rp = ctx->rope;
  int nl = 0;
  const cudaError_t e = csa2::launch_attend_paged(reinterpret_cast<cudaStream_t>(stream), ctx->num_sms, ctx->cfg.kv_format,
                                                  a, v, lo, window, n_first, workspace, &nl);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "attend_paged");
  ctx->last_launches = nl;
  return CSA2_OK;
}

csa2_status csa2_append_paged(csa2_ctx* ctx, void* stream, const csa2_paged_kv* kv, int32_t dtype, const void* rows,
                              int64_t n_tokens, const int64_t* tok_off, const int64_t* first_pos) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "append_paged");
  if (s != CSA2_OK) return s;
  csa2::PagedView v{};
  if ((s = check_kv(ctx, "append_paged", kv, &v)) != CSA2_OK) return s;
  if (dtype != CSA2_DTYPE_BF16 && dtype != CSA2_DTYPE_FP32)
    return fail(ctx, CSA2_ERR_UNSUPPORTED, "append_paged: rows must be bf16 or fp32");
  if (n_tokens < 0) return fail(ctx, CSA2_ERR_INVALID_ARG, "append_paged: n_tokens");
  if (n_tokens == 0) return CSA2_OK;
  if (!rows || !tok_off || !first_pos || !aligned(rows, 16) || !aligned_all(8, tok_off, first_pos))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "append_paged: null or misaligned buffer");
  const cudaError_t e = csa2::launch_append_paged(reinterpret_cast<cudaStream_t>(stream), dtype, rows, n_tokens, kv->n_seq,
                                                  tok_off, first_pos, v, ctx->cfg.kv_format, ctx->rope, ctx->d_flags);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "append_paged");
  ctx->last_launches = 1;
  return CSA2_OK;
}

csa2_status csa2_append_slots(csa2_ctx* ctx, void* stream, const csa2_paged_kv* kv, int32_t dtype, const void* rows,
                              int64_t n_tokens, const int64_t* pos, const int64_t* slots) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "append_slots");
  if (s != CSA2_OK) return s;
  csa2::PagedView v{};
  if ((s = check_kv(ctx, "append_slots", kv, &v, false)) != CSA2_OK) return s;
  if (dtype != CSA2_DTYPE_BF16 && dtype != CSA2_DTYPE_FP32)
    return fail(ctx, CSA2_ERR_UNSUPPORTED, "append_slots: rows must be bf16 or fp32");
  if (n_tokens < 0) return fail(ctx, CSA2_ERR_INVALID_ARG, "append_slots: n_tokens");
  if (n_tokens == 0) return CSA2_OK;
  if (!rows || !slots || !aligned(rows, 16) || !aligned_all(8, pos, slots))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "append_slots: null or misaligned buffer");
  const cudaError_t e = csa2::launch_append_slots(reinterpret_cast<cudaStream_t>(stream), dtype, rows, n_tokens, pos, slots, v,
                                                  ctx->cfg.kv_format, ctx->rope, ctx->d_flags);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "append_slots");
  ctx->last_launches = 1;
  return CSA2_OK;
}

csa2_status csa2_batch_tables(csa2_ctx* ctx, void* stream, const csa2_page_pool* pool, int32_t n_req, const int32_t* seqs,
                              const int64_t* n_new, const csa2_batch* batch) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "batch_tables");
  if (s != CSA2_OK) return s;
  csa2::BatchParams p{};
  if ((s = check_pool(ctx, "batch_tables", pool, 0, &p.pool)) != CSA2_OK) return s;
  if (!batch || n_req < 0 || batch->max_tokens < 0) return fail(ctx, CSA2_ERR_INVALID_ARG, "batch_tables: n_req or max_tokens");
  if (n_req > 1 << 20 || batch->max_tokens > (int64_t)1 << 32)
    return fail(ctx, CSA2_ERR_UNSUPPORTED, "batch_tables: at most 2^20 requests and 2^32 tokens");
  if (!batch->tok_off || !aligned(batch->tok_off, 8)) return fail(ctx, CSA2_ERR_INVALID_ARG, "batch_tables: tok_off");
  if (n_req > 0 && (!seqs || !n_new || !batch->table || !batch->first_pos || !aligned_all(4, seqs, batch->table) ||
                    !aligned_all(8, n_new, batch->first_pos) || batch->table_ld < pool->max_pages))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "batch_tables: null or misaligned buffer, or table_ld below the pool's max_pages");
  if (batch->max_tokens > 0 && (!batch->req_of_tok || !batch->tok_pos || !batch->tok_slot || !aligned(batch->req_of_tok, 4) ||
                                !aligned_all(8, batch->tok_pos, batch->tok_slot)))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "batch_tables: null or misaligned token arrays");
  // rows are copied by many CTAs at once: from one table into another
  const uint64_t pb = reinterpret_cast<uintptr_t>(pool->table), bb = reinterpret_cast<uintptr_t>(batch->table);
  const uint64_t pe = pb + 4 * ((uint64_t)(pool->n_seq - 1) * (uint64_t)pool->table_ld + (uint64_t)pool->max_pages);
  const uint64_t be = bb + 4 * ((uint64_t)std::max(n_req - 1, 0) * (uint64_t)batch->table_ld + (uint64_t)pool->max_pages);
  if (n_req > 0 && pb < be && bb < pe) return fail(ctx, CSA2_ERR_INVALID_ARG, "batch_tables: the batch's table overlaps the pool's");
  // and every CTA reads the requests while others write
  const Extent out[] = {extent(batch->table, n_req, batch->table_ld, pool->max_pages), extent(batch->tok_off, n_req + (int64_t)1),
                        extent(batch->first_pos, n_req), extent(batch->req_of_tok, batch->max_tokens),
                        extent(batch->tok_pos, batch->max_tokens), extent(batch->tok_slot, batch->max_tokens)};
  const Extent in[] = {extent(pool->table, pool->n_seq, pool->table_ld, pool->max_pages), extent(pool->seq_len, pool->n_seq),
                       extent(seqs, n_req), extent(n_new, n_req)};
  if (any_meet(out, in)) return fail(ctx, CSA2_ERR_INVALID_ARG, "batch_tables: an output overlaps an input or another output");
  p.seqs = seqs;
  p.n_new = n_new;
  p.table = batch->table;
  p.table_ld = batch->table_ld;
  p.tok_off = batch->tok_off;
  p.first_pos = batch->first_pos;
  p.req_of_tok = batch->req_of_tok;
  p.tok_pos = batch->tok_pos;
  p.tok_slot = batch->tok_slot;
  p.max_tokens = batch->max_tokens;
  p.n_req = n_req;
  int nl = 0;
  const cudaError_t e = csa2::launch_batch_tables(reinterpret_cast<cudaStream_t>(stream), p, &nl);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "batch_tables");
  ctx->last_launches = nl;
  return CSA2_OK;
}

csa2_status csa2_query_groups(csa2_ctx* ctx, void* stream, const int32_t* table, int64_t table_ld, int32_t max_pages,
                              int32_t n_pages, int32_t page_size, int32_t n_seq, int32_t n_query, const int64_t* q_pos,
                              const int32_t* seq_of_q, int64_t min_shared, int32_t* order, int32_t* head, int64_t* shared,
                              int32_t* n_groups) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "query_groups");
  if (s != CSA2_OK) return s;
  if ((s = check_table(ctx, "query_groups", table, table_ld, max_pages, n_pages, page_size, n_seq)) != CSA2_OK) return s;
  if (n_query < 0 || min_shared < 1) return fail(ctx, CSA2_ERR_INVALID_ARG, "query_groups: n_query or min_shared");
  if (n_query > csa2::kMaxGroupQueries)
    return fail(ctx, CSA2_ERR_UNSUPPORTED, "query_groups: at most " + std::to_string(csa2::kMaxGroupQueries) + " queries");
  if (!aligned(n_groups, 4)) return fail(ctx, CSA2_ERR_INVALID_ARG, "query_groups: misaligned n_groups");
  if (n_query == 0) {  // no groups
    if (n_groups == nullptr) return CSA2_OK;
    const cudaError_t e = cudaMemsetAsync(n_groups, 0, sizeof(*n_groups), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? CSA2_OK : cuda_fail(ctx, e, "query_groups");
  }
  if (!q_pos || !seq_of_q || !order || !head || !shared || !aligned_all(8, q_pos, shared) || !aligned_all(4, seq_of_q, order, head))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "query_groups: null or misaligned buffer");
  // (the second launch reads the queries again)
  const Extent out[] = {extent(order, n_query), extent(head, n_query), extent(shared, n_query), extent(n_groups, n_groups ? 1 : 0)};
  const Extent in[] = {extent(table, n_seq, table_ld, max_pages), extent(q_pos, n_query), extent(seq_of_q, n_query)};
  if (any_meet(out, in)) return fail(ctx, CSA2_ERR_INVALID_ARG, "query_groups: an output overlaps an input or another output");
  csa2::GroupParams p{};
  p.table = table;
  p.table_ld = table_ld;
  p.q_pos = q_pos;
  p.seq_of_q = seq_of_q;
  p.order = order;
  p.head = head;
  p.shared = shared;
  p.n_groups = n_groups;
  p.flags = ctx->d_flags;
  p.n_query = n_query;
  p.n_seq = n_seq;
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.page_shift = page_shift(page_size);
  // more columns than a table has: no groups
  p.columns = (int)std::min((min_shared - 1) / page_size + 1, (int64_t)max_pages + 1);
  const cudaError_t e = csa2::launch_query_groups(reinterpret_cast<cudaStream_t>(stream), p);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "query_groups");
  ctx->last_launches = 2;
  return CSA2_OK;
}

size_t csa2_attend_shared_workspace_size(const csa2_ctx* ctx, int32_t n_query) {
  return ctx != nullptr && n_query > 0 ? csa2::attend_shared_workspace_bytes(ctx->num_sms, n_query) : 0;
}

csa2_status csa2_attend_shared(csa2_ctx* ctx, void* stream, const csa2_paged_kv* kv, int32_t n_query, const uint16_t* q,
                               const int64_t* q_pos, const int32_t* seq_of_q, const int32_t* order, const int32_t* head,
                               const int64_t* shared, const float* sink, uint16_t* out, float* lse, void* workspace,
                               size_t workspace_bytes) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "attend_shared");
  if (s != CSA2_OK) return s;
  csa2::PagedView v{};
  if ((s = check_kv(ctx, "attend_shared", kv, &v)) != CSA2_OK) return s;
  if (n_query < 0) return fail(ctx, CSA2_ERR_INVALID_ARG, "attend_shared: n_query must not be negative");
  if (n_query > 1 << 20) return fail(ctx, CSA2_ERR_UNSUPPORTED, "attend_shared: at most 2^20 queries");
  if (n_query == 0) return CSA2_OK;
  if (!q || !q_pos || !seq_of_q || !order || !head || !shared || !out || !aligned_all(16, q, out) ||
      !aligned_all(8, q_pos, shared) || !aligned_all(4, seq_of_q, order, head, sink, lse))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "attend_shared: null or misaligned buffer");
  // a pair of CTAs may store one query's out before another has read its q
  const uint64_t qb = reinterpret_cast<uintptr_t>(q), ob = reinterpret_cast<uintptr_t>(out);
  if ((ob > qb ? ob - qb : qb - ob) < (uint64_t)n_query * csa2::kHeads * csa2::kDim * 2)
    return fail(ctx, CSA2_ERR_INVALID_ARG, "attend_shared: out overlaps q");
  s = check_ws(ctx, "attend_shared", workspace, workspace_bytes, csa2::attend_shared_workspace_bytes(ctx->num_sms, n_query));
  if (s != CSA2_OK) return s;
  csa2::AttendParams a{};
  a.q = q;
  a.q_pos = q_pos;
  a.seq_of_q = seq_of_q;
  a.sink = sink;
  a.out = out;
  a.lse = lse;
  a.flags = ctx->d_flags;
  a.n_seq = kv->n_seq;
  a.n_query = n_query;
  a.scale_log2 = ctx->cfg.softmax_scale * 1.4426950408889634f;
  a.rp = ctx->rope;
  int nl = 0;
  const cudaError_t e = csa2::launch_attend_shared(reinterpret_cast<cudaStream_t>(stream), ctx->num_sms, ctx->cfg.kv_format,
                                                   a, v, order, head, shared, workspace, &nl);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "attend_shared");
  ctx->last_launches = nl;
  return CSA2_OK;
}

size_t csa2_pages_workspace_size(const csa2_ctx* ctx, const csa2_page_pool* pool) {
  if (!ctx || !pool || pool->n_seq < 1 || pool->n_pages < 1) return 0;
  return csa2::pages_workspace_bytes(pool->n_seq, pool->n_pages);
}

csa2_status csa2_pages_extend(csa2_ctx* ctx, void* stream, const csa2_page_pool* pool, int32_t n, const int32_t* seqs,
                              const int64_t* new_len, void* workspace, size_t workspace_bytes) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "pages_extend");
  if (s != CSA2_OK) return s;
  csa2::PagePool P{};
  if ((s = check_pool(ctx, "pages_extend", pool, n, &P)) != CSA2_OK) return s;
  if (n == 0) return CSA2_OK;
  if (!seqs || !new_len || !aligned(seqs, 4) || !aligned(new_len, 8))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "pages_extend: null or misaligned buffer");
  s = check_ws(ctx, "pages_extend", workspace, workspace_bytes, csa2::pages_workspace_bytes(P.n_seq, P.n_pages));
  if (s != CSA2_OK) return s;
  const cudaError_t e = csa2::launch_pages_extend(reinterpret_cast<cudaStream_t>(stream), P, n, seqs, new_len, workspace);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "pages_extend");
  ctx->last_launches = 1;
  return CSA2_OK;
}

csa2_status csa2_pages_fork(csa2_ctx* ctx, void* stream, const csa2_page_pool* pool, int32_t n, const int32_t* parents,
                            const int32_t* children, int32_t deep, int32_t n_arrays, const csa2_page_array* arrays,
                            void* workspace, size_t workspace_bytes) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "pages_fork");
  if (s != CSA2_OK) return s;
  csa2::PagePool P{};
  csa2::PageArrays A{};
  if ((s = check_pool(ctx, "pages_fork", pool, n, &P)) != CSA2_OK) return s;
  if ((s = check_arrays(ctx, "pages_fork", pool->page_size, n_arrays, arrays, &A)) != CSA2_OK) return s;
  if (n == 0) return CSA2_OK;
  if (!parents || !children || !aligned_all(4, parents, children))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "pages_fork: null or misaligned buffer");
  s = check_ws(ctx, "pages_fork", workspace, workspace_bytes, csa2::pages_workspace_bytes(P.n_seq, P.n_pages));
  if (s != CSA2_OK) return s;
  const cudaError_t e = csa2::launch_pages_fork(reinterpret_cast<cudaStream_t>(stream), ctx->num_sms, P, n, parents,
                                                children, deep != 0, A, workspace);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "pages_fork");
  ctx->last_launches = 2;
  return CSA2_OK;
}

static csa2_status do_free(csa2_ctx* ctx, const char* where, void* stream, const csa2_page_pool* pool, int32_t n,
                           const int32_t* seqs, int64_t window, int64_t n_first, const int64_t* lo) {
  csa2_status s = begin(ctx, where);
  if (s != CSA2_OK) return s;
  csa2::PagePool P{};
  if ((s = check_pool(ctx, where, pool, n, &P)) != CSA2_OK) return s;
  if (n == 0) return CSA2_OK;
  if (!seqs || !aligned(seqs, 4) || !aligned(lo, 8))
    return fail(ctx, CSA2_ERR_INVALID_ARG, std::string(where) + ": null or misaligned buffer");
  const cudaError_t e = csa2::launch_pages_free(reinterpret_cast<cudaStream_t>(stream), P, n, seqs, window, n_first, lo);
  if (e != cudaSuccess) return cuda_fail(ctx, e, where);
  ctx->last_launches = 1;
  return CSA2_OK;
}

csa2_status csa2_pages_free(csa2_ctx* ctx, void* stream, const csa2_page_pool* pool, int32_t n, const int32_t* seqs) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  return do_free(ctx, "pages_free", stream, pool, n, seqs, -1, 0, nullptr);
}

csa2_status csa2_pages_trim(csa2_ctx* ctx, void* stream, const csa2_page_pool* pool, int32_t n, const int32_t* seqs,
                            int64_t window, int64_t n_first, const int64_t* lo) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  if (window < 1 || n_first < 0) {
    ctx->last_launches = 0;
    return fail(ctx, CSA2_ERR_INVALID_ARG, "pages_trim: window must be positive and n_first not negative");
  }
  // beyond any table's rows the sums below would only overflow
  const int64_t cap = (int64_t)1 << 40;
  return do_free(ctx, "pages_trim", stream, pool, n, seqs, std::min(window, cap), std::min(n_first, cap), lo);
}

csa2_status csa2_pages_compact(csa2_ctx* ctx, void* stream, const csa2_page_pool* pool, int32_t n_arrays,
                               const csa2_page_array* arrays, int32_t* n_live, void* workspace,
                               size_t workspace_bytes) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "pages_compact");
  if (s != CSA2_OK) return s;
  csa2::PagePool P{};
  csa2::PageArrays A{};
  if ((s = check_pool(ctx, "pages_compact", pool, 0, &P)) != CSA2_OK) return s;
  if ((s = check_arrays(ctx, "pages_compact", pool->page_size, n_arrays, arrays, &A)) != CSA2_OK) return s;
  if (!aligned(n_live, 4)) return fail(ctx, CSA2_ERR_INVALID_ARG, "pages_compact: misaligned buffer");
  s = check_ws(ctx, "pages_compact", workspace, workspace_bytes, csa2::pages_workspace_bytes(P.n_seq, P.n_pages));
  if (s != CSA2_OK) return s;
  const cudaError_t e = csa2::launch_pages_compact(reinterpret_cast<cudaStream_t>(stream), ctx->num_sms, P, A, n_live, workspace);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "pages_compact");
  ctx->last_launches = 2;
  return CSA2_OK;
}

csa2_status csa2_rope_table_init(csa2_rope_table* t, int32_t rope_dim, int32_t offset, int32_t layout, double theta,
                                 int32_t scaling, double factor, double orig_len, double beta_fast, double beta_slow,
                                 double amplitude) {
  if (!t) return CSA2_ERR_INVALID_ARG;
  std::memset(t, 0, sizeof(*t));
  if (rope_dim < 0 || rope_dim > 2 * CSA2_ROPE_MAX_PAIRS || (rope_dim & 1) || offset < 0 || (offset & 1))
    return CSA2_ERR_UNSUPPORTED;
  if (layout != CSA2_ROPE_INTERLEAVED && layout != CSA2_ROPE_HALF) return CSA2_ERR_INVALID_ARG;
  if (scaling < CSA2_ROPE_NONE || scaling > CSA2_ROPE_YARN) return CSA2_ERR_INVALID_ARG;
  if (!(theta > 0) || !std::isfinite(theta) || !(factor >= 1) || !std::isfinite(factor) || !std::isfinite(amplitude))
    return CSA2_ERR_INVALID_ARG;
  if (scaling == CSA2_ROPE_YARN &&
      (!(theta > 1) || !(orig_len > 0) || !std::isfinite(orig_len) || !(beta_fast > 0) || !(beta_slow > 0)))
    return CSA2_ERR_INVALID_ARG;
  t->rope_dim = rope_dim;
  t->offset = offset;
  t->layout = layout;
  t->amplitude = amplitude;
  if (scaling == CSA2_ROPE_NTK && rope_dim > 2) theta *= std::pow(factor, (double)rope_dim / (rope_dim - 2));
  const bool yarn = scaling == CSA2_ROPE_YARN;
  csa2::rope_frequencies(rope_dim, theta, yarn ? factor : 1.0, orig_len, beta_fast, beta_slow, t->freq);
  if (scaling == CSA2_ROPE_LINEAR)
    for (int i = 0; i < rope_dim / 2; ++i) t->freq[i] /= factor;
  return CSA2_OK;
}

csa2_status csa2_rope(csa2_ctx* ctx, void* stream, const csa2_rope_table* table, int32_t dtype, int64_t n_tokens,
                      int32_t n_heads, int32_t head_dim, const void* x, int64_t x_tok_stride, int64_t x_head_stride,
                      const int64_t* pos, void* out, int64_t out_tok_stride, int64_t out_head_stride,
                      int32_t transpose) {
  if (!ctx) return CSA2_ERR_INVALID_ARG;
  csa2_status s = begin(ctx, "rope");
  if (s != CSA2_OK) return s;
  if (!table) return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: no table");
  if (dtype < CSA2_DTYPE_BF16 || dtype > CSA2_DTYPE_FP32) return fail(ctx, CSA2_ERR_UNSUPPORTED, "rope: dtype");
  if (n_tokens < 0 || n_heads < 0 || x_tok_stride < 0 || x_head_stride < 0 || out_tok_stride < 0 || out_head_stride < 0)
    return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: negative size or stride");
  if (head_dim < 2 || head_dim > 1024 || (head_dim & 1) || n_heads > 65535)
    return fail(ctx, CSA2_ERR_UNSUPPORTED, "rope: head_dim must be even, 2..1024, and n_heads at most 65535");
  if (table->rope_dim < 0 || table->rope_dim > 2 * CSA2_ROPE_MAX_PAIRS || (table->rope_dim & 1) || table->offset < 0 ||
      (table->offset & 1) || (int64_t)table->offset + table->rope_dim > head_dim)
    return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: the table's channels must lie inside the head");
  if (table->layout != CSA2_ROPE_INTERLEAVED && table->layout != CSA2_ROPE_HALF)
    return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: the table's layout");
  if (!std::isfinite(table->amplitude)) return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: the table's amplitude");
  for (int k = 0; k < table->rope_dim / 2; ++k)
    if (!(std::fabs(table->freq[k]) < 4294967296.0))
      return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: a frequency of the table is not finite or 2^32 and more");
  if (n_tokens == 0 || n_heads == 0) return CSA2_OK;
  const uintptr_t size = dtype == CSA2_DTYPE_FP32 ? 4 : 2;
  if (!x || !out || !pos || !aligned_all(size, x, out) || !aligned(pos, 8))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: null or misaligned buffer");
  // strides of axes of one are never used
  if (n_tokens == 1) x_tok_stride = out_tok_stride = 0;
  if (n_heads == 1) x_head_stride = out_head_stride = 0;
  // extents are sums of products below 2^63
  const double far = (double)n_tokens * (double)std::max(x_tok_stride, out_tok_stride) +
                     (double)n_heads * (double)std::max(x_head_stride, out_head_stride);
  if (far > 0x1p56) return fail(ctx, CSA2_ERR_UNSUPPORTED, "rope: a tensor of more than 2^56 elements");
  const bool in_place = out == x;
  if (in_place && (x_tok_stride != out_tok_stride || x_head_stride != out_head_stride))
    return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: in place, x and out must have the same strides");
  // the rows of out must lie apart: each axis strides over a row at least, and
  // one of them over the other's whole extent
  const int64_t tok_span = (n_tokens - 1) * out_tok_stride + head_dim, head_span = (n_heads - 1) * out_head_stride + head_dim;
  const bool tok_ok = n_tokens == 1 || out_tok_stride >= head_dim, head_ok = n_heads == 1 || out_head_stride >= head_dim;
  const bool apart = tok_ok && head_ok &&
                     (n_tokens == 1 || n_heads == 1 || out_tok_stride >= head_span || out_head_stride >= tok_span);
  if (!apart) return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: out's rows overlap each other");
  if (!in_place) {
    const uintptr_t xb = reinterpret_cast<uintptr_t>(x), ob = reinterpret_cast<uintptr_t>(out);
    const uintptr_t xe = xb + size * ((n_tokens - 1) * x_tok_stride + (n_heads - 1) * x_head_stride + head_dim);
    const uintptr_t oe = ob + size * ((n_tokens - 1) * out_tok_stride + (n_heads - 1) * out_head_stride + head_dim);
    if (xb < oe && ob < xe) {
      // one inside the other's span: parts of one buffer, as the queries and keys of a fused projection, lie apart
      if (x_tok_stride != out_tok_stride || x_head_stride != out_head_stride)
        return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: x and out of different strides lie within each other's span");
      const int64_t delta = ((int64_t)ob - (int64_t)xb) / (int64_t)size;
      const bool tok_outer = n_heads == 1 || (n_tokens > 1 && out_tok_stride >= head_span);
      if (tok_outer ? share_elements(delta, n_tokens, out_tok_stride, n_heads, out_head_stride, head_dim)
                    : share_elements(delta, n_heads, out_head_stride, n_tokens, out_tok_stride, head_dim))
        return fail(ctx, CSA2_ERR_INVALID_ARG, "rope: x and out overlap without being the same");
    }
  }
  int nl = 0;
  const cudaError_t e = csa2::launch_rope(reinterpret_cast<cudaStream_t>(stream), ctx->num_sms, *table, dtype, x, out, pos,
                                          n_tokens, n_heads, head_dim, x_tok_stride, x_head_stride, out_tok_stride,
                                          out_head_stride, transpose != 0, in_place, &nl);
  if (e != cudaSuccess) return cuda_fail(ctx, e, "rope");
  ctx->last_launches = nl;
  return CSA2_OK;
}

}  // extern "C"

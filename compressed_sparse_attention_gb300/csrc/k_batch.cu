// The tables of a batch, made on the device from its requests' lengths
// (csa2_batch_tables), and the groups of its queries whose sequences share
// leading pages (csa2_query_groups).
#include <algorithm>

#include "launchers.cuh"

namespace csa2 {

namespace {

constexpr int kBatchThreads = 256;
constexpr int kBatchReqs = 1024;   // requests whose offsets lie in shared memory at once
constexpr int kTokThreads = 4;     // tokens of a thread
constexpr int kRowCols = 2048;     // table columns of a CTA
// Scans of 1,024 requests that token CTAs make between them at most; where it would
// be more, CTA 0 alone scans, and the others search its offsets behind a second
// launch. Scans by all and search: 16 x 16 scans (16,384 requests, as many tokens)
// 45.5 and 56.5 us, 3 x 98 11.8 and 18.8, 4 x 977 26.4 and 25.9, 64 x 64 180 and 186,
// 8 x 977 46.0 and 37.0, 64 x 1,024 340 and 198.
constexpr int64_t kMostScans = 4096;

// Request i: its sequence (-1: none, or not to be carried out), its length and new tokens.
struct Request {
  int32_t seq;
  int64_t len, n_new;
};
__device__ __forceinline__ Request request_at(const BatchParams& p, int i, uint32_t& bad) {
  Request r{p.seqs[i], 0, 0};
  if (r.seq >= 0 && r.seq < p.pool.n_seq) {
    r.len = p.pool.seq_len[r.seq];
    r.n_new = p.n_new[i];
    const int64_t cap = (int64_t)p.pool.max_pages << p.pool.page_shift;
    if (r.n_new >= 0 && r.n_new <= r.len && r.len <= cap) return r;
  }
  if (r.seq != -1) bad |= CSA2_FLAG_BAD_SEQ;
  return Request{-1, 0, 0};
}
// Place t of the token arrays: token at pos of request i, sequence seq.
__device__ __forceinline__ void put_token(const BatchParams& p, int64_t t, int i, int32_t seq, int64_t pos, uint32_t& bad) {
  const int32_t page = p.pool.table[(int64_t)seq * p.pool.table_ld + (pos >> p.pool.page_shift)];
  const bool there = (uint32_t)page < (uint32_t)p.pool.n_pages;
  if (!there) bad |= CSA2_FLAG_BAD_PAGE;
  p.req_of_tok[t] = i;
  p.tok_pos[t] = pos;
  p.tok_slot[t] = there ? ((int64_t)page << p.pool.page_shift) + (pos & ((1 << p.pool.page_shift) - 1)) : -1;
}
__device__ __forceinline__ void put_padding(const BatchParams& p, int64_t t) {
  p.req_of_tok[t] = -1;
  p.tok_pos[t] = -1;
  p.tok_slot[t] = -1;
}

}  // namespace

// csa2_batch_tables. CTAs below p.tok_ctas take 1,024 places of the token arrays
// each, every one with a scan of its own over the requests up to the last that has
// a token there (the lengths of 1,024 requests come from the L2 in two round trips,
// which up to as many requests is what the call takes; a scan in a launch of its own
// would add one more); CTA 0 scans all, for the offsets. The others copy table
// rows. 64 requests 3.7 us (3.5 in a graph), 512 with rows of 2,050 columns 5.8 us;
// launched plainly instead of programmatically 6.2 and 8.3. Each further 1,024
// requests are 2.8 us of CTA 0.
__global__ void __launch_bounds__(kBatchThreads) batch_tables_kernel(const __grid_constant__ BatchParams p) {
  __shared__ int64_t off[kBatchReqs + 1];
  __shared__ int64_t first[kBatchReqs];
  __shared__ int32_t seq_of[kBatchReqs];
  __shared__ int64_t sums[kBatchThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t bad = 0;
  pdl_trigger();
  pdl_wait();
  if ((int)blockIdx.x >= p.tok_ctas) {
    const int64_t at = (int64_t)blockIdx.x - p.tok_ctas;
    const int i = (int)(at / p.row_ctas), c0 = (int)(at % p.row_ctas) * kRowCols;
    const Request r = request_at(p, i, bad);
    const int64_t used = r.seq < 0 ? 0 : (r.len + (1 << p.pool.page_shift) - 1) >> p.pool.page_shift;
    const int32_t* src = p.pool.table + (int64_t)max(r.seq, 0) * p.pool.table_ld;
    int32_t* dst = p.table + (int64_t)i * p.table_ld;
#pragma unroll 4
    for (int j = c0 + tid; j < min(c0 + kRowCols, p.pool.max_pages); j += kBatchThreads) dst[j] = j < used ? src[j] : -1;
    return;
  }
  const int64_t t0 = (int64_t)blockIdx.x * kBatchThreads * kTokThreads;
  constexpr int kPer = kBatchReqs / kBatchThreads;
  int64_t before = 0;  // tokens of the requests so far
  bool full = false;
  if (blockIdx.x == 0 && tid == 0) p.tok_off[0] = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < p.n_req; i0 += kBatchReqs) {
    Request r[kPer];
    int64_t mine = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = i0 + kPer * tid + k;
      r[k] = i < p.n_req ? request_at(p, i, bad) : Request{-1, 0, 0};
      mine += r[k].n_new;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();  // (also: the last requests' places have been searched)
    int64_t at = before + incl - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kBatchThreads / 32; ++w) {
      if (w < warp) at += sums[w];
      all += sums[w];
    }
    // A request whose tokens do not all fit has none, nor has any later one:
    // the next one's offset is the end of the last that fits.
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int e = kPer * tid + k;
      off[e] = full ? before : at;
      first[e] = r[k].len - r[k].n_new;
      seq_of[e] = r[k].seq;
      at += r[k].n_new;
    }
    if (tid == kBatchThreads - 1) off[kBatchReqs] = full ? before : at;
    __syncthreads();
    if (!full && before + all > p.max_tokens) {
      // the first request past the end, by all threads
      int lo = 0, hi = kBatchReqs;  // off[lo] <= max, off[hi] > max
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= p.max_tokens) lo = mid;
        else hi = mid;
      }
      const int64_t end = off[lo];
      __syncthreads();
      for (int e = lo + tid; e <= kBatchReqs; e += kBatchThreads) off[e] = end;
      if (blockIdx.x == 0 && tid == 0) bad |= CSA2_FLAG_BATCH_FULL;
      __syncthreads();
      full = true;
      before = end;
    } else if (!full) {
      before += all;
    }
    const int n = min(kBatchReqs, p.n_req - i0);
    if (blockIdx.x == 0) {
      for (int e = tid; e < n; e += kBatchThreads) {
        p.tok_off[i0 + e + 1] = off[e + 1];
        p.first_pos[i0 + e] = first[e];
      }
    }
#pragma unroll
    for (int k = 0; k < kTokThreads; ++k) {
      const int64_t t = t0 + kBatchThreads * k + tid;
      if (t >= p.max_tokens || t < off[0] || t >= off[n]) continue;
      int lo = 0, hi = n;  // off[lo] <= t < off[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= t) lo = mid;
        else hi = mid;
      }
      put_token(p, t, i0 + lo, seq_of[lo], first[lo] + (t - off[lo]), bad);
    }
    // (CTA 0 goes on to the last request, for the offsets)
    if (blockIdx.x != 0 && (full || before >= t0 + kBatchThreads * kTokThreads)) break;
  }
  // places behind the last token
#pragma unroll
  for (int k = 0; k < kTokThreads; ++k) {
    const int64_t t = t0 + kBatchThreads * k + tid;
    if (t >= before && t < p.max_tokens) put_padding(p, t);
  }
  if (blockIdx.x != 0) bad &= ~(uint32_t)CSA2_FLAG_BAD_SEQ;  // CTA 0 has seen them all
  if (bad) set_flag(p.pool.flags, bad);
}

// Places of the token arrays from `from` on, their requests found by a search in
// the offsets that the launch before has written.
__global__ void __launch_bounds__(kBatchThreads) batch_tokens_kernel(const __grid_constant__ BatchParams p, int64_t from) {
  uint32_t bad = 0;
  pdl_trigger();
  pdl_wait();
  const int64_t used = p.tok_off[p.n_req];
#pragma unroll 1
  for (int k = 0; k < kTokThreads; ++k) {
    const int64_t t = from + ((int64_t)blockIdx.x * kTokThreads + k) * kBatchThreads + threadIdx.x;
    if (t >= p.max_tokens) break;
    if (t >= used) {
      put_padding(p, t);
      continue;
    }
    const int i = find_segment(p.tok_off, p.n_req, t);
    put_token(p, t, i, p.seqs[i], p.first_pos[i] + (t - p.tok_off[i]), bad);
  }
  if (bad) set_flag(p.pool.flags, bad);
}

cudaError_t launch_batch_tables(cudaStream_t st, BatchParams p, int* n_launch) {
  const int64_t per = kBatchThreads * kTokThreads;
  const int64_t tok = p.max_tokens > 0 ? (p.max_tokens + per - 1) / per : 1;
  const int64_t scans = (p.n_req + kBatchReqs - 1) / kBatchReqs;
  const bool search = scans > 1 && tok > 1 && scans * tok > kMostScans;
  p.row_ctas = (p.pool.max_pages + kRowCols - 1) / kRowCols;
  const int64_t ctas = (search ? 1 : tok) + (int64_t)p.n_req * p.row_ctas;
  if (ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  p.tok_ctas = search ? 1 : (int)tok;
  cudaError_t e = launch_ex(batch_tables_kernel, dim3((unsigned)ctas), dim3(kBatchThreads), 0, st, true, 0, p);
  ++*n_launch;
  if (e != cudaSuccess || !search) return e;
  e = launch_ex(batch_tokens_kernel, dim3((unsigned)(tok - 1)), dim3(kBatchThreads), 0, st, true, 0, p, per);
  ++*n_launch;
  return e;
}

// ---------------------------------------------------------------------------
// csa2_query_groups. The first launch, one CTA, finds each query's group by
// its key (the page at the column that min_shared ends in) in a hash table of
// shared memory that keeps the lowest query of each key, and places the
// queries group by group: ranks within a group from sixteen warps' counts. The
// second compares each query's row with its group's first, a warp a query, and
// keeps the least common run. Nothing depends on timing: minima and sums of
// whole numbers. Bound by latency: 64 queries 5.4 us, 2,047 over 313 columns 11.0.
// ---------------------------------------------------------------------------
namespace {

constexpr int kGroupThreads = 1024;
constexpr int kRankWarps = 16;

__device__ __forceinline__ uint32_t hash_slot(int32_t key, uint32_t mask) { return ((uint32_t)key * 2654435761u >> 7) & mask; }

// whole pages that query i sees of its sequence, 0 for a query without one
__device__ __forceinline__ int64_t whole_pages(const GroupParams& p, int i, int32_t& seq) {
  const int32_t b = p.seq_of_q[i];
  const int64_t t = p.q_pos[i];
  seq = b >= 0 && b < p.n_seq && t >= 0 ? b : -1;
  return seq < 0 ? 0 : min((min(t, (int64_t)1 << 40) + 1) >> p.page_shift, (int64_t)p.max_pages);
}

// The columns at which the rows of queries i and j (both keyed: both have
// sequences) name the same page, from the first column on, bounded by the whole
// pages that both see; by a warp.
__device__ __forceinline__ int64_t common_columns(const GroupParams& p, int i, int j, int lane) {
  int32_t seq, first;
  const int64_t mine = whole_pages(p, i, seq);
  const int64_t run = min(mine, whole_pages(p, j, first));
  const int32_t* a = p.table + (int64_t)seq * p.table_ld;
  const int32_t* b = p.table + (int64_t)first * p.table_ld;
  constexpr int kAhead = 4;
  for (int64_t c0 = 0; c0 < run; c0 += 32 * kAhead) {
    int32_t x[kAhead], y[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t c = c0 + 32 * u + lane;
      x[u] = c < run ? a[c] : -1;
      y[u] = c < run ? b[c] : -1;
    }
    int64_t stop = run;
#pragma unroll
    for (int u = kAhead - 1; u >= 0; --u) {
      const uint32_t off = __ballot_sync(0xffffffffu, x[u] != y[u] || (uint32_t)x[u] >= (uint32_t)p.n_pages);
      if (off) stop = min(run, c0 + 32 * u + __ffs((int)off) - 1);
    }
    if (stop < run) return stop;
  }
  return run;
}

}  // namespace

size_t query_groups_smem(int n) {
  int slots = 64;
  while (slots < 2 * n) slots *= 2;
  // lead, size (then start), rank, whole pages; the hash table, whose place the counts take later
  return (size_t)n * 16 + std::max((size_t)slots * 8, (size_t)n * 2 * kRankWarps) + 64;
}

__global__ void __launch_bounds__(kGroupThreads, 1) query_groups_kernel(const __grid_constant__ GroupParams p, int slots) {
  extern __shared__ __align__(16) int32_t sh[];
  const int n = p.n_query, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* lead = sh;
  int32_t* size = sh + n;
  int32_t* rank = sh + 2 * n;
  int32_t* whole = sh + 3 * n;
  int32_t* key = sh + 4 * n;           // [slots]
  int32_t* low = key + slots;          // [slots]
  uint16_t* count = reinterpret_cast<uint16_t*>(key);  // [kRankWarps][n], once the table has been read
  __shared__ int32_t warp_sum[32];
  __shared__ int32_t groups;
  const uint32_t mask = (uint32_t)slots - 1;
  pdl_trigger();
  pdl_wait();
  uint32_t bad = 0;
  for (int s = tid; s < slots; s += kGroupThreads) {
    key[s] = -1;
    low[s] = 0x7FFFFFFF;
  }
  if (tid == 0) groups = 0;
  __syncthreads();
  // a thread's queries together: their keys are two dependent round trips to the L2
  constexpr int kPer = kMaxGroupQueries / kGroupThreads;
  int32_t page[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid + u * kGroupThreads;
    page[u] = -1;
    if (i >= n) continue;
    const int32_t b = p.seq_of_q[i];
    if (b != -1 && (b < 0 || b >= p.n_seq || p.q_pos[i] < -1)) bad |= CSA2_FLAG_BAD_QUERY;
    int32_t seq;
    const int64_t seen = whole_pages(p, i, seq);
    whole[i] = (int32_t)seen;
    if (seen >= p.columns) page[u] = p.table[(int64_t)seq * p.table_ld + p.columns - 1];
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid + u * kGroupThreads;
    if (i >= n) break;
    size[i] = 0;
    lead[i] = i;
    if (page[u] < 0 || page[u] >= p.n_pages) continue;
    uint32_t s = hash_slot(page[u], mask);
    // (at most half of the slots fill: the search ends)
    for (;; s = (s + 1) & mask) {
      const int32_t was = atomicCAS(key + s, -1, page[u]);
      if (was == -1 || was == page[u]) break;
    }
    atomicMin(low + s, i);
    lead[i] = -1 - (int)s;
  }
  if (bad) set_flag(p.flags, bad);
  __syncthreads();
  for (int i = tid; i < n; i += kGroupThreads) {
    if (lead[i] < 0) lead[i] = low[-1 - lead[i]];
    atomicAdd(size + lead[i], 1);
  }
  __syncthreads();
  // counts of a warp's share of the queries, group by group, and each query's rank in them
  static_assert(kRankWarps % 8 == 0);
  for (int s = tid; s < kRankWarps / 8 * n; s += kGroupThreads) reinterpret_cast<uint4*>(count)[s] = make_uint4(0u, 0u, 0u, 0u);
  __syncthreads();
  const int per = ((n + kRankWarps - 1) / kRankWarps + 31) & ~31;
  if (warp < kRankWarps) {
    uint16_t* mine = count + warp * n;
    for (int i0 = warp * per; i0 < min(n, (warp + 1) * per); i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < n;
      const int g = in ? lead[i] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, g);
      const int before = __popc(same & ((1u << lane) - 1));
      int base = 0;
      if (in) base = mine[g];
      __syncwarp();
      if (in) {
        rank[i] = base + before;
        if (before == 0) mine[g] = (uint16_t)(base + __popc(same));
      }
      __syncwarp();
    }
  }
  // places: the groups in the order of their first queries. A thread's share
  // of the queries is contiguous.
  const int share = (n + kGroupThreads - 1) / kGroupThreads, lo = min(n, tid * share), hi = min(n, lo + share);
  int sum = 0, heads = 0;
  for (int i = lo; i < hi; ++i) {
    if (lead[i] == i) {
      sum += size[i];
      ++heads;
    }
  }
  if (heads) atomicAdd(&groups, heads);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int at = incl - sum;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  for (int i = lo; i < hi; ++i) {
    if (lead[i] != i) continue;
    const int many = size[i];
    int before = 0;  // counts -> places of each warp's first
    for (int w = 0; w < kRankWarps; ++w) {
      const int c = count[w * n + i];
      count[w * n + i] = (uint16_t)before;
      before += c;
    }
    size[i] = at;
    p.shared[at] = many > 1 ? (int64_t)whole[i] << p.page_shift : 0;
    at += many;
  }
  __syncthreads();
  // (through shared memory: one SM writes a sector a clock, and places in the
  // order of the queries are a sector each, 3 us for 2,000 of them)
  int32_t place[kPer], start[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid + u * kGroupThreads;
    if (i >= n) break;
    const int g = lead[i];
    start[u] = size[g];
    place[u] = start[u] + count[(i / per) * n + g] + rank[i];
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = tid + u * kGroupThreads;
    if (i >= n) break;
    rank[place[u]] = i;
    whole[place[u]] = start[u];
  }
  __syncthreads();
  for (int k = tid; k < n; k += kGroupThreads) {
    p.order[k] = rank[k];
    p.head[k] = whole[k];
    if (whole[k] != k) p.shared[k] = 0;
  }
  if (tid == 0 && p.n_groups != nullptr) *p.n_groups = groups;
}

// A warp a place: the common run of its query and its group's first.
__global__ void __launch_bounds__(256) query_groups_run_kernel(const __grid_constant__ GroupParams p) {
  const int lane = threadIdx.x & 31, k = (int)blockIdx.x * 8 + (threadIdx.x >> 5);
  pdl_wait();
  if (k >= p.n_query) return;
  const int h = p.head[k];
  if (h == k) return;
  const int64_t run = common_columns(p, p.order[k], p.order[h], lane);
  if (lane == 0) atomicMin(reinterpret_cast<long long*>(p.shared + h), (long long)(run << p.page_shift));
}

cudaError_t launch_query_groups(cudaStream_t st, const GroupParams& p) {
  int slots = 64;
  while (slots < 2 * p.n_query) slots *= 2;
  const size_t smem = query_groups_smem(p.n_query);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(query_groups_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)query_groups_smem(kMaxGroupQueries));
  if (e != cudaSuccess) return e;
  e = launch_ex(query_groups_kernel, dim3(1), dim3(kGroupThreads), smem, st, true, 0, p, slots);
  if (e != cudaSuccess) return e;
  return launch_ex(query_groups_run_kernel, dim3((unsigned)((p.n_query + 7) / 8)), dim3(256), 0, st, true, 0, p);
}

}  // namespace csa2

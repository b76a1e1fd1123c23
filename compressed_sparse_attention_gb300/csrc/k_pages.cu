// Page operations of a paged cache: sequences grow (extend), share or copy
// another's rows (fork), give pages back (free, trim), and the pages in use
// move together (compact). All of it is planned on the device from the tables
// and reference counts, so that a captured graph replays it on what they hold
// then; a page is free when its count is 0, and pages are handed out lowest
// index first, in the order of the call's entries, so that results do not
// depend on timing.
//
// Planning runs in one CTA (a scan over the reference counts; counts and
// offsets of the entries); the work that grows with the call (table rows,
// page copies) in a second launch over all SMs. The copies are bound by
// memory: 2 x the bytes moved.
#include "launchers.cuh"
#include "pages.cuh"

namespace csa2 {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kCopyThreads = 256;
constexpr int kCopyChunk = 16384;  // bytes of a page that a CTA copies in one go: 4 x 16 a thread
constexpr int kNoOwner = 0x7FFFFFFF;
constexpr int kSharedSeqs = 2048;  // sequences whose plan fits shared memory, 24 KB

// What the plan keeps of its entries: in shared memory, which spares it a round
// trip to the L2 after each of its barriers, or for very many sequences in the
// workspace.
struct Entries {
  int32_t *owner, *need, *off;
};
struct EntriesShared {
  int32_t owner[kSharedSeqs], need[kSharedSeqs], off[kSharedSeqs];
};
__device__ __forceinline__ Entries entries_of(const PagePool& P, const PagePlan& W, EntriesShared& sh) {
  return P.n_seq <= kSharedSeqs ? Entries{sh.owner, sh.need, sh.off} : Entries{W.owner, W.need, W.off};
}

// The counts and lengths that the plan reads late, on their way to the L2.
__device__ __forceinline__ void plan_prefetch(const PagePool& P) {
  const int64_t t = threadIdx.x;
  if (t * 32 < P.n_pages) asm volatile("prefetch.global.L2 [%0];" ::"l"(P.ref + t * 32));
  if (t * 16 < P.n_seq) asm volatile("prefetch.global.L2 [%0];" ::"l"(P.seq_len + t * 16));
}

// The plans run once, on instructions that come from memory, each issued as
// often as there are warps: short code, one scan for all of them and 512
// threads (free, fork of 24 children and extend over 2,048 pages: 18.5 us, and
// 20.1 with 1,024 threads and a scan inlined at each place).

// Exclusive scan of one value a thread over the plan's CTA; total: the sum.
// Sums stop at cap (values at most cap, cap below 2^31).
__device__ __noinline__ uint32_t cta_scan(uint32_t x, uint32_t cap, uint32_t* total) {
  __shared__ uint32_t sums[kPlanWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t before = 0;
#pragma unroll
  for (int level = 0; level < 2; ++level) {  // the warp's threads, then the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = min(x + v, cap);
    }
    if (level == 0) {
      const uint32_t left = __shfl_up_sync(0xffffffffu, x, 1);
      before = lane > 0 ? left : 0u;
      if (lane == 31) sums[warp] = x;
      __syncthreads();
      x = lane < kPlanWarps ? sums[lane] : 0u;
    }
  }
  *total = __shfl_sync(0xffffffffu, x, 31);
  const uint32_t left = __shfl_sync(0xffffffffu, x, warp > 0 ? warp - 1 : 0);
  __syncthreads();  // sums is free for the next scan
  return warp > 0 ? min(before + left, cap) : before;
}

// The lowest `want` free pages in ascending order into list; returns how many
// there are (at most want). By the plan's CTA, in rounds of 4 counts a thread,
// or of 16 for pools of more than four such rounds, whose barriers then count
// (a million counts: 0.34 ms with 4).
__device__ int take_free(const PagePool& P, int want, int32_t* list) {
  const int each = P.n_pages > 16 * kPlanThreads ? 16 : 4;
  const bool wide = (reinterpret_cast<uintptr_t>(P.ref) & 15u) == 0;
  int found = 0;
#pragma unroll 1
  for (int64_t base = 0; base < P.n_pages && found < want; base += kPlanThreads * each) {
    const int64_t first = base + (int64_t)threadIdx.x * each;
    uint32_t free_bits = 0;
#pragma unroll 4
    for (int u = 0; u < each; u += 4) {
      const int64_t g = first + u;
      int4 r = make_int4(1, 1, 1, 1);
      if (wide && g + 4 <= P.n_pages) {
        r = *reinterpret_cast<const int4*>(P.ref + g);
      } else {
        if (g < P.n_pages) r.x = P.ref[g];
        if (g + 1 < P.n_pages) r.y = P.ref[g + 1];
        if (g + 2 < P.n_pages) r.z = P.ref[g + 2];
        if (g + 3 < P.n_pages) r.w = P.ref[g + 3];
      }
      free_bits |= (uint32_t)((r.x == 0) | (r.y == 0) << 1 | (r.z == 0) << 2 | (r.w == 0) << 3) << u;
    }
    uint32_t total;
    int at = found + (int)cta_scan(__popc(free_bits), 0x7FFFFFFFu, &total);
    for (; free_bits != 0u && at < want; free_bits &= free_bits - 1) list[at++] = (int32_t)first + __ffs(free_bits) - 1;
    found += (int)total;
  }
  __syncthreads();
  return min(found, want);
}

// Marks every valid sequence named in `seqs` with the first entry naming it.
__device__ void claim(const PagePool& P, const int32_t* seqs, int n, int32_t* owner) {
  int b = (int)threadIdx.x < n ? seqs[threadIdx.x] : -1;  // on its way during the reset
#pragma unroll 1
  for (int k = threadIdx.x; k < P.n_seq; k += kPlanThreads) owner[k] = kNoOwner;
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    if (i >= kPlanThreads) b = seqs[i];
    if (b >= 0 && b < P.n_seq) atomicMin(&owner[b], i);
  }
  __syncthreads();
}

__device__ __forceinline__ int64_t pages_for(const PagePool& P, int64_t len) {
  return (len + (1 << P.page_shift) - 1) >> P.page_shift;
}

__device__ __forceinline__ bool is_page(const PagePool& P, int32_t g) { return (uint32_t)g < (uint32_t)P.n_pages; }

// Offsets of the entries' fresh pages and the pages themselves. need[i] < 0:
// an entry that is not carried out. An entry whose pages are not there, and
// with it every later one that needs any, is refused (need[i] = -1).
__device__ void place_entries(const PagePool& P, const PagePlan& W, const Entries& E, int n) {
  // offsets past the pool mean that the entry is refused below
  const uint32_t cap = (uint32_t)P.n_pages + 1u;
  uint32_t carry = 0;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
    const int i = i0 + (int)threadIdx.x;
    uint32_t total;
    const uint32_t at = cta_scan(i < n ? min((uint32_t)max(E.need[i], 0), cap) : 0u, cap, &total);
    if (i < n) E.off[i] = (int32_t)min(carry + at, cap);
    carry = min(carry + total, cap);
  }
  const int n_free = take_free(P, (int)min(carry, (uint32_t)P.n_pages), W.fresh);
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int need = E.need[i];
    if (need > 0 && (int64_t)E.off[i] + need > n_free) {
      E.need[i] = -1;
      set_flag(P.flags, CSA2_FLAG_OUT_OF_PAGES);
    }
  }
  __syncthreads();
}

// ---------------------------------------------------------------- extend
__global__ void __launch_bounds__(kPlanThreads, 1) pages_extend_kernel(const PagePool P, const PagePlan W, int n,
                                                                    const int32_t* __restrict__ seqs,
                                                                    const int64_t* __restrict__ new_len) {
  __shared__ EntriesShared sh;
  const Entries E = entries_of(P, W, sh);
  plan_prefetch(P);
  claim(P, seqs, n, E.owner);
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    const int b = seqs[i];
    int need = -1;
    if (b >= 0 && b < P.n_seq && E.owner[b] == i) {
      const int64_t len = P.seq_len[b], to = new_len[i];
      if (to >= len && len >= 0 && to <= ((int64_t)P.max_pages << P.page_shift))
        need = (int)(pages_for(P, to) - pages_for(P, len));
    }
    E.need[i] = need;
    if (need < 0 && b != -1) set_flag(P.flags, CSA2_FLAG_BAD_SEQ);
  }
  __syncthreads();
  place_entries(P, W, E, n);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = warp; i < n; i += kPlanWarps) {
    const int need = E.need[i];
    if (need < 0) continue;
    const int b = seqs[i];
    int32_t* row = P.table + (int64_t)b * P.table_ld + pages_for(P, P.seq_len[b]);
    for (int k = lane; k < need; k += 32) {
      const int g = W.fresh[E.off[i] + k];
      row[k] = g;
      P.ref[g] = 1;
    }
    __syncwarp();
    if (lane == 0) P.seq_len[b] = new_len[i];
  }
}

// ---------------------------------------------------------------- fork
// The plan: what each entry needs, where its fresh pages lie, and the pairs
// (source page, rows in use) to be copied into them, in the order of the pages.
__global__ void __launch_bounds__(kPlanThreads, 1) pages_fork_plan_kernel(const PagePool P, const PagePlan W, int n,
                                                                       const int32_t* __restrict__ parents,
                                                                       const int32_t* __restrict__ children, int deep) {
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ EntriesShared sh;
  const Entries E = entries_of(P, W, sh);
  plan_prefetch(P);
  claim(P, children, n, E.owner);
#pragma unroll 1
  for (int i = warp; i < n; i += kPlanWarps) {
    const int p = parents[i], c = children[i];
    int need = -1;
    if (p >= 0 && p < P.n_seq && c >= 0 && c < P.n_seq) {
      const int64_t len = P.seq_len[p], child_len = P.seq_len[c];
      const int64_t np = pages_for(P, len);
      if (E.owner[c] == i && E.owner[p] == kNoOwner && child_len == 0 && len >= 0 && np <= P.max_pages) {
        const int32_t* row = P.table + (int64_t)p * P.table_ld;
        if (deep) {
          int mine = 0;
#pragma unroll 4
          for (int j = lane; j < np; j += 32) mine += is_page(P, row[j]) ? 1 : 0;
          need = __reduce_add_sync(0xffffffffu, mine);
        } else {
          need = (len & ((1 << P.page_shift) - 1)) != 0 && is_page(P, row[np - 1]) ? 1 : 0;
        }
      }
    }
    if (lane == 0) {
      E.need[i] = need;
      if (need < 0 && c != -1) set_flag(P.flags, CSA2_FLAG_BAD_SEQ);
    }
  }
  __syncthreads();
  place_entries(P, W, E, n);
  __shared__ int s_pairs;
  if (threadIdx.x == 0) s_pairs = 0;
  __syncthreads();
  for (int i = warp; i < n; i += kPlanWarps) {
    const int need = E.need[i];
    if (need <= 0) continue;
    const int64_t len = P.seq_len[parents[i]];
    const int np = (int)pages_for(P, len), ps = 1 << P.page_shift;
    const int32_t* row = P.table + (int64_t)parents[i] * P.table_ld;
    int at = E.off[i];
#pragma unroll 1
    for (int j0 = deep ? 0 : np - 1; j0 < np; j0 += 32) {
      const int j = j0 + lane;
      const int32_t g = j < np ? row[j] : -1;
      const unsigned has = __ballot_sync(0xffffffffu, is_page(P, g));
      if (is_page(P, g)) {
        const int k = at + __popc(has & ((1u << lane) - 1u));
        W.src[k] = g;
        W.rows[k] = (int32_t)min((int64_t)ps, len - (int64_t)j * ps);
      }
      at += __popc(has);
    }
    if (lane == 0) atomicMax(&s_pairs, at);
  }
  __syncthreads();
  if (threadIdx.x == 0) W.count[0] = s_pairs;
  if (E.need != W.need)
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
      W.need[i] = E.need[i];
      W.off[i] = E.off[i];
    }
}

// Copies `count` pages (rows[k] rows of page src[k], all rows where rows is
// null) into pages dst[k], in every array: units of 16 KB, strided over the
// n_ctas CTAs.
__device__ void copy_pages(const PageArrays& A, const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
                           const int32_t* __restrict__ rows, int count, int page_rows, int cta, int n_ctas) {
  int64_t base = 0;
  int64_t u = cta;
  for (int a = 0; a < A.n; ++a) {
    const PageArray& ar = A.a[a];
    const int64_t page_bytes = (int64_t)page_rows * ar.row_bytes;
    const int chunks = (int)((page_bytes + kCopyChunk - 1) / kCopyChunk);
    const int64_t end = base + (int64_t)count * chunks;
    for (; u < end; u += n_ctas) {
      const int64_t k = (u - base) / chunks;
      const int64_t lo = ((u - base) - k * chunks) * (int64_t)kCopyChunk;
      const int64_t bytes = rows != nullptr ? (int64_t)rows[k] * ar.row_bytes : page_bytes;
      const int n = (int)min((int64_t)kCopyChunk, bytes - lo);
      if (n <= 0) continue;
      const uint8_t* s = ar.base + (int64_t)src[k] * ar.stride + lo;
      uint8_t* d = ar.base + (int64_t)dst[k] * ar.stride + lo;
      int done = 0;
      if (ar.wide) {
        const int n16 = n >> 4;
        uint4 v[kCopyChunk / 16 / kCopyThreads];
#pragma unroll
        for (int q = 0; q < kCopyChunk / 16 / kCopyThreads; ++q) {
          const int i = (int)threadIdx.x + q * kCopyThreads;
          if (i < n16) v[q] = ldg_stream16(s + 16 * i);
        }
#pragma unroll
        for (int q = 0; q < kCopyChunk / 16 / kCopyThreads; ++q) {
          const int i = (int)threadIdx.x + q * kCopyThreads;
          if (i < n16) *reinterpret_cast<uint4*>(d + 16 * i) = v[q];
        }
        done = n16 << 4;
      }
      for (int i = done + (int)threadIdx.x; i < n; i += kCopyThreads) d[i] = s[i];
    }
    base = end;
  }
}

// The fork itself: the first n CTAs write one entry's table row and counts
// each, the others copy the pairs' pages.
__global__ void __launch_bounds__(kCopyThreads) pages_fork_apply_kernel(const PagePool P, const PagePlan W, int n,
                                                                        const int32_t* __restrict__ parents,
                                                                        const int32_t* __restrict__ children, int deep,
                                                                        const __grid_constant__ PageArrays A) {
  pdl_wait();
  if ((int)blockIdx.x >= n) {
    copy_pages(A, W.src, W.fresh, W.rows, W.count[0], 1 << P.page_shift, (int)blockIdx.x - n, (int)gridDim.x - n);
    return;
  }
  __shared__ int warp_n[kCopyThreads / 32];
  const int i = blockIdx.x;
  if (W.need[i] < 0) return;
  const int p = parents[i], c = children[i];
  const int64_t len = P.seq_len[p];
  const int np = (int)pages_for(P, len), ps = 1 << P.page_shift;
  const int32_t* from = P.table + (int64_t)p * P.table_ld;
  int32_t* to = P.table + (int64_t)c * P.table_ld;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int at = W.off[i];
  for (int j0 = 0; j0 < np; j0 += kCopyThreads) {
    const int j = j0 + (int)threadIdx.x;
    const int32_t g = j < np ? from[j] : -1;
    const bool has = is_page(P, g);
    const bool fresh = has && (deep != 0 || (j == np - 1 && (len & (ps - 1)) != 0));
    const unsigned m = __ballot_sync(0xffffffffu, fresh);
    if (lane == 0) warp_n[warp] = __popc(m);
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kCopyThreads / 32; ++w) {
      if (w < warp) before += warp_n[w];
      all += warp_n[w];
    }
    if (j < np) {
      int32_t v = -1;
      if (fresh) {
        v = W.fresh[at + before + __popc(m & ((1u << lane) - 1u))];
        P.ref[v] = 1;
      } else if (has) {
        v = g;
        atomicAdd(&P.ref[g], 1);
      }
      to[j] = v;
    }
    at += all;
    __syncthreads();  // warp_n is free for the next round
  }
  if (threadIdx.x == 0) P.seq_len[c] = len;
}

// ---------------------------------------------------------------- free / trim
// One CTA an entry. An entry's table slots are emptied by exchange, so that a
// sequence named twice gives its pages back once. window < 0: all its pages;
// otherwise only those no query from position len - 1 on can see.
__global__ void __launch_bounds__(256) pages_free_kernel(const PagePool P, const int32_t* __restrict__ seqs,
                                                         int64_t window, int64_t n_first,
                                                         const int64_t* __restrict__ lo_of) {
  const int b = seqs[blockIdx.x];
  if (b < 0 || b >= P.n_seq) {
    if (threadIdx.x == 0 && b != -1) set_flag(P.flags, CSA2_FLAG_BAD_SEQ);
    return;
  }
  int32_t* row = P.table + (int64_t)b * P.table_ld;
  const int64_t len = P.seq_len[b];
  int64_t head_lo = 0, head_hi = 0, tail = 0;
  int n_cols = P.max_pages;
  if (window >= 0) {
    head_lo = lo_of != nullptr ? min(max(lo_of[b], (int64_t)0), (int64_t)1 << 40) : 0;  // past any row
    head_hi = head_lo + n_first;
    tail = max(head_lo, len - window);
    n_cols = (int)min((int64_t)P.max_pages, pages_for(P, max(len, (int64_t)0)));
  }
  for (int j = threadIdx.x; j < n_cols; j += blockDim.x) {
    if (row[j] < 0) continue;
    if (window >= 0) {
      // rows [a, e) of this page: kept if the first tokens or the tail reach in
      const int64_t a = (int64_t)j << P.page_shift, e = a + (1 << P.page_shift);
      if ((a < head_hi && e > head_lo) || (e > tail && a < len)) continue;
    }
    const int32_t g = atomicExch(&row[j], -1);
    if (g < 0) continue;
    if (!is_page(P, g)) {
      set_flag(P.flags, CSA2_FLAG_BAD_PAGE);
    } else if (atomicSub(&P.ref[g], 1) <= 0) {  // more references than counted
      atomicAdd(&P.ref[g], 1);
      set_flag(P.flags, CSA2_FLAG_BAD_PAGE);
    }
  }
  if (window < 0) {
    __syncthreads();
    if (threadIdx.x == 0) P.seq_len[b] = 0;
  }
}

// ---------------------------------------------------------------- compact
// The plan: with L pages in use, the free pages below L in ascending order
// take the pages in use from L on in ascending order. map[g] (g >= L) is a
// page's new index, -1 for a free one.
__global__ void __launch_bounds__(kPlanThreads, 1) pages_compact_plan_kernel(const PagePool P, const PagePlan W,
                                                                          int32_t* __restrict__ n_live_out) {
  pdl_trigger();
  uint32_t live = 0;
#pragma unroll 4
  for (int g = threadIdx.x; g < P.n_pages; g += kPlanThreads) live += P.ref[g] > 0 ? 1 : 0;
  uint32_t total;
  cta_scan(live, 0x7FFFFFFFu, &total);
  const int L = (int)total;
  int n_dst = 0, n_src = 0;
  constexpr int kEach = 8;
  for (int base = 0; base < P.n_pages; base += kPlanThreads * kEach) {
    const int first = base + (int)threadIdx.x * kEach;
    uint32_t dst_bits = 0, src_bits = 0;
#pragma unroll
    for (int u = 0; u < kEach; ++u) {
      const int g = first + u;
      if (g < P.n_pages) {
        const int r = P.ref[g];
        if (g < L && r <= 0) dst_bits |= 1u << u;
        if (g >= L) {
          if (r > 0) src_bits |= 1u << u;
          else W.map[g] = -1;
        }
      }
    }
    // both counts in one scan: at most 4,096 of each a round
    const uint32_t at = cta_scan((uint32_t)(__popc(dst_bits) | __popc(src_bits) << 16), 0x7FFFFFFFu, &total);
    int d = n_dst + (int)(at & 0xFFFFu), s = n_src + (int)(at >> 16);
    for (; dst_bits != 0u; dst_bits &= dst_bits - 1) W.fresh[d++] = first + __ffs(dst_bits) - 1;
    for (; src_bits != 0u; src_bits &= src_bits - 1) W.src[s++] = first + __ffs(src_bits) - 1;
    n_dst += (int)(total & 0xFFFFu);
    n_src += (int)(total >> 16);
  }
  __syncthreads();  // the lists, of equal length, are complete
  for (int k = threadIdx.x; k < n_src; k += kPlanThreads) {
    const int s = W.src[k], d = W.fresh[k];
    W.map[s] = d;
    P.ref[d] = P.ref[s];
    P.ref[s] = 0;
  }
  if (threadIdx.x == 0) {
    W.count[0] = n_src;
    W.count[1] = L;
    if (n_live_out != nullptr) *n_live_out = L;
  }
}

constexpr int kRemapEach = 2048;  // table entries a remapping CTA takes

__global__ void __launch_bounds__(kCopyThreads) pages_compact_apply_kernel(const PagePool P, const PagePlan W,
                                                                           int remap_ctas,
                                                                           const __grid_constant__ PageArrays A) {
  pdl_wait();
  if ((int)blockIdx.x >= remap_ctas) {
    copy_pages(A, W.src, W.fresh, nullptr, W.count[0], 1 << P.page_shift, (int)blockIdx.x - remap_ctas,
               (int)gridDim.x - remap_ctas);
    return;
  }
  const int L = W.count[1];
  const int64_t n = (int64_t)P.n_seq * P.max_pages;
  for (int64_t at = (int64_t)blockIdx.x * kRemapEach; at < n; at += (int64_t)remap_ctas * kRemapEach) {
    for (int64_t i = at + threadIdx.x; i < min(at + kRemapEach, n); i += kCopyThreads) {
      const int64_t b = i / P.max_pages;
      int32_t* e = P.table + b * P.table_ld + (i - b * P.max_pages);
      const int32_t g = *e;
      if (g < L) continue;
      const int32_t to = g < P.n_pages ? W.map[g] : -1;
      if (to < 0) set_flag(P.flags, CSA2_FLAG_BAD_PAGE);
      *e = to;
    }
  }
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

PagePlan plan_of(const PagePool& P, void* ws) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto take = [&](size_t n) {
    int32_t* p = reinterpret_cast<int32_t*>(w);
    w += al256(n * 4);
    return p;
  };
  PagePlan W;
  W.owner = take(P.n_seq);
  W.need = take(P.n_seq);
  W.off = take(P.n_seq);
  W.fresh = take(P.n_pages);
  W.src = take(P.n_pages);
  W.rows = take(P.n_pages);
  W.map = take(P.n_pages);
  W.count = take(4);
  return W;
}

// CTAs that copy `pages` pages at most: eight resident a SM keep 128 KB of
// loads under way on each, and no more than there are units
int copy_ctas(int num_sms, const PageArrays& A, int64_t pages, int page_rows) {
  int64_t units = 0;
  for (int a = 0; a < A.n; ++a)
    units += pages * (((int64_t)page_rows * A.a[a].row_bytes + kCopyChunk - 1) / kCopyChunk);
  return (int)(units < 8 * num_sms ? units : 8 * num_sms);
}

}  // namespace

size_t pages_workspace_bytes(int n_seq, int n_pages) {
  return 3 * al256((size_t)n_seq * 4) + 4 * al256((size_t)n_pages * 4) + al256(16);
}

cudaError_t launch_pages_extend(cudaStream_t st, const PagePool& P, int n, const int32_t* seqs, const int64_t* new_len,
                                void* ws) {
  pages_extend_kernel<<<1, kPlanThreads, 0, st>>>(P, plan_of(P, ws), n, seqs, new_len);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(cudaStream_t st, int num_sms, const PagePool& P, int n, const int32_t* parents,
                              const int32_t* children, bool deep, const PageArrays& A, void* ws) {
  const PagePlan W = plan_of(P, ws);
  pages_fork_plan_kernel<<<1, kPlanThreads, 0, st>>>(P, W, n, parents, children, deep ? 1 : 0);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_ex(pages_fork_apply_kernel, dim3((unsigned)(n + copy_ctas(num_sms, A, deep ? P.n_pages : n, 1 << P.page_shift))), dim3(kCopyThreads), 0, st, true,
                   0, P, W, n, parents, children, deep ? 1 : 0, A);
}

cudaError_t launch_pages_free(cudaStream_t st, const PagePool& P, int n, const int32_t* seqs, int64_t window,
                              int64_t n_first, const int64_t* lo) {
  pages_free_kernel<<<n, 256, 0, st>>>(P, seqs, window, n_first, lo);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(cudaStream_t st, int num_sms, const PagePool& P, const PageArrays& A, int32_t* n_live,
                                 void* ws) {
  const PagePlan W = plan_of(P, ws);
  pages_compact_plan_kernel<<<1, kPlanThreads, 0, st>>>(P, W, n_live);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t entries = (int64_t)P.n_seq * P.max_pages;
  const int64_t want = (entries + kRemapEach - 1) / kRemapEach;
  const int remap = (int)(want < num_sms ? want : num_sms);
  return launch_ex(pages_compact_apply_kernel, dim3((unsigned)(remap + copy_ctas(num_sms, A, P.n_pages, 1 << P.page_shift))), dim3(kCopyThreads), 0, st,
                   true, 0, P, W, remap, A);
}

}  // namespace csa2

// csa2_attend_paged: attention of new tokens over a paged cache.
//
// For query q at position t of sequence b, with q~ = RoPE_t(q), over the
// visible rows p (all of [lo, t], or the last `window` of them and the first
// `n_first`):  s_p = scale q~ . row_p,  o = sum_p e^{s_p} row_p /
// (sum_p e^{s_p} + e^{sink}), its rope channels rotated back by -t.
//
// The visible rows of a query, packed, make 128-row tiles (a query that sees
// nothing makes one empty tile, which writes its zeros). All queries' tiles,
// one query after another, are cut into equal runs, one run per CTA and one
// CTA per SM: a long sequence is split over many CTAs and a CTA takes many
// short ones. A query that lies whole in one run is written at once; the runs'
// ends leave unnormalised fp32 partials, at most two a CTA, which the join
// kernel sums. The products and softmax of a tile are those of attend_tile.cuh.
#include "attend_tile.cuh"
#include "paged.cuh"

namespace csa2 {

struct PagedAttendParams {
  AttendParams a;       // q, positions, sink, outputs, scale, RoPE, flags, part_*
  PagedView kv;
  const int64_t* lo;    // [n_seq], nullable
  int64_t window;       // 0: every row
  int64_t n_first;
  int2* joins;          // [min(n_query, gridDim.x)]: first and last CTA of a query to be joined (-1: none)
  int32_t* join_query;  // the query of each
};

namespace {

constexpr int kJoinThreads = 512;

struct QuerySpan {
  Visible vis;
  int64_t t;
  int b;       // sequence, -1 for a padding query
  bool ok;     // a query with a sequence and a position
  int n_tiles;
};

__device__ __forceinline__ QuerySpan query_span(const PagedAttendParams& p, int qi) {
  QuerySpan s;
  s.t = p.a.q_pos[qi];
  s.b = p.a.seq_of_q[qi];
  s.ok = s.b >= 0 && s.b < p.kv.n_seq && s.t >= 0;
  const int64_t cap = (int64_t)p.kv.max_pages << p.kv.page_shift;
  const int64_t lo = (s.ok && p.lo != nullptr) ? p.lo[s.b] : 0;
  s.vis = visible_rows(s.ok ? s.t : -1, lo, p.window, p.n_first, cap);
  s.n_tiles = max(1, (s.vis.count + kTileRows - 1) / kTileRows);
  return s;
}

// Slots of the partials: CTA c leaves at most two, 2c for a query that began
// in an earlier CTA and 2c + 1 for one that it begins and does not end.
__device__ __forceinline__ int part_slot(int c, bool begins) { return 2 * c + (begins ? 1 : 0); }

}  // namespace

template <int KVF>
__global__ void __launch_bounds__(kAttThreads, 1) attend_paged_kernel(const PagedAttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base_s - raw_s);
  float* m_run = reinterpret_cast<float*>(sm + SM_MRUN);
  float* l_run = reinterpret_cast<float*>(sm + SM_LRUN);
  int64_t* rows = reinterpret_cast<int64_t*>(sm + SM_ROWS);  // page << 16 | row in the page, -1 for none
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + SM_MISC);
  float2* rope_tab = reinterpret_cast<float2*>(sm + SM_ROPE);
  const uint32_t mbar = base_s + SM_MISC;
  const uint32_t tslot = base_s + SM_MISC + 8;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int quad = warp & 3;
  const int row = quad * 32 + lane;

  pdl_trigger();
  if (warp == 0) {
    tmem_alloc(tslot, kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    mbar_init(mbar, 1);
    fence_mbar_init();
    misc[3] = 0;
  }
  pdl_wait();

  // ---- this CTA's run of tiles: thread x counts the tiles of its share of
  // the queries, a scan places the shares, and the thread whose share holds
  // the run's first tile finds its query
  const int Q = p.a.n_query;
  __shared__ int64_t warp_sum[kAttWarps];
  __shared__ int64_t s_first_tile;  // first tile of query s_query among all
  __shared__ int s_query;
  const int per = (Q + kAttThreads - 1) / kAttThreads;
  const int q_lo = min(Q, tid * per), q_hi = min(Q, q_lo + per);
  int64_t mine = 0;
  for (int i = q_lo; i < q_hi; ++i) mine += query_span(p, i).n_tiles;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int64_t base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kAttWarps; ++w) {
    if (w < warp) base += warp_sum[w];
    total += warp_sum[w];
  }
  // no run is empty: the CTAs of a split query are neighbours
  const int c = (int)blockIdx.x;
  const int G = (int)min((int64_t)gridDim.x, total);
  const int64_t run0 = c < G ? (int64_t)c * total / G : total, run1 = c < G ? (int64_t)(c + 1) * total / G : total;
  const int64_t before = base + incl - mine;
  if (run0 >= before && run0 < before + mine) {
    int64_t at = before;
    int i = q_lo;
    for (;; ++i) {
      const int n = query_span(p, i).n_tiles;
      if (run0 < at + n) break;
      at += n;
    }
    s_query = i;
    s_first_tile = at;
  }
  const float sink_l2 = (tid < kHeads && p.a.sink != nullptr) ? p.a.sink[tid] * 1.4426950408889634f : -INFINITY;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = misc[2];
  const uint32_t tmem_s = taddr, tmem_o = taddr + 64;
  const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
  uint32_t phase = 0;
  bool aborted = false;
  const bool rope = p.a.rp.pairs > 0;
  const bool by_query = Q < (int)gridDim.x;  // the index of a join: its query, or the CTA that begins it

  int qi = 0;
  int64_t q0 = 0;
  if (run0 < run1) {
    qi = s_query;
    q0 = s_first_tile;
  }
  int my_join_query = -1;
  int2 my_join = make_int2(-1, -1);
  for (int64_t at = run0; at < run1 && !aborted; ++qi) {
    const QuerySpan qs = query_span(p, qi);
    const int tile_begin = (int)(at - q0);
    const int tile_end = (int)min((int64_t)qs.n_tiles, run1 - q0);
    const bool begins = tile_begin == 0, ends = tile_end == qs.n_tiles;
    const bool has_rows = qs.vis.count > 0;
    if (begins && tid == 0) {
      if (!qs.ok && !(qs.b == -1) && !(qs.b >= 0 && qs.b < p.kv.n_seq && qs.t == -1))
        set_flag(p.a.flags, CSA2_FLAG_BAD_QUERY);
      if (qs.ok && qs.vis.past_table) set_flag(p.a.flags, CSA2_FLAG_BAD_PAGE);
    }
    const int2 jn = (begins && !ends) ? make_int2(c, (int)(((q0 + qs.n_tiles) * G - 1) / total)) : make_int2(-1, -1);
    if (by_query) {
      if (begins && tid == 0) {
        p.joins[qi] = jn;
        p.join_query[qi] = qi;
      }
    } else if (begins && !ends) {
      my_join = jn;
      my_join_query = qi;
    }
    if (has_rows) {
      copy_q_async(p.a, base_s, qi);
      cp_async_commit();
    }
    if (tid < p.a.rp.pairs) {
      float cc = 1.f, sn = 0.f;
      if (qs.ok) rope_cs(p.a.rp, tid, qs.t, cc, sn);
      rope_tab[tid] = make_float2(cc, sn);
    }
    if (tid < kHeads) {
      m_run[tid] = -INFINITY;
      l_run[tid] = 0.f;
    }
    float lsum[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) lsum[k] = 0.f;
    for (int tile = tile_begin; has_rows && tile < tile_end; ++tile) {
      if (tid < kTileRows) {
        const int i = tile * kTileRows + tid;
        int64_t src = -1;
        if (i < qs.vis.count) {
          const int64_t pos = visible_pos(qs.vis, i);
          const int32_t g = page_of(p.kv, qs.b, pos);
          if (g >= 0) src = ((int64_t)g << 16) | (pos & ((1 << p.kv.page_shift) - 1));
          else set_flag(p.a.flags, CSA2_FLAG_BAD_PAGE);
        }
        rows[tid] = src;
      }
      __syncthreads();
      // a warp takes rows warp, warp + 8, ..., eight rows' loads in flight
      constexpr int kBatch = 8;
#pragma unroll 1
      for (int r0 = warp; r0 < kTileRows; r0 += kAttWarps * kBatch) {
        if constexpr (KVF == 0) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int r = r0 + kAttWarps * j;
            const int64_t src = rows[r];
            const uint8_t* g = p.kv.pages + (src >= 0 ? (src >> 16) * p.kv.page_stride + (src & 0xFFFF) * 1024 : 0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int cc = lane + 32 * u;
              const uint32_t dst = base_s + SM_KV + (uint32_t)(cc >> 3) * 16384u + (uint32_t)r * 128u +
                                   ((uint32_t)((cc & 7) ^ (r & 7)) << 4);
              cp_async16(dst, g + 16 * cc, src >= 0 ? 16u : 0u);
            }
          }
        } else {
          uint4 codes[kBatch];
          uint32_t sb[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int64_t src = rows[r0 + kAttWarps * j];
            codes[j] = make_uint4(0u, 0u, 0u, 0u);
            sb[j] = 0;
            if (src >= 0) {
              const int64_t g = src >> 16, r = src & 0xFFFF;
              if constexpr (KVF == 1) {
                codes[j] = ldg_stream16(p.kv.pages + g * p.kv.page_stride + r * 512 + 16 * lane);
                sb[j] = p.kv.scales[g * p.kv.scale_stride + r * 16 + (lane >> 1)];
              } else {
                const uint2 w = ldg_stream8(p.kv.pages + g * p.kv.page_stride + r * 256 + 8 * lane);
                codes[j].x = w.x;
                codes[j].y = w.y;
                sb[j] = p.kv.scales[g * p.kv.scale_stride + r * 32 + lane];
              }
            }
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int r = r0 + kAttWarps * j;
            uint32_t o[8];
            if constexpr (KVF == 1) {
              const float sc = ue8m0_value(sb[j]);
              const uint32_t cw[4] = {codes[j].x, codes[j].y, codes[j].z, codes[j].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 a = e4m3x2_to_float2((uint16_t)(cw[k] & 0xFFFFu));
                const float2 b = e4m3x2_to_float2((uint16_t)(cw[k] >> 16));
                o[2 * k] = pack_bf16(a.x * sc, a.y * sc);
                o[2 * k + 1] = pack_bf16(b.x * sc, b.y * sc);
              }
            } else {
              const float sc = e4m3_value(sb[j]) * kE2M1Unscale;
#pragma unroll
              for (int b = 0; b < 8; ++b) {
                const float2 f = e2m1x2_to_float2_scaled(((b < 4 ? codes[j].x : codes[j].y) >> (8 * (b & 3))) & 0xFFu);
                o[b] = pack_bf16(f.x * sc, f.y * sc);  // exact: <= 6 significant bits
              }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int cc = 2 * lane + u;
              const uint32_t off = SM_KV + (uint32_t)(cc >> 3) * 16384u + (uint32_t)r * 128u +
                                   ((uint32_t)((cc & 7) ^ (r & 7)) << 4);
              *reinterpret_cast<uint4*>(sm + off) = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
          }
        }
      }
      cp_async_wait_all();
      if (tile == tile_begin && rope) {
        __syncthreads();
        q_rope_split(sm, p.a.rp);
      }
      fence_proxy_async_smem();
      __syncthreads();
      if (tid == 0) {
        tc_fence_after();
        issue_qk(base_s, tmem_s, 0, 1, rope);
        mma_commit(mbar);
      }
      bool ok = mbar_wait(mbar, phase, p.a.flags);
      phase ^= 1u;
      if (!__syncthreads_and(ok)) { aborted = true; break; }
      tc_fence_after();
      tile_softmax<true>(p.a, sm, tmem_s, tmem_o, lane_base, rows[row] >= 0, tile == tile_begin, &misc[3], lsum, SyncCta{});
      if (tid == 0) {
        tc_fence_after();
        issue_pv(base_s, tmem_o, tile > tile_begin);
        mma_commit(mbar);
      }
      ok = mbar_wait(mbar, phase, p.a.flags);
      phase ^= 1u;
      if (!__syncthreads_and(ok)) { aborted = true; break; }
      tc_fence_after();
    }
    __syncthreads();
    if (!aborted && qs.b != -1) {
      AttendParams st = p.a;
      st.direct = (begins && ends) ? 1 : 2;
      attend_store(st, sm, st.direct == 1 ? qi : part_slot(c, begins), 0, has_rows, lsum, tmem_o, lane_base, sink_l2,
                   SyncCta{});
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    at = q0 + tile_end;
    q0 += qs.n_tiles;
  }
  if (!by_query && tid == 0) {
    p.joins[c] = my_join;
    p.join_query[c] = my_join_query;
  }
  cp_async_wait_all();
  if (aborted) mbar_wait(mbar, phase ^ 1u, p.a.flags, 1000000000ull);  // tensor-core work in flight lands first
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(taddr, kTmemCols);
}

// Join of a split query's partials: one CTA per (query, head). With M the
// largest reference of its parts and the sink, o = sum_g e^(m_g - M) O_g /
// (sum_g e^(m_g - M) l_g + e^(sink - M)), its rope channels rotated back.
// Four groups of 128 threads take every fourth part, 4 channels a thread.
__global__ void __launch_bounds__(kJoinThreads) attend_paged_join_kernel(const PagedAttendParams p) {
  __shared__ float wpart[512];
  __shared__ float red[kJoinThreads / 32];
  __shared__ float4 acc_s[4][128];
  pdl_wait();
  const int2 jn = p.joins[blockIdx.x];
  if (jn.x < 0) return;
  const int qi = p.join_query[blockIdx.x];
  const int h = blockIdx.y;
  const int n = jn.y - jn.x + 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float sk = p.a.sink != nullptr ? p.a.sink[h] : -INFINITY;
  auto slot = [&](int k) { return (int64_t)(k == 0 ? part_slot(jn.x, true) : part_slot(jn.x + k, false)); };
  // n <= gridDim of the tile kernel <= 512 parts: one a thread
  const float m = tid < n ? p.a.part_m[slot(tid) * kHeads + h] : -INFINITY;
  const float l = tid < n ? p.a.part_l[slot(tid) * kHeads + h] : 0.f;
  float M = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[warp] = M;
  __syncthreads();
  M = sk;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) M = fmaxf(M, red[w]);
  const float e = (M == -INFINITY || m == -INFINITY) ? 0.f : expf(m - M);
  wpart[tid] = e;
  float den = e * l;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  __syncthreads();
  if (lane == 0) red[warp] = den;
  __syncthreads();
  den = M == -INFINITY ? 0.f : expf(sk - M);
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) den += red[w];
  const int g = tid >> 7, ch = 4 * (tid & 127);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = g; k < n; k += 4) {
    const float w = wpart[k];
    const float4 v = *reinterpret_cast<const float4*>(p.a.part_o + (slot(k) * kHeads + h) * kDim + ch);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  acc_s[g][tid & 127] = acc;
  __syncthreads();
  if (g != 0) return;
#pragma unroll
  for (int k = 1; k < 4; ++k) {
    const float4 v = acc_s[k][tid];
    acc.x += v.x;
    acc.y += v.y;
    acc.z += v.z;
    acc.w += v.w;
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
  acc.x *= inv;
  acc.y *= inv;
  acc.z *= inv;
  acc.w *= inv;
  const int first_rope = kDim - 2 * p.a.rp.pairs;
  if (ch >= first_rope) {
    const int64_t t = p.a.q_pos[qi];
    float c0, s0, c1, s1;
    rope_cs(p.a.rp, (ch - first_rope) >> 1, t, c0, s0);
    rope_cs(p.a.rp, ((ch - first_rope) >> 1) + 1, t, c1, s1);
    acc = make_float4(acc.x * c0 + acc.y * s0, acc.y * c0 - acc.x * s0, acc.z * c1 + acc.w * s1,
                      acc.w * c1 - acc.z * s1);
  }
  *reinterpret_cast<uint2*>(p.a.out + ((int64_t)qi * kHeads + h) * kDim + ch) =
      make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
  if (tid == 0 && p.a.lse != nullptr) p.a.lse[(int64_t)qi * kHeads + h] = M == -INFINITY ? -INFINITY : M + logf(den);
}

namespace {
constexpr size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
// Every CTA sums the tile counts of all queries before it starts: 16 a thread
// at this many. More queries go in launches of this many, one after another.
constexpr int kMaxQueries = 4096;
}  // namespace

int attend_paged_ctas(int num_sms) { return num_sms < 512 ? num_sms : 512; }

size_t attend_paged_workspace_bytes(int num_sms) {
  const size_t slots = 2 * (size_t)attend_paged_ctas(num_sms);
  return al256(slots * kHeads * kDim * 4) + 2 * al256(slots * kHeads * 4) + al256(slots * 8) + al256(slots * 4);
}

cudaError_t launch_attend_paged(cudaStream_t st, int num_sms, int kv_fmt, AttendParams a, const PagedView& kv,
                                const int64_t* lo, int64_t window, int64_t n_first, void* ws, int* n_launch) {
  const int G = attend_paged_ctas(num_sms);
  const size_t slots = 2 * (size_t)G;
  uint8_t* w = static_cast<uint8_t*>(ws);
  PagedAttendParams p{};
  p.a = a;
  p.kv = kv;
  p.lo = lo;
  p.window = window;
  p.n_first = n_first;
  p.a.part_o = reinterpret_cast<float*>(w);
  w += al256(slots * kHeads * kDim * 4);
  p.a.part_m = reinterpret_cast<float*>(w);
  w += al256(slots * kHeads * 4);
  p.a.part_l = reinterpret_cast<float*>(w);
  w += al256(slots * kHeads * 4);
  p.joins = reinterpret_cast<int2*>(w);
  w += al256(slots * 8);
  p.join_query = reinterpret_cast<int32_t*>(w);
  const int Q = a.n_query;
  for (int q0 = 0; q0 < Q; q0 += kMaxQueries) {
    const int nq = Q - q0 < kMaxQueries ? Q - q0 : kMaxQueries;
    p.a.n_query = nq;
    p.a.q = a.q + (int64_t)q0 * kHeads * kDim;
    p.a.q_pos = a.q_pos + q0;
    p.a.seq_of_q = a.seq_of_q + q0;
    p.a.out = a.out + (int64_t)q0 * kHeads * kDim;
    p.a.lse = a.lse != nullptr ? a.lse + (int64_t)q0 * kHeads : nullptr;
    cudaError_t e;
#define CSA2_PAGED(F)                                                                                              \
  do {                                                                                                             \
    e = cudaFuncSetAttribute(attend_paged_kernel<F>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kAttSmemBytes); \
    if (e == cudaSuccess)                                                                                          \
      e = launch_ex(attend_paged_kernel<F>, dim3(G), dim3(kAttThreads), kAttSmemBytes, st, false, 0, p);             \
  } while (0)
    if (kv_fmt == 0) CSA2_PAGED(0);
    else if (kv_fmt == 1) CSA2_PAGED(1);
    else CSA2_PAGED(2);
#undef CSA2_PAGED
    if (e != cudaSuccess) return e;
    *n_launch += 1;
    e = launch_ex(attend_paged_join_kernel, dim3((unsigned)(nq < G ? nq : G), kHeads), dim3(kJoinThreads), 0, st, true, 0, p);
    if (e != cudaSuccess) return e;
    *n_launch += 1;
  }
  return cudaGetLastError();
}

}  // namespace csa2

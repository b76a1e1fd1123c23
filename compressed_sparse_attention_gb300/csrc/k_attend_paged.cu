// csa2_attend_paged: attention of new tokens over a paged cache.
//
// For query q at position t of sequence b, with q~ = RoPE_t(q), over the
// visible rows p (all of [lo, t], or the last `window` of them and the first
// `n_first`):  s_p = scale q~ . row_p,  o = sum_p e^{s_p} row_p /
// (sum_p e^{s_p} + e^{sink}), its rope channels rotated back by -t.
//
// The chunks of a query's visible rows (paged.cuh) make 128-row tiles (a query
// that sees nothing makes one empty tile, which writes its zeros). All
// queries' tiles, one query after another, are cut into runs of equal cost,
// one run per CTA and one CTA per SM: a long sequence is split over many CTAs
// and a CTA takes many short ones. A query that lies whole in one run is
// written at once; the runs' ends leave unnormalised fp32 partials, at most two
// a CTA, which the join kernel sums. A tile's place in shared memory and its
// products are those of attend_tile.cuh.
//
// What bounds it. bf16 rows from memory: 128 KB a tile and SM, 5,640 cycles at
// the copy rate, against 5,600 to 6,000 measured from tile to tile in a long
// run; over rows in the L2 (a prompt's queries share theirs) the tile's own
// chain is as long: the products' 3,264 cycles (48 each for 6 KB of operands,
// shared memory's 128 bytes a clock), the scores' weights (1,000) and the
// waits between them, with one tile in shared memory at a time. fp8 and fp4
// rows: the same chain with the conversion's stores in it, 8,700 cycles. Short
// calls: launch, cut, first rows and join, 14 us together. Calls of many short
// queries: 6,000 cycles an output (reading tensor memory, scaling, exchanging
// between lanes; with its stores left out it takes as long). Measured: 32
// ragged sequences to 8K 48.5 us (3.2 TB/s), 8 x 128K fp8 262 us, 1,200 prompt
// queries under a window of 512 167 us, one query over 2K rows 14.6 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <atomic>
#include <type_traits>

#include "attend_tile.cuh"
#include "paged.cuh"

namespace csa2 {

struct PagedAttendParams {
  CUtensorMap q_map;     // Q: [64 n_query heads][512], boxes of 64 heads x 64 channels
  CUtensorMap kv_map;    // bf16 pages: [n_pages][page_size][512], boxes of one chunk x 64 channels
  AttendParams a;       // q, positions, sink, outputs, scale, RoPE, flags, part_*
  PagedView kv;
  const int64_t* lo;    // [n_seq], nullable
  int64_t window;       // 0: every row
  int64_t n_first;
  int4* joins;          // [min(n_query, gridDim.x)]: first and last CTA of a query to be joined (-1: none), the query
};

namespace {

constexpr int kMaxCtas = 512;  // of the tile kernel: the most parts of a query

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
  const int32_t cap = p.kv.max_pages << p.kv.page_shift;  // at most 2^30
  const int64_t lo = (s.ok && p.lo != nullptr) ? p.lo[s.b] : 0;
  const int cs = chunk_shift(p.kv.page_shift);
  s.vis = visible_rows(s.ok ? s.t : -1, lo, p.window, p.n_first, cap, cs);
  s.n_tiles = max(1, ((s.vis.n_chunks << cs) + kTileRows - 1) / kTileRows);
  return s;
}

// A partial O: four heads' values of one dim side by side (what a thread of
// the tile kernel holds of them), dims next to each other: quad hq = head / 4.
__device__ __forceinline__ int part_at(int hq, int dim) { return hq * kDim + dim; }

// Slots of the partials: CTA c leaves at most two, 2c for a query that began
// in an earlier CTA and 2c + 1 for one that it begins and does not end.
__device__ __forceinline__ int part_slot(int c, bool begins) { return 2 * c + (begins ? 1 : 0); }

}  // namespace

// ---------------------------------------------------------------------------
// The tile kernel. Roles of a CTA's warps:
//   0 .. 7   math: softmax of a tile, and the outputs at a query's end
//   8 ..     producers: Q, and the rows of the tiles
//   last     (bf16) issues the tensor-core products, so that the next query's
//            scores come while this one's output is written. fp8 and fp4 have
//            eight producer warps, and a seventeenth warp would take a quarter
//            of everyone's registers: math warp 0 issues there.
// A tile's 512 channels are eight 64-channel blocks in eight slots of shared
// memory (the layout of attend_tile.cuh); full[b] says that block b of a tile
// has landed, empty[m] that the products of output dims 128 m .. have read
// blocks 2m and 2m + 1. QK^T runs block by block as they land, PV frees them
// two at a time, so that the next tile's rows load while this one's PV runs.
// Everything a role waits for, it waits for with a limit (wait_phase).
//
// The code that runs for every tile is kept small, its loops rolled: the roles
// run different code at the same time, and with everything unrolled the
// instruction cache missed one request in five (warps without an instruction
// were 2.3 times those that issued; a tile of bf16 rows took 8,850 cycles).
// ---------------------------------------------------------------------------
constexpr int kFirstProducer = kAttWarps;
template <int KVF>
struct Roles {
  // bf16 rows are copied by TMA; fp8 and fp4 rows pass through registers and
  // are converted there, which takes twice the warps
  static constexpr int kProducers = KVF == 0 ? 4 : 8;
  static constexpr int kProducerThreads = 32 * kProducers;
  static constexpr bool kOwnIssuer = KVF == 0;
  static constexpr int kIssuer = kFirstProducer + kProducers;  // warp, where it has one
  static constexpr int kThreads = 32 * (kFirstProducer + kProducers + (kOwnIssuer ? 1 : 0));
};

// shared memory behind attend_tile.cuh's layout
constexpr uint32_t SM_BAR = SM_TOTAL;                 // mbarriers
constexpr uint32_t SM_ROWOK = SM_BAR + 256;           // uint8 [2][128]: rows that are there, by the tile's parity
constexpr uint32_t SM_GONE = SM_ROWOK + 256;          // uint32 [2][4]: rows to be cleared, by the tile's parity
constexpr uint32_t SM_RUN = SM_GONE + 64;            // the CTA's run
constexpr uint32_t SM_ROWAT = SM_RUN + 256;           // int32 [2][128][2]: page and row in it of a tile's rows
constexpr uint32_t SM_ROPETAB = SM_ROWAT + 2048;      // float2 [4][32]: cos, sin of four queries' positions
constexpr uint32_t SM_PAGED_TOTAL = SM_ROPETAB + 1024;
constexpr uint32_t kPagedSmemBytes = SM_PAGED_TOTAL + 1024;

enum Bar : uint32_t { kFull = 0, kEmpty = 8, kQFull = 12, kQEmpty = 13, kScores = 14, kOut = 15, kWeights = 16, kDrained = 17, kCleared = 18, kBars = 22 };

// Bounded wait on an mbarrier phase: 100,000 suspensions of up to 20 us, then
// CSA2_FLAG_WAIT_TIMEOUT and false. (mbar_wait with its clock is 40
// instructions at each of a dozen places; see the note on code size below.)
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t phase, uint32_t* flags) {
#pragma unroll 1
  for (int i = 0; i < 100000; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(phase), "r"(20000u)
        : "memory");
    if (ok != 0u) return true;
  }
  set_flag(flags, CSA2_FLAG_WAIT_TIMEOUT);
  return false;
}
// A warp arrives once, and waits, by its first lane (an arrival of every lane
// is one atomic each, in turn).
__device__ __forceinline__ void warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0)
    asm volatile("{\n.reg .b64 t;\nmbarrier.arrive.shared::cta.b64 t, [%0];\n}" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t phase, uint32_t* flags) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_phase(bar, phase, flags);
  return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
}
// Tensor-core and TMA instructions take their operands from uniform registers:
// the warps that issue them run the issuing code whole, one lane's predicate
// on the instruction itself. (Inside a branch that one thread takes, every
// operand is moved over one by one: a product took 95 cycles instead of 48, a
// block's copy 230. The same holds for loops and branches on values that come
// from memory, which the compiler cannot know to be the same in every lane:
// they go through a shuffle or a vote first.)
__device__ __forceinline__ int uniform(int v, int lane = 0) { return __shfl_sync(0xffffffffu, v, lane); }
__device__ __forceinline__ bool uniform(bool v) { return __any_sync(0xffffffffu, v) != 0; }
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r;
}
__device__ __forceinline__ void mma_one(uint32_t leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p, e;\n"
      "setp.ne.u32 p, %4, 0;\n"
      "setp.ne.u32 e, %5, 0;\n"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ uint32_t phase_done(uint32_t bar, uint32_t phase) {
  uint32_t ok;
  asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(phase)
               : "memory");
  return ok;
}
// wait_phase by every lane of a warp
__device__ __forceinline__ bool wait_all_lanes(uint32_t bar, uint32_t phase, uint32_t* flags) {
  return __all_sync(0xffffffffu, wait_phase(bar, phase, flags)) != 0;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// largest value of the warp's lanes
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// named barrier 1: the 256 math threads
struct SyncMath {
  __device__ __forceinline__ void sync() const { asm volatile("bar.sync 1, 256;" ::: "memory"); }
  __device__ __forceinline__ bool any(bool v) const {
    uint32_t r;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, 1, 256, p;\nselp.u32 %0, 1, 0, q;\n}"
        : "=r"(r)
        : "r"((uint32_t)v)
        : "memory");
    return r != 0;
  }
};

// named barrier 2: the producer threads
template <int N>
__device__ __forceinline__ void sync_producers() {
  asm volatile("bar.sync 2, %0;" ::"n"(N) : "memory");
}
// How the tiles are cut into runs. On a line where a tile is kTileCost long and
// a query starts with kQueryCost (its Q, its first tile's references, an
// output or partial more), run c of `ctas` has the tiles that start in the
// c-th of equal parts. With fewer tiles than two a CTA, the queries' starts are
// left out: one tile a CTA where they suffice. Parts of a query lie in
// neighbouring CTAs, none of them empty: the parts are longer than a tile.
constexpr int kTileCost = 4, kQueryCost = 5;
// a / b of values >= 0: 32-bit where they fit (a 64-bit division is several
// hundred cycles, before any row is asked for)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// CTAs that share a tile, each with as many of its output dims: with fewer
// tiles than half or a quarter of the CTAs two or four of them form the same
// scores, and each has a share of the output's products and of its way out
// of tensor memory (a partial takes 4,600 cycles whole and 1,200 in quarters; one
// query over 2K rows 16.6 -> 14.5 us). As a shift: 2, 1 or 0.
__device__ __forceinline__ int dim_shift(int64_t tiles, int grid) { return 4 * tiles <= grid ? 2 : (2 * tiles <= grid ? 1 : 0); }
struct RunCut {
  int64_t cost;
  int ctas, start;  // ctas: runs (of 1 << dim_shift CTAs each); start: kQueryCost or 0
  // where query i starts, b tiles coming before it
  __device__ __forceinline__ int64_t at(int64_t b, int i) const { return kTileCost * b + (int64_t)start * i; }
  // Run c begins with the first tile whose place, ctas-fold, is y = c * cost
  // or more (products where the quotient's division would take as long as all
  // else); of a query of n tiles, this many come before it
  __device__ __forceinline__ int tiles_before(int64_t y, int64_t b, int i, int n) const {
    const int64_t left = y - ctas * (at(b, i) + start), step = kTileCost * ctas;
    return left <= 0 ? 0 : (int)min((int64_t)n, quotient(left + step - 1, step));
  }
  // run of tile j of query i
  __device__ __forceinline__ int run_of(int64_t b, int i, int j) const {
    return (int)quotient((at(b, i) + start + (int64_t)kTileCost * j) * ctas, cost);
  }
};
__device__ __forceinline__ RunCut run_cut(int64_t tiles, int n_query, int grid) {
  RunCut r;
  r.start = tiles > 2 * (int64_t)grid ? kQueryCost : 0;
  r.cost = kTileCost * tiles + (int64_t)r.start * n_query;
  r.ctas = (int)min((int64_t)(grid >> dim_shift(tiles, grid)), tiles);
  return r;
}

// The CTA's run of tiles, walked tile by tile; every role has its own.
struct Cursor {
  int64_t at, run1, q0;  // tile, end of the run, first tile of query qi
  int qi;
  QuerySpan span;
  __device__ __forceinline__ bool more() const { return at < run1; }
  __device__ __forceinline__ uint32_t tiles() const { return (uint32_t)uniform((int)(run1 - at)); }
  __device__ __forceinline__ int tile() const { return (int)(at - q0); }
  // the last tile of this query in the run
  __device__ __forceinline__ bool last() const { return uniform(at + 1 == run1 || at + 1 == q0 + span.n_tiles); }
  __device__ __forceinline__ void next(const PagedAttendParams& p) {
    ++at;
    if (at < run1 && at == q0 + span.n_tiles) {
      q0 = at;
      span = query_span(p, ++qi);
    }
  }
};

struct Run {
  Cursor cur;     // at the run's first tile
  int64_t total;  // tiles of all queries
  int index;      // the run's number
  int m0, m1;     // this CTA's output dims, 128 m0 .. 128 m1
};
static_assert(sizeof(Run) <= 256, "SM_RUN");

__device__ __forceinline__ void expect_one(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n.reg .b64 t;\n.reg .pred e;\nsetp.ne.u32 e, %2, 0;\n@e mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n}" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_2d_one(uint32_t leader, uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %5, 0;\n"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_3d_one(uint32_t leader, uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                           uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %6, 0;\n"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(leader)
      : "memory");
}

// Q of a query: its plain 64-channel blocks by TMA, its rope channels (the
// last block) rotated and split into hi + lo (see q_rope_split) by the
// producer threads (t: index among N, warp: a uniform register's t / 32). The
// (cos, sin) of the query's position are formed once, a pair a lane of the last
// warp (freq: that lane's frequency), and left for the outputs' rotation back
// (seg: the query's number in the run; four tables in turn: the output of one
// query may still be written while the Q of the second after it arrives).
// kQFull completes when all is there. ask() puts the loads under way, take() waits for them.
template <int N>
struct QLoad {
  uint4 v[8 * kHeads / N];
  double freq;
  __device__ __forceinline__ void ask(const PagedAttendParams& p, uint8_t* sm, uint32_t base_s, int qi, int64_t pos, uint32_t seg,
                                      int t, int warp) {
    const uint32_t bar = base_s + SM_BAR + 8 * kQFull;
    const bool rope = p.a.rp.pairs > 0;
    if (warp == 0) {
      const uint32_t leader = elect_one();
      const int plain = rope ? 7 : 8;
      expect_one(leader, bar, 8192u * plain);
#pragma unroll 1
      for (int b = 0; b < plain; ++b) tma_2d_one(leader, base_s + SM_Q + 8192u * b, &p.q_map, 64 * b, kHeads * uniform(qi), bar);
    }
    if (rope) {
      // thread: chunk 56 + (t & 7) of heads t >> 3, ...: always the same four pairs
      const uint16_t* q = p.a.q + (int64_t)qi * kHeads * kDim + 8 * (56 + (t & 7));
#pragma unroll
      for (int u = 0; u < 8 * kHeads / N; ++u) v[u] = *reinterpret_cast<const uint4*>(q + (int64_t)((t >> 3) + u * (N / 8)) * kDim);
      if (warp == N / 32 - 1) {
        float cs, sn;
        angle_cs((double)max(pos, (int64_t)0) * freq, cs, sn);
        reinterpret_cast<float2*>(sm + SM_ROPETAB)[32 * (seg & 3u) + (t & 31)] = make_float2(cs, sn);
      }
    }
  }
  __device__ __forceinline__ void take(const PagedAttendParams& p, uint8_t* sm, uint32_t base_s, uint32_t seg, int t) {
    if (p.a.rp.pairs > 0) {
      const int c = 56 + (t & 7);
      const float2* table = reinterpret_cast<const float2*>(sm + SM_ROPETAB) + 32 * (seg & 3u);
      sync_producers<N>();
#pragma unroll
      for (int u = 0; u < 8 * kHeads / N; ++u) {
        const int h = (t >> 3) + u * (N / 8);
        uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w}, lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 cs = table[4 * (t & 7) + k];
          const float x0 = bf16lo(w[k]), x1 = bf16hi(w[k]);
          const float y0 = x0 * cs.x - x1 * cs.y, y1 = x0 * cs.y + x1 * cs.x;
          w[k] = pack_bf16(y0, y1);
          lo[k] = pack_bf16(y0 - bf16lo(w[k]), y1 - bf16hi(w[k]));
        }
        const uint32_t at = (uint32_t)h * 128u + ((uint32_t)((c & 7) ^ (h & 7)) << 4);
        *reinterpret_cast<uint4*>(sm + SM_Q + 7u * 8192u + at) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(sm + SM_Q + 8u * 8192u + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
    }
    warp_arrive(base_s + SM_BAR + 8 * kQFull);
  }
};

// Row r of the cursor's tile: the page of its chunk and the row in it (page -1:
// the query has no such chunk, or its page is missing), and whether the query
// sees it.
struct RowAt {
  int32_t page, in_page;
  bool seen;
  __device__ __forceinline__ bool there() const { return seen && page >= 0; }
};
__device__ __forceinline__ RowAt row_at(const PagedAttendParams& p, const Cursor& cur, int r) {
  const int cs = chunk_shift(p.kv.page_shift);
  const Visible& v = cur.span.vis;
  const int i = cur.tile() * kTileRows + r, k = i >> cs;
  const bool have = k < v.n_chunks;
  const int32_t pos = have ? chunk_pos(v, k, i & ((1 << cs) - 1), cs) : 0;
  RowAt a;
  a.seen = have && is_seen(v, pos);
  a.in_page = pos & ((1 << p.kv.page_shift) - 1);
  a.page = have ? page_of(p.kv, cur.span.b, pos) : -1;
  return a;
}

// 16 zero bytes into shared memory if hit != 0, without a branch
__device__ __forceinline__ void zero16_if(uint32_t hit, uint32_t dst) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %0, 0;\n@p st.shared.v4.u32 [%1], {%2, %2, %2, %2};\n}" ::"r"(hit), "r"(dst), "r"(0u)
               : "memory");
}

__device__ __forceinline__ void prefetch_l2_line(const void* ptr) { asm volatile("prefetch.global.L2 [%0];" ::"l"(ptr)); }
__device__ __forceinline__ void prefetch_l2(const void* ptr, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ptr), "r"(bytes) : "memory");
}

// bf16 producers. Thread t finds row t of a tile one tile ahead and the first
// row of each chunk asks for the chunk in L2: shared memory holds one tile, so
// that the memory would idle between a tile's last block and its first PV;
// with the next tile on its way to L2 it does not. Warp w copies blocks 2w and
// 2w + 1 by TMA, chunk by chunk, as soon as their slots are free (TMA:
// chunks of at least the 8 rows of a swizzle atom; smaller ones are copied by
// the threads, 16 bytes each). Chunks that the tile lacks, or whose pages are
// missing, are read past the pages' end, where TMA writes zeros; rows of a
// chunk that are not the query's are cleared after they land: their weights are
// 0, but 0 times a NaN is not.
template <int N, bool TMA>
__device__ __forceinline__ void produce_bf16(const PagedAttendParams& p, uint8_t* sm, uint32_t base_s, Cursor cur, int t,
                                             int warp, double freq) {
  static_assert(N == kTileRows);
  const uint32_t bars = base_s + SM_BAR;
  const int lane = t & 31;
  const int cs = chunk_shift(p.kv.page_shift);
  const int n_ch = kTileRows >> cs;  // chunks of a tile
  int2* at = reinterpret_cast<int2*>(sm + SM_ROWAT);
  uint32_t* gone = reinterpret_cast<uint32_t*>(sm + SM_GONE);  // rows to be cleared, a bit each
  QLoad<N> ql;
  ql.freq = freq;
  RowAt mine = row_at(p, cur, t);
  // this thread's row of tile n: what math and the copies need to know of it
  auto publish = [&](uint32_t n) {
    if (mine.page >= 0 && (t & ((1 << cs) - 1)) == 0)
      prefetch_l2(p.kv.pages + mine.page * p.kv.page_stride + (int64_t)mine.in_page * 1024, 1024u << cs);
    if (mine.seen && mine.page < 0) set_flag(p.a.flags, CSA2_FLAG_BAD_PAGE);
    at[128 * (n & 1u) + t] = make_int2(mine.page, mine.in_page);
    sm[SM_ROWOK + 128 * (n & 1u) + t] = mine.there();
    const uint32_t bits = __ballot_sync(0xffffffffu, mine.page >= 0 && !mine.seen);
    if (lane == 0) gone[4 * (n & 1u) + warp] = bits;
    sync_producers<N>();
  };
  publish(0);
  bool first = true, live = true;  // live: see math_role
  uint32_t seg = 0, n = 0;
  const uint32_t leader = elect_one();
  const uint32_t tiles = cur.tiles();
#pragma unroll 1
  for (; n < tiles; ++n) {
    const bool q_here = first;
    first = cur.last();
    // Q comes before the rows, whose slots are free later; at the run's start,
    // where both are, the rows come first: memory is the slower
    if (q_here && n > 0) {
      live = live && wait_all_lanes(bars + 8 * kQEmpty, (seg & 1u) ^ 1u, p.a.flags);
      ql.ask(p, sm, base_s, cur.qi, cur.span.t, seg, t, warp);
      ql.take(p, sm, base_s, seg, t);
    }
    if constexpr (TMA) {
      // lane k has chunk k
      int2 src = lane < n_ch ? at[128 * (n & 1u) + (lane << cs)] : make_int2(0, 0);
      if (src.x < 0) src = make_int2(p.kv.n_pages, 0);  // past the end: zeros
      if (n > 0) live = live && wait_all_lanes(bars + 8 * (kEmpty + warp), (n & 1u) ^ 1u, p.a.flags);
      if (live) {
        const uint32_t full = bars + 8 * (kFull + 2 * warp), dst = base_s + SM_KV + (uint32_t)(2 * warp) * 16384u;
        expect_one(leader, full, 16384u);
        expect_one(leader, full + 8, 16384u);
#pragma unroll 2
        for (int k = 0; k < n_ch; ++k) {
          const int page = uniform(src.x, k), row = uniform(src.y, k);
          tma_3d_one(leader, dst + ((uint32_t)k << (7 + cs)), &p.kv_map, 128 * warp, row, page, full);
          tma_3d_one(leader, dst + 16384u + ((uint32_t)k << (7 + cs)), &p.kv_map, 128 * warp + 64, row, page, full + 8);
        }
      }
    } else {
      int64_t src[8];  // rows t >> 3, + 16, ...: 16-byte chunk t & 7 of every block
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int r = (t >> 3) + 16 * u;
        const int2 a = at[128 * (n & 1u) + r];
        src[u] = sm[SM_ROWOK + 128 * (n & 1u) + r] ? a.x * p.kv.page_stride + (int64_t)a.y * 1024 + 16 * (t & 7) : -1;
      }
#pragma unroll 1
      for (int b = 0; b < 8; ++b) {
        if (b % 2 == 0 && n > 0) live = live && warp_wait(bars + 8 * (kEmpty + b / 2), (n & 1u) ^ 1u, p.a.flags);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = (t >> 3) + 16 * u;
          cp_async16(base_s + SM_KV + (uint32_t)b * 16384u + (uint32_t)r * 128u + ((uint32_t)((t & 7) ^ (r & 7)) << 4),
                     p.kv.pages + (src[u] >= 0 ? src[u] + 128 * b : 0), src[u] >= 0 ? 16u : 0u);
        }
      }
      cp_async_wait_all();
      fence_proxy_async_smem();
#pragma unroll 1
      for (int b = 0; b < 8; ++b) warp_arrive(bars + 8 * (kFull + b));
    }
    if (q_here && n == 0) {
      ql.ask(p, sm, base_s, cur.qi, cur.span.t, seg, t, warp);
      ql.take(p, sm, base_s, seg, t);
    }
    if (q_here) ++seg;
    if constexpr (TMA) {
      // this warp's two blocks, four rows a store: eight lanes a row
      const uint4 g = *reinterpret_cast<const uint4*>(gone + 4 * (n & 1u));
      if (uniform((g.x | g.y | g.z | g.w) != 0u)) {
        for (int b = 2 * warp; b < 2 * warp + 2; ++b) live = live && wait_all_lanes(bars + 8 * (kFull + b), n & 1u, p.a.flags);
        const uint32_t dst = base_s + SM_KV + (uint32_t)(2 * warp) * 16384u + 16u * lane;
#pragma unroll
        for (int i = 0; i < kTileRows / 4; ++i) {
          const uint32_t bits = i < 8 ? g.x : (i < 16 ? g.y : (i < 24 ? g.z : g.w));
          const uint32_t hit = (bits >> (4 * (i & 7) + (lane >> 3))) & 1u;
          zero16_if(hit, dst + 512u * i);
          zero16_if(hit, dst + 512u * i + 16384u);
        }
        fence_proxy_async_smem();
      }
      warp_arrive(bars + 8 * (kCleared + warp));
    }
    cur.next(p);
    if (cur.more()) mine = row_at(p, cur, t);
    if (first && t == 0 && cur.more()) prefetch_l2(p.a.q + (int64_t)cur.qi * kHeads * kDim, 2u * kHeads * kDim);
    if (cur.more()) publish(n + 1);
  }
  if (!live && TMA && n > 0) {  // no copy may still be landing when the CTA exits
    warp_wait(bars + 8 * kQFull, (seg - 1) & 1u, p.a.flags);
    for (int b = 0; b < 8 && warp_wait(bars + 8 * (kFull + b), (n - 1) & 1u, p.a.flags); ++b) {}
  }
}

// 16 bf16 channels (two 16-byte chunks) from 16 e4m3 codes and their scale, by
// the hardware's conversions (72 cycles a warp and 16 values; assembling the
// bits with integer operations and one bf16 product took 91).
__device__ __forceinline__ void fp8_to_bf16(const uint4& codes, uint32_t scale, uint32_t (&o)[8]) {
  const float sc = ue8m0_value(scale);
  const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 a = e4m3x2_to_float2((uint16_t)(cw[k] & 0xFFFFu));
    const float2 b = e4m3x2_to_float2((uint16_t)(cw[k] >> 16));
    o[2 * k] = pack_bf16(a.x * sc, a.y * sc);
    o[2 * k + 1] = pack_bf16(b.x * sc, b.y * sc);
  }
}
// 16 bf16 channels from 16 E2M1 codes and their e4m3 scale (at most 6
// significant bits: exact)
__device__ __forceinline__ void fp4_to_bf16(uint32_t lo, uint32_t hi, uint32_t scale, uint32_t (&o)[8]) {
  const float sc = e4m3_value(scale);
  uint32_t h[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    e2m1x8_to_f16x2x4_cvt(k == 0 ? lo : hi, h);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      __half2_raw r;
      r.x = (unsigned short)(h[u] & 0xFFFFu);
      r.y = (unsigned short)(h[u] >> 16);
      const float2 f = __half22float2(__half2(r));
      o[4 * k + u] = pack_bf16(f.x * sc, f.y * sc);
    }
  }
}

// fp8 / fp4 producers: the codes pass through registers, a pair of blocks ahead
// of the conversion, and are asked for in L2 two tiles earlier (loads that
// wait for memory hold up the queue that the math warps' shared-memory and
// tensor-memory loads go through). Four pairs take 5,200 of a tile's 8,700
// cycles; with no conversion at all it would be 8,400: the stores share shared
// memory with the products, and a pair's registers are loaded again only when
// they have been converted. More pairs ahead spill (128 registers a thread);
// converted pairs kept in the free columns of tensor memory spill too and took
// 274 to 333 us where this took 265 (8 x 128K rows; fp4 as it stands spills 76
// bytes a thread, fp8 nothing). Of a pair of blocks thread t has 16
// channels, chunk t & 7, of rows t >> 3, + 32, ...: a load takes whole 128-byte
// lines (fp8) of four rows.
template <int KVF, int N>
__device__ __forceinline__ void produce_codes(const PagedAttendParams& p, uint8_t* sm, uint32_t base_s, Cursor cur, int t,
                                              int warp, double freq) {
  constexpr int kRowBytes = KVF == 1 ? 512 : 256, kScaleBytes = KVF == 1 ? 16 : 32;
  constexpr int R = kTileRows * 8 / N;  // rows of a thread
  using Code = typename std::conditional<KVF == 1, uint4, uint2>::type;
  const uint32_t bars = base_s + SM_BAR;
  const int c = t & 7, row0 = t >> 3;
  const int cs = chunk_shift(p.kv.page_shift);
  int2* at = reinterpret_cast<int2*>(sm + SM_ROWAT);
  Cursor ahead = cur;  // the tile whose rows are found next
  // threads 0 .. 127: row t of tile n, two tiles before its conversion
  auto publish = [&](uint32_t n) {
    if (t < kTileRows && ahead.more()) {
      const RowAt mine = row_at(p, ahead, t);
      if (mine.page >= 0 && (t & ((1 << cs) - 1)) == 0) {
        prefetch_l2(p.kv.pages + mine.page * p.kv.page_stride + (int64_t)mine.in_page * kRowBytes, (uint32_t)kRowBytes << cs);
        prefetch_l2(p.kv.scales + mine.page * p.kv.scale_stride + (int64_t)mine.in_page * kScaleBytes, (uint32_t)kScaleBytes << cs);
      }
      if (mine.seen && mine.page < 0) set_flag(p.a.flags, CSA2_FLAG_BAD_PAGE);
      at[128 * (n & 1u) + t] = mine.there() ? make_int2(mine.page, mine.in_page) : make_int2(-1, 0);
    }
    if (ahead.more()) ahead.next(p);
    sync_producers<N>();
  };
  // a thread's codes and scale bytes of one tile; codes null: the row is not there
  struct Rows {
    const uint8_t* codes[R];
    const uint8_t* scale[R];
  };
  auto find = [&](uint32_t n, Rows& r) {
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int2 a = at[128 * (n & 1u) + row0 + u * (N / 8)];
      r.codes[u] = a.x >= 0 ? p.kv.pages + a.x * p.kv.page_stride + (int64_t)a.y * kRowBytes + (kRowBytes / 32) * c : nullptr;
      r.scale[u] = a.x >= 0 ? p.kv.scales + a.x * p.kv.scale_stride + (int64_t)a.y * kScaleBytes + (KVF == 1 ? c >> 1 : c) : nullptr;
    }
  };
  Code code[2][R];
  uint8_t scale[2][R];
  auto load = [&](const Rows& r, int m, int slot) {  // pair m into register set `slot`
#pragma unroll
    for (int u = 0; u < R; ++u) {
      if constexpr (KVF == 1) code[slot][u] = r.codes[u] != nullptr ? ldg_stream16(r.codes[u] + 128 * m) : make_uint4(0u, 0u, 0u, 0u);
      else code[slot][u] = r.codes[u] != nullptr ? ldg_stream8(r.codes[u] + 64 * m) : make_uint2(0u, 0u);
      scale[slot][u] = r.codes[u] != nullptr ? __ldg(r.scale[u] + (kScaleBytes / 4) * m) : 0;
    }
  };
  QLoad<N> ql;
  ql.freq = freq;
  Rows now;
  publish(0);
  ql.ask(p, sm, base_s, cur.qi, cur.span.t, 0u, t, warp);
  find(0, now);
  load(now, 0, 0);
  load(now, 1, 1);
  publish(1);
  bool first = true, live = true;  // live: see math_role
  const uint32_t tiles = cur.tiles();
#pragma unroll 1
  for (uint32_t n = 0, seg = 0; n < tiles; ++n) {
    const bool more = n + 1 < tiles;
    if (first) {
      if (seg > 0) {
        live = live && warp_wait(bars + 8 * kQEmpty, (seg & 1u) ^ 1u, p.a.flags);
        ql.ask(p, sm, base_s, cur.qi, cur.span.t, seg, t, warp);
      }
      ql.take(p, sm, base_s, seg, t);
      ++seg;
    }
    first = cur.last();
    // (a look at a barrier takes some 300 cycles: the next pair's is under way
    // while this one is converted)
    uint32_t free = n == 0 ? 1u : phase_done(bars + 8 * kEmpty, (n & 1u) ^ 1u);
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int m = 2 * half + j;
        if (!uniform(free != 0u)) live = live && warp_wait(bars + 8 * (kEmpty + m), (n & 1u) ^ 1u, p.a.flags);
        if (n > 0 && m < 3) free = phase_done(bars + 8 * (kEmpty + m + 1), (n & 1u) ^ 1u);
#pragma unroll
        for (int u = 0; u < R; ++u) {
          const int r = row0 + u * (N / 8);
          if (m == 0 && c == 0) sm[SM_ROWOK + 128 * (n & 1u) + r] = now.codes[u] != nullptr;
          uint32_t o[8];
          if constexpr (KVF == 1) fp8_to_bf16(code[j][u], scale[j][u], o);
          else fp4_to_bf16(code[j][u].x, code[j][u].y, scale[j][u], o);
          uint8_t* dst = sm + SM_KV + (uint32_t)(2 * m + (c >> 2)) * 16384u + (uint32_t)r * 128u;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<uint4*>(dst + (((2 * (c & 3) + k) ^ (r & 7)) << 4)) =
                make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
        }
        fence_proxy_async_smem();
        warp_arrive(bars + 8 * (kFull + 2 * m));
        warp_arrive(bars + 8 * (kFull + 2 * m + 1));
        if (half == 0) load(now, 2 + j, j);
      }
    }
    if (more) {
      find(n + 1, now);
      load(now, 0, 0);
      load(now, 1, 1);
    }
    cur.next(p);
    if (first && t == 0 && more) prefetch_l2(p.a.q + (int64_t)cur.qi * kHeads * kDim, 2u * kHeads * kDim);
    if (more) publish(n + 2);
  }
}

// The products of one tile, by one warp (leader: 1 in the lane that issues);
// false: a wait ran out and nothing more was issued. n: the tile's number in
// the run, seg: its query's.
template <bool SPLIT>  // whether CTAs share tiles (dim_shift)
struct Issuer {
  uint32_t bars, tmem_s, tmem_o, base_s, leader;
  uint32_t* flags;
  const uint4* gone;  // by the tile's parity; null: no rows are cleared after they land
  bool rope;
  uint32_t m0, m1;  // this CTA's output dims, 128 m0 .. 128 m1
  // S^T = KV Q^T, block by block as the rows land; the rope channels once more
  // against q's residual
  __device__ __forceinline__ bool scores(uint32_t n, uint32_t seg, bool first, bool last) const {
    const uint64_t kv = sdesc_sw128(base_s + SM_KV, 16u, 1024u), q = sdesc_sw128(base_s + SM_Q, 16u, 1024u);
    if (first && !wait_all_lanes(bars + 8 * kQFull, seg & 1u, flags)) return false;
    // a block's barrier is looked at while the products of the block before
    // are issued (a look takes 200 cycles from the instruction to the branch)
    uint32_t landed = phase_done(bars + 8 * kFull, n & 1u);
    bool clear = false;
#pragma unroll
    for (uint32_t b = 0; b < 8; ++b) {
      if (!uniform(landed != 0u) && !wait_all_lanes(bars + 8 * (kFull + b), n & 1u, flags)) return false;
      if (b == 0 && gone != nullptr) {
        const uint4 g = gone[n & 1u];
        clear = uniform((g.x | g.y | g.z | g.w) != 0u);
      }
      if (b % 2 == 0 && clear && !wait_all_lanes(bars + 8 * (kCleared + b / 2), n & 1u, flags)) return false;
      if (b < 7) landed = phase_done(bars + 8 * (kFull + b + 1), n & 1u);
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        mma_one(leader, tmem_s, sdesc_add(kv, b * 16384u + 32u * k), sdesc_add(q, b * 8192u + 32u * k), kIdescQK, b | k);
    }
    if (rope) {
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k)
        mma_one(leader, tmem_s, sdesc_add(kv, 7u * 16384u + 32u * k), sdesc_add(q, 8u * 8192u + 32u * k), kIdescQK, 1u);
    }
    commit_one(leader, bars + 8 * kScores);
    if (last) commit_one(leader, bars + 8 * kQEmpty);
    return true;
  }
  // O^T (+)= KV^T P^T, 128 output dims at a time
  __device__ __forceinline__ void output(bool first, bool last) const {
    const uint64_t kv = sdesc_sw128(base_s + SM_KV, 16384u, 1024u), pt = sdesc_sw128(base_s + SM_P, 8192u, 1024u);
    tc_fence_after();
    auto dims = [&](uint32_t m) {
#pragma unroll
      for (uint32_t k = 0; k < 8; ++k)
        mma_one(leader, tmem_o + 64u * m, sdesc_add(kv, m * 32768u + 2048u * k), sdesc_add(pt, 2048u * k), kIdescPV,
                k > 0 || !first ? 1u : 0u);
    };
    if constexpr (SPLIT) {
#pragma unroll 1
      for (uint32_t m = m0; m < m1; ++m) dims(m);
#pragma unroll 1
      for (uint32_t m = 0; m < 4; ++m) commit_one(leader, bars + 8 * (kEmpty + m));
    } else {
#pragma unroll
      for (uint32_t m = 0; m < 4; ++m) {
        dims(m);
        commit_one(leader, bars + 8 * (kEmpty + m));
      }
    }
    if (last) commit_one(leader, bars + 8 * kOut);
  }
  // after a wait that ran out: products still in flight land before tensor memory is freed
  __device__ __forceinline__ void drain() const {
    commit_one(leader, bars + 8 * kDrained);
    wait_phase(bars + 8 * kDrained, 0u, flags);
  }
};

// The products of a run, by the issuing warp.
template <bool SPLIT>
__device__ __forceinline__ void issue_role(const Issuer<SPLIT>& mma, Cursor cur, const PagedAttendParams& p) {
  const uint32_t tiles = cur.tiles();
  bool live = true, first = true;
#pragma unroll 1
  for (uint32_t n = 0, seg = 0; n < tiles; ++n) {
    const bool last = cur.last();
    if (live) live = uniform(mma.scores(n, seg, first, last));
    cur.next(p);  // the next query is looked up while the weights are formed
    if (live) live = wait_all_lanes(mma.bars + 8 * kWeights, n & 1u, mma.flags);
    if (live) mma.output(first, last);
    first = last;
    seg += last ? 1u : 0u;
  }
  if (!live) mma.drain();
}

// A head's reference moves only when a row's score exceeds it by more than
// this (log2 units). Weights then reach 2^32, which bf16 and fp32 hold with
// the same relative precision as weights below 1, and rows whose weight
// underflows are 2^-126 of the reference's. With 2^8 a few rows four times as
// large as the others moved some head's reference in nearly every tile, at
// 1.0 us a move (decode of 128K rows, fp8). The price: an output sums up to 2^32
// times what it would with the exact maximum before it is divided, so n rows
// above 2^95 / n in size can overflow to an infinity.
constexpr float kRefSlack = 32.f;
// What scores are taken against while no row has set a head's reference (its
// rows so far are missing, or -inf or NaN): the first finite one exceeds it.
constexpr float kNoRef = -1e38f;

// Softmax of one tile (thread: row = TMEM lane, heads 32 hh .. +31 of warp w,
// hh = w / 4) and, at a query's end, its output or partial. Most tiles need
// one vote on the references and neither a reduction nor a rescale; the
// weights are summed in fp32 and rounded to bf16 for the product.
// ISSUE: warp 0 issues the products too.
template <bool ISSUE, bool SPLIT>
__device__ __forceinline__ void math_role(const PagedAttendParams& p, uint8_t* sm, uint32_t base_s, uint32_t tmem_s,
                                          uint32_t tmem_o, const Issuer<SPLIT>& mma, Cursor cur, const Run& run, int warp) {
  const SyncMath sy;
  const uint32_t bars = base_s + SM_BAR;
  const int tid = threadIdx.x, lane = tid & 31;
  const int quad = warp & 3, hh = warp >> 2, row = quad * 32 + lane;
  const uint32_t lane_base = (uint32_t)(quad * 32) << 16;
  float* red = reinterpret_cast<float*>(sm + SM_RED);
  float* m_run = reinterpret_cast<float*>(sm + SM_MRUN);
  float* m_use = reinterpret_cast<float*>(sm + SM_MUSE);
  float* alpha = reinterpret_cast<float*>(sm + SM_ALPHA);
  const float4* mu4 = reinterpret_cast<const float4*>(m_use + 32 * hh);
  const float scale = p.a.scale_log2;
  const bool by_query = p.a.n_query < (int)gridDim.x;  // a join's index: its query, or the CTA that begins it
  const int m0 = SPLIT ? run.m0 : 0, m1 = SPLIT ? run.m1 : 4;
  int2 my_join = make_int2(-1, -1);
  int my_query = -1;
  float lsum[32];
  bool first = true, begins = false;
  // A wait that ran out is recorded; from then on nothing is waited for or
  // issued, and the loop only runs out, all threads meeting at its barriers.
  bool live = true;
  const uint32_t tiles = cur.tiles();
#pragma unroll 1
  for (uint32_t n = 0, seg = 0; n < tiles; ++n) {
    const bool last = cur.last();
    if (ISSUE && warp == 0 && live) live = uniform(mma.scores(n, seg, first, last));
    if (first) {
      begins = cur.tile() == 0;
      const bool ends = cur.q0 + cur.span.n_tiles <= cur.run1;
      if (begins && tid == 0 && m0 == 0) {
        const QuerySpan& s = cur.span;
        const bool seq_ok = s.b >= 0 && s.b < p.kv.n_seq;
        if (s.b != -1 && !(seq_ok && s.t >= -1)) set_flag(p.a.flags, CSA2_FLAG_BAD_QUERY);
        if (s.ok && s.vis.past_table) set_flag(p.a.flags, CSA2_FLAG_BAD_PAGE);
        const int2 jn = ends ? make_int2(-1, -1)
                             : make_int2(run.index, run_cut(run.total, p.a.n_query, (int)gridDim.x).run_of(cur.q0, cur.qi, s.n_tiles - 1));
        if (by_query) {
          p.joins[cur.qi] = make_int4(jn.x, jn.y, cur.qi, 0);
        } else if (!ends) {
          my_join = jn;
          my_query = cur.qi;
        }
      }
      if (tid < kHeads) {
        m_run[tid] = -INFINITY;
        m_use[tid] = kNoRef;
      }
#pragma unroll
      for (int k = 0; k < 32; ++k) lsum[k] = 0.f;
      sy.sync();
    }
    live = live && warp_wait(bars + 8 * kScores, n & 1u, p.a.flags);
    live = live && warp_wait(bars + 8 * kFull, n & 1u, p.a.flags);  // the producers' row flags and rope table
    tc_fence_after();
    const bool valid = sm[SM_ROWOK + 128 * (n & 1u) + row] != 0;
    // Weights from the references as they stand, and with the barrier that
    // hands them to the products a vote whether a row exceeded one: then (and
    // at a query's first tile) the references move and the weights are formed
    // once more.
    float x[32];  // score - reference (log2 units) of this row and 32 heads, then its weight
    bool move = first;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      if (move) {
        uint32_t r[32];
        tmem_ld32(tmem_s + lane_base + 32 * hh, r);
        tmem_wait_ld();
        // the largest of each head: over this warp's rows (lane k keeps head k), then over the four quadrants
        float mine = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const float v = warp_max(valid ? __uint_as_float(r[k]) * scale : -INFINITY);
          if (lane == k) mine = v;
        }
        red[quad * 64 + 32 * hh + lane] = mine;
        sy.sync();
        bool moved = false;
        if (tid < kHeads) {
          const float top = fmaxf(fmaxf(red[tid], red[64 + tid]), fmaxf(red[128 + tid], red[192 + tid]));
          const float mo = m_run[tid];
          const float mn = (mo == -INFINITY || top > mo + kRefSlack) ? fmaxf(mo, top) : mo;
          const float al = (mo == -INFINITY) ? 1.f : exp2f(mo - mn);
          m_use[tid] = mn == -INFINITY ? kNoRef : mn;
          alpha[tid] = al;
          m_run[tid] = mn;
          moved = al != 1.f;
        }
        if (sy.any(moved)) {
#pragma unroll
          for (int k = 0; k < 32; ++k) lsum[k] *= alpha[32 * hh + k];
          // (the products before this tile's scores are complete: they came first)
#pragma unroll 1
          for (int mt = m0; mt < m1; ++mt) {
            const uint32_t a = tmem_o + (uint32_t)(64 * mt + 32 * hh) + lane_base;
            tmem_ld32(a, r);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha[32 * hh + k]);
            tmem_st32(a, r);
          }
          tmem_wait_st();
        }
      }
      {
        uint32_t r[32];
        tmem_ld32(tmem_s + lane_base + 32 * hh, r);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 m = mu4[k];
          x[4 * k] = fmaf(__uint_as_float(r[4 * k]), scale, -m.x);
          x[4 * k + 1] = fmaf(__uint_as_float(r[4 * k + 1]), scale, -m.y);
          x[4 * k + 2] = fmaf(__uint_as_float(r[4 * k + 2]), scale, -m.z);
          x[4 * k + 3] = fmaf(__uint_as_float(r[4 * k + 3]), scale, -m.w);
        }
      }
      float over = x[0];
#pragma unroll
      for (int k = 1; k < 32; ++k) over = fmaxf(over, x[k]);
      uint32_t packed[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        x[2 * k] = exp2_approx(x[2 * k]);
        x[2 * k + 1] = exp2_approx(x[2 * k + 1]);
        packed[k] = valid ? pack_bf16(x[2 * k], x[2 * k + 1]) : 0u;
      }
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) {
        const int c = 4 * hh + c4;
        *reinterpret_cast<uint4*>(sm + SM_P + (uint32_t)row * 128u + ((uint32_t)(c ^ (row & 7)) << 4)) =
            make_uint4(packed[4 * c4], packed[4 * c4 + 1], packed[4 * c4 + 2], packed[4 * c4 + 3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      move = sy.any(valid && over > kRefSlack);
      if (!move) break;
    }
    if (!ISSUE) warp_arrive(bars + 8 * kWeights);
    else if (warp == 0 && live) mma.output(first, last);
    if (valid) {
#pragma unroll
      for (int k = 0; k < 32; ++k) lsum[k] += x[k];
    }
    first = false;
    if (last) {
      const bool whole = begins && cur.q0 + cur.span.n_tiles <= cur.run1;
      red[quad * 64 + 32 * hh + lane] = reduce_scatter32<false>(lsum, lane);
      sy.sync();
      if (tid < kHeads) {
        const float l = red[tid] + red[64 + tid] + red[128 + tid] + red[192 + tid];
        const float mr = m_run[tid];
        if (whole) {
          // fo = e^{m - M} / den, den = l e^{m - M} + e^{sink - M}
          const float sk = p.a.sink != nullptr ? p.a.sink[tid] : -INFINITY, sk2 = sk * 1.4426950408889634f;
          const float M = fmaxf(mr, sk2);
          float fo = 0.f, lse = sk;  // no row seen: the denominator is the sink's
          if (mr != -INFINITY || l != l) {  // (scores that are all NaN set no reference)
            const float em = exp2f(mr - M);
            const float den = l * em + exp2f(sk2 - M);
            fo = em / den;
            lse = (M + log2f(den)) * 0.6931471805599453f;
          }
          alpha[tid] = fo;
          if (p.a.lse != nullptr && cur.span.b != -1 && m0 == 0) p.a.lse[(int64_t)cur.qi * kHeads + tid] = lse;
        } else {
          const int64_t at = (int64_t)part_slot(run.index, begins) * kHeads + tid;
          if (m0 == 0) {
            p.a.part_m[at] = mr;
            p.a.part_l[at] = l;
          }
        }
      }
      sy.sync();
      const int qi = cur.qi;
      const bool padding = cur.span.b == -1;
      cur.next(p);  // the next query is looked up while the products run
      live = live && warp_wait(bars + 8 * kOut, seg & 1u, p.a.flags);
      tc_fence_after();
      const float2* rope_tab = reinterpret_cast<const float2*>(sm + SM_ROPETAB) + 32 * (seg & 3u);
      const int first_rope = kDim - 2 * p.a.rp.pairs;
      if (!whole) {
        float* po = p.a.part_o + (int64_t)part_slot(run.index, begins) * kHeads * kDim;
#pragma unroll 1
        for (int mt = m0; mt < m1; ++mt) {
          uint32_t r[32];
          tmem_ld32(tmem_o + (uint32_t)(64 * mt + 32 * hh) + lane_base, r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            reinterpret_cast<uint4*>(po)[part_at(8 * hh + k, 128 * mt + row)] =
                make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
        }
      } else if (!padding) {
        // Lanes hold neighbouring dims: a pair of lanes swaps so that the even
        // one has two dims of one head and the odd one of the next, and each
        // store instruction writes 64 bytes of two heads. (Staged through shared
        // memory for 16-byte stores, with two barriers a block of 128 dims, an
        // output took 8,200 cycles, more than a tile.)
        uint32_t* out = reinterpret_cast<uint32_t*>(p.a.out + (int64_t)qi * kHeads * kDim);
        const bool odd = (lane & 1) != 0;
#pragma unroll 1
        for (int mt = m0; mt < m1; ++mt) {
          const int d = 128 * mt + row;
          uint32_t r[32];
          tmem_ld32(tmem_o + (uint32_t)(64 * mt + 32 * hh) + lane_base, r);
          tmem_wait_ld();
          float v[32];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 f = *reinterpret_cast<const float4*>(alpha + 32 * hh + 4 * k);
            v[4 * k] = __uint_as_float(r[4 * k]) * f.x;
            v[4 * k + 1] = __uint_as_float(r[4 * k + 1]) * f.y;
            v[4 * k + 2] = __uint_as_float(r[4 * k + 2]) * f.z;
            v[4 * k + 3] = __uint_as_float(r[4 * k + 3]) * f.w;
          }
          // rope channels rotated back by -t: only warps that hold some
          // exchange values with the pair's other lane (warp-uniform test)
          if (p.a.rp.pairs > 0 && 128 * mt + 32 * quad + 31 >= first_rope) {
            const bool rope = d >= first_rope;
            const float2 cs = rope ? rope_tab[(d - first_rope) >> 1] : make_float2(1.f, 0.f);
#pragma unroll
            for (int k = 0; k < 32; ++k) {
              const float partner = __shfl_xor_sync(0xffffffffu, v[k], 1);
              if (rope) v[k] = odd ? (v[k] * cs.x - partner * cs.y) : (v[k] * cs.x + partner * cs.y);
            }
          }
          uint32_t* dst = out + ((32 * hh + (odd ? 1 : 0)) * kDim + (d & ~1)) / 2;
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float recv = __shfl_xor_sync(0xffffffffu, odd ? v[k] : v[k + 1], 1);
            dst[k * (kDim / 2)] = odd ? pack_bf16(recv, v[k + 1]) : pack_bf16(v[k], recv);
          }
        }
      }
      ++seg;
      first = true;
      tc_fence_before();  // O^T has been read
      sy.sync();          // and red, alpha and the rope table are free for the next query
    } else {
      cur.next(p);
    }
  }
  if (ISSUE && warp == 0 && !live) mma.drain();
  if (!by_query && tid == 0) {
    p.joins[blockIdx.x] = make_int4(my_join.x, my_join.y, my_query, 0);
  }
}

// TMA: of bf16 rows (see produce_bf16)
template <int KVF, bool TMA>
__global__ void __launch_bounds__(Roles<KVF>::kThreads, 1) attend_paged_kernel(const __grid_constant__ PagedAttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base_s - raw_s);
  const uint32_t bars = base_s + SM_BAR;
  uint32_t* misc = reinterpret_cast<uint32_t*>(sm + SM_MISC);
  Run* run = reinterpret_cast<Run*>(sm + SM_RUN);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // in a uniform register

  pdl_trigger();
  // frequencies of the last producer warp's lanes (parameters come from memory
  // the first time, a line at a time)
  const double freq = warp == kFirstProducer + Roles<KVF>::kProducers - 1 && lane < p.a.rp.pairs ? p.a.rp.freq[lane] : 0.0;
  if (tid * 16 < p.a.n_query) prefetch_l2_line(p.a.q_pos + tid * 16);
  if (tid * 32 < p.a.n_query) prefetch_l2_line(p.a.seq_of_q + tid * 32);
  if (p.lo != nullptr && tid * 16 < p.kv.n_seq) prefetch_l2_line(p.lo + tid * 16);
  if (warp == 0) {
    tmem_alloc(base_s + SM_MISC + 8, kTmemCols);
    tmem_relinquish();
  }
  if (tid == kFirstProducer * 32) {
    constexpr uint32_t np = Roles<KVF>::kProducers;
    for (uint32_t b = 0; b < kBars; ++b)
      mbar_init(bars + 8 * b, b < kEmpty ? (TMA ? 1u : np) : (b == kQFull ? np + 1 : (b == kWeights ? (uint32_t)kAttWarps : 1u)));
    fence_mbar_init();
  }
  pdl_wait();
  // ---- this CTA's run of tiles: math thread x counts the tiles of its share
  // of the queries, a scan places the shares, and the thread whose share
  // holds the run's first tile finds its query
  const int Q = p.a.n_query;
  __shared__ int64_t warp_sum[kAttWarps];
  const int per = (Q + kAttThreads - 1) / kAttThreads;
  const int q_lo = min(Q, tid * per), q_hi = min(Q, q_lo + per);
  QuerySpan span;
  int64_t mine = 0, incl = 0;
  if (warp < kAttWarps) {
#pragma unroll 2  // (code before the first row is asked for comes from memory: unrolled by 4, 1 us more)
    for (int i = q_lo; i < q_hi; ++i) {
      span = query_span(p, i);
      mine += span.n_tiles;
    }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_sum[warp] = incl;
  }
  __syncthreads();
  if (warp < kAttWarps) {
    int64_t before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kAttWarps; ++w) {
      if (w < warp) before += warp_sum[w];
      total += warp_sum[w];
    }
    const int shift = dim_shift(total, (int)gridDim.x), c = (int)blockIdx.x >> shift;
    const RunCut cut = run_cut(total, Q, (int)gridDim.x);
    if (tid == 0) {
      run->total = total;
      run->index = c;
      run->m0 = ((int)blockIdx.x - (c << shift)) * (4 >> shift);
      run->m1 = run->m0 + (4 >> shift);
      run->cur.at = run->cur.run1 = total;  // unless found below
    }
    __shared__ int64_t ends[2];  // first tile of this run and of the next
    if (tid == 0) ends[0] = ends[1] = total;
    asm volatile("bar.sync 1, 256;" ::: "memory");
    // the thread whose share holds a cut finds the first tile from it on
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const int64_t y = min(c + e, cut.ctas) * cut.cost;
      if (y >= cut.ctas * cut.at(before, q_lo) && y < cut.ctas * cut.at(before + mine, q_hi)) {
        int64_t b = before;
        for (int i = q_lo;; ++i) {
          const int n = per > 1 ? query_span(p, i).n_tiles : span.n_tiles;
          if (y < cut.ctas * cut.at(b + n, i + 1)) {
            ends[e] = b + cut.tiles_before(y, b, i, n);
            break;
          }
          b += n;
        }
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    const int64_t run0 = ends[0], run1 = ends[1];
    if (run0 < run1 && run0 >= before && run0 < before + mine) {
      int i = q_lo;
      if (per > 1) {
        for (;; ++i) {
          span = query_span(p, i);
          if (run0 < before + span.n_tiles) break;
          before += span.n_tiles;
        }
      }
      run->cur.at = run0;
      run->cur.run1 = run1;
      run->cur.q0 = before;
      run->cur.qi = i;
      run->cur.span = span;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t taddr = (uint32_t)uniform((int)misc[2]);
  const uint32_t tmem_s = taddr, tmem_o = taddr + 64;
  Cursor cur = run->cur;
  if (uniform(cur.more())) {
    auto work = [&](auto split) {  // products, weights and outputs
      constexpr bool kSplit = decltype(split)::value;
      const Issuer<kSplit> mma{bars, tmem_s, tmem_o, base_s, elect_one(), p.a.flags,
                               TMA ? reinterpret_cast<const uint4*>(sm + SM_GONE) : nullptr, p.a.rp.pairs > 0,
                               (uint32_t)run->m0, (uint32_t)run->m1};
      if (Roles<KVF>::kOwnIssuer && warp == Roles<KVF>::kIssuer) issue_role(mma, cur, p);
      else math_role<!Roles<KVF>::kOwnIssuer>(p, sm, base_s, tmem_s, tmem_o, mma, cur, *run, warp);
    };
    if (warp >= kFirstProducer && !(Roles<KVF>::kOwnIssuer && warp == Roles<KVF>::kIssuer)) {
      const int t = tid - 32 * kFirstProducer;
      if constexpr (KVF == 0) produce_bf16<Roles<KVF>::kProducerThreads, TMA>(p, sm, base_s, cur, t, warp - kFirstProducer, freq);
      else produce_codes<KVF, Roles<KVF>::kProducerThreads>(p, sm, base_s, cur, t, warp - kFirstProducer, freq);
      cp_async_wait_all();  // no copy may still be landing when the CTA exits
    } else if (uniform(run->m1 - run->m0 == 4)) {
      work(std::false_type{});
    } else {
      work(std::true_type{});
    }
  }
  if (cur.at >= cur.run1 && Q >= (int)gridDim.x && tid == 0) p.joins[blockIdx.x] = make_int4(-1, -1, -1, 0);
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(taddr, kTmemCols);
}

// Join of a split query's partials. With M the largest reference of its parts
// and the sink, o = sum_g e^(m_g - M) O_g / (sum_g e^(m_g - M) l_g +
// e^(sink - M)), its rope channels rotated back. Latency-bound (128 KB a part,
// from L2): a warp takes four heads and 32 dims and needs no barrier; lanes
// (part, head) hold the weights of eight parts, which the lanes' dims take by
// shuffles, and the first eight parts are under way before their weights are
// known. GROUPS 1: four warps a CTA, next to each other in dims, each `spans`
// times 32 of them one after another (CTAs start at 0.6 a nanosecond: 9,728 of
// them took 17 us). GROUPS 8: the eight warps of a CTA share the dims and take
// every eighth batch of parts, for the few queries that have many.
constexpr int kJoinLanes = 8;  // parts whose weights a warp's lanes hold at once
constexpr int kJoinBatch = 4;  // parts whose values are under way at once
template <int GROUPS>
__global__ void __launch_bounds__(GROUPS == 1 ? 128 : 32 * GROUPS, GROUPS == 1 ? 8 : 4)
    attend_paged_join_kernel(const __grid_constant__ PagedAttendParams p, int spans) {
  constexpr int kWarps = GROUPS == 1 ? 4 : GROUPS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = GROUPS == 1 ? 0 : warp;
  // this warp's dims: `spans` times 32 from d on
  const int unit = GROUPS == 1 ? (int)blockIdx.y * kWarps + warp : (int)blockIdx.y, per_head = kDim / 32 / spans;
  const int hq = unit / per_head;
  int d = (unit % per_head) * 32 * spans + lane;
  // the frequency of this lane's rope channel, if its last span has one, and
  // the line of parameters it lies in, before the wait
  const int first_rope = kDim - 2 * p.a.rp.pairs, d_last = d + 32 * (spans - 1);
  const double freq = d_last >= first_rope ? p.a.rp.freq[(d_last - first_rope) >> 1] : 0.0;
  pdl_wait();
  const int4 jn = p.joins[blockIdx.x];
  if (jn.x < 0) return;
  const int qi = jn.z;
  const int n = jn.y - jn.x + 1;
  auto slot = [&](int k) { return (int64_t)(k == 0 ? part_slot(jn.x, true) : part_slot(jn.x + k, false)); };
  float4 v[kJoinBatch];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kJoinBatch; ++u)
      v[u] = k0 + u < n ? reinterpret_cast<const float4*>(p.a.part_o + slot(k0 + u) * kHeads * kDim)[part_at(hq, d)]
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  fetch(kJoinLanes * group);
  const int head = 4 * hq + (lane & 3), mine = lane >> 2;  // this lane's head, and its part of a batch
  // the first of the head's references and sums that this lane reads
  const float m0 = mine < n ? p.a.part_m[slot(mine) * kHeads + head] : -INFINITY;
  const float l0 = mine < n ? p.a.part_l[slot(mine) * kHeads + head] : 0.f;
  const double t = (double)p.a.q_pos[qi];
  const float sink = p.a.sink != nullptr ? p.a.sink[head] : -INFINITY;
  const float sk = sink * 1.4426950408889634f;  // references and scores are in log2 units
  // every warp forms the head's maximum and denominator over all parts
  float M = m0;
  for (int k = mine + kJoinLanes; k < n; k += kJoinLanes) M = fmaxf(M, p.a.part_m[slot(k) * kHeads + head]);
#pragma unroll
  for (int o = 16; o >= 4; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const bool none = M == -INFINITY;  // no row in any part
  M = fmaxf(M, sk);
  float den = (m0 == -INFINITY ? 0.f : exp2f(m0 - M)) * l0;  // 0 times NaN stays
  for (int k = mine + kJoinLanes; k < n; k += kJoinLanes) {
    const float m = p.a.part_m[slot(k) * kHeads + head];
    den += (m == -INFINITY ? 0.f : exp2f(m - M)) * p.a.part_l[slot(k) * kHeads + head];
  }
#pragma unroll
  for (int o = 16; o >= 4; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  den = none ? den + 1.f : den + exp2f(sk - M);
  const float inv = none ? 0.f : 1.f / den;
  if (d < 4 && group == 0 && p.a.lse != nullptr)  // lanes 0 .. 3 of the warp of dims 0 ..: a head each
    p.a.lse[(int64_t)qi * kHeads + head] = none && den == 1.f ? sink : (M + log2f(den)) * 0.6931471805599453f;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.a.out + ((int64_t)qi * kHeads + 4 * hq) * kDim);
  for (int span = 0; span < spans; ++span, d += 32) {
  if (span > 0) fetch(kJoinLanes * group);
  float o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k8 = kJoinLanes * group; k8 < n; k8 += kJoinLanes * GROUPS) {
    const float m = k8 == 0 ? m0 : (k8 + mine < n ? p.a.part_m[slot(k8 + mine) * kHeads + head] : -INFINITY);
    const float e = m == -INFINITY ? 0.f : exp2f(m - M);
#pragma unroll
    for (int k4 = 0; k4 < kJoinLanes; k4 += kJoinBatch) {
      if (k8 + k4 >= n) break;
      if (k4 > 0 || k8 > kJoinLanes * group) fetch(k8 + k4);
#pragma unroll
      for (int u = 0; u < kJoinBatch; ++u) {
        o[0] = fmaf(__shfl_sync(0xffffffffu, e, 4 * (k4 + u)), v[u].x, o[0]);
        o[1] = fmaf(__shfl_sync(0xffffffffu, e, 4 * (k4 + u) + 1), v[u].y, o[1]);
        o[2] = fmaf(__shfl_sync(0xffffffffu, e, 4 * (k4 + u) + 2), v[u].z, o[2]);
        o[3] = fmaf(__shfl_sync(0xffffffffu, e, 4 * (k4 + u) + 3), v[u].w, o[3]);
      }
    }
  }
  if constexpr (GROUPS > 1) {
    __shared__ float4 acc[kWarps - 1][32];
    if (warp > 0) acc[warp - 1][lane] = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int k = 0; k < kWarps - 1; ++k) {
      const float4 a = acc[k][lane];
      o[0] += a.x;
      o[1] += a.y;
      o[2] += a.z;
      o[3] += a.w;
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) o[u] *= __shfl_sync(0xffffffffu, inv, u);  // lane u holds head u's
  if ((d | 31) >= first_rope) {  // whole warps: a warp's dims are 32 in a row
    float cs = 1.f, sn = 0.f;
    if (d >= first_rope) angle_cs(t * (d == d_last ? freq : p.a.rp.freq[(d - first_rope) >> 1]), cs, sn);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float partner = __shfl_xor_sync(0xffffffffu, o[u], 1);
      o[u] = (d & 1) ? o[u] * cs - partner * sn : o[u] * cs + partner * sn;
    }
  }
  // even lanes store heads 0 and 1, odd lanes heads 2 and 3, two dims a store
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const float give = (d & 1) ? o[u] : o[2 + u], keep = (d & 1) ? o[2 + u] : o[u];
    const float got = __shfl_xor_sync(0xffffffffu, give, 1);
    const int h = (d & 1) ? 2 + u : u;
    out[(h * kDim + (d & ~1)) >> 1] = (d & 1) ? pack_bf16(got, keep) : pack_bf16(keep, got);
  }
  }
}

namespace {
constexpr size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
// Tensor map of bf16 rows, boxes of 64 channels (128 bytes, the swizzle's width).
cudaError_t encode_bf16_map(CUtensorMap* map, int rank, const void* base, const uint64_t* dims, const uint64_t* strides,
                            const uint32_t* box) {
  // looked up by the first call; host threads with contexts of their own may make it at once
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> looked_up{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 encode = looked_up.load(std::memory_order_acquire);
  if (encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    looked_up.store(encode, std::memory_order_release);
  }
  const uint32_t ones[3] = {1u, 1u, 1u};
  cuuint64_t d[3], st[2];
  cuuint32_t bx[3], es[3];
  for (int i = 0; i < rank; ++i) {
    d[i] = dims[i];
    bx[i] = box[i];
    es[i] = ones[i];
    if (i + 1 < rank) st[i] = strides[i];
  }
  auto fill = [&] {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), d, st, bx, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = fill();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // a host thread's first CUDA call: the device's context is made the
    // thread's, as a launch would do
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    r = fill();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// Every CTA sums the tile counts of all queries before it starts: 16 a thread
// at this many. More queries go in launches of this many, one after another.
constexpr int kMaxQueries = 4096;
}  // namespace

int attend_paged_ctas(int num_sms) { return num_sms < kMaxCtas ? num_sms : kMaxCtas; }

size_t attend_paged_workspace_bytes(int num_sms) {
  const size_t slots = 2 * (size_t)attend_paged_ctas(num_sms);
  return al256(slots * kHeads * kDim * 4) + 2 * al256(slots * kHeads * 4) + al256(slots * 16);
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
  p.joins = reinterpret_cast<int4*>(w);
  const int Q = a.n_query;
  const int chunk = 1 << chunk_shift(kv.page_shift);
  const uint64_t kv_dims[3] = {(uint64_t)kDim, 1ull << kv.page_shift, (uint64_t)kv.n_pages};
  const uint64_t kv_strides[2] = {2u * kDim, (uint64_t)kv.page_stride};
  const uint32_t kv_box[3] = {64u, (uint32_t)chunk, 1u};
  for (int q0 = 0; q0 < Q; q0 += kMaxQueries) {
    const int nq = Q - q0 < kMaxQueries ? Q - q0 : kMaxQueries;
    p.a.n_query = nq;
    p.a.q = a.q + (int64_t)q0 * kHeads * kDim;
    p.a.q_pos = a.q_pos + q0;
    p.a.seq_of_q = a.seq_of_q + q0;
    p.a.out = a.out + (int64_t)q0 * kHeads * kDim;
    p.a.lse = a.lse != nullptr ? a.lse + (int64_t)q0 * kHeads : nullptr;
    const uint64_t q_dims[2] = {(uint64_t)kDim, (uint64_t)kHeads * nq}, q_strides[1] = {2u * kDim};
    const uint32_t q_box[2] = {64u, (uint32_t)kHeads};
    cudaError_t e = encode_bf16_map(&p.q_map, 2, p.a.q, q_dims, q_strides, q_box);
    if (e == cudaSuccess && kv_fmt == 0) e = encode_bf16_map(&p.kv_map, 3, kv.pages, kv_dims, kv_strides, kv_box);
    if (e != cudaSuccess) return e;
#define CSA2_PAGED(F, T)                                                                                               \
  do {                                                                                                                \
    e = cudaFuncSetAttribute(attend_paged_kernel<F, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kPagedSmemBytes); \
    if (e == cudaSuccess)                                                                                             \
      e = launch_ex(attend_paged_kernel<F, T>, dim3(G), dim3(Roles<F>::kThreads), kPagedSmemBytes, st, true, 0, p);  \
  } while (0)
    if (kv_fmt == 0 && chunk >= 8) CSA2_PAGED(0, true);
    else if (kv_fmt == 0) CSA2_PAGED(0, false);
    else if (kv_fmt == 1) CSA2_PAGED(1, false);
    else CSA2_PAGED(2, false);
#undef CSA2_PAGED
    if (e != cudaSuccess) return e;
    *n_launch += 1;
    const int joins = nq < G ? nq : G;
    // A query has more than two batches of parts only where there are few
    // queries. Otherwise spans of 32 dims a warp until the CTAs are resident at once
    // (32 warps an SM): fewer CTAs to start, the same loads under way.
    if (joins * 2 * kJoinLanes <= G) {
      e = launch_ex(attend_paged_join_kernel<8>, dim3((unsigned)joins, kHeads / 4 * (kDim / 32)), dim3(256), 0, st, true, 0, p, 1);
    } else {
      int spans = 1;
      while (spans < kDim / 32 && joins * (kHeads / 4) * (kDim / 32) / spans > 32 * num_sms) spans *= 2;
      e = launch_ex(attend_paged_join_kernel<1>, dim3((unsigned)joins, kHeads / 4 * (kDim / 32) / 4 / spans), dim3(128), 0, st, true, 0, p, spans);
    }
    if (e != cudaSuccess) return e;
    *n_launch += 1;
  }
  return cudaGetLastError();
}

}  // namespace csa2

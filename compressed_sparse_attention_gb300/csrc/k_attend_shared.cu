// csa2_attend_shared: attention of a batch whose queries share rows.
//
// Places k = 0 .. n_query - 1 hold the queries group by group (order), head[k]
// is the first place of k's group and shared[head[k]] the number of leading
// positions whose rows the group shares: position p < shared is read through
// the table row of the group's first query, any other through the query's own.
// Query i at t = q_pos[i] sees every p <= t; formula as for csa2_attend_paged.
//
// A row serves the 64 heads of one query with 128 operations a byte, fewer
// than the GPU has for a byte from memory (284) and, from the L2, with two
// products of 128 x 64 x 16 that take 48 cycles each where the operations take
// 32 (shared memory delivers 128 bytes a clock). Two queries that share it make it
// a matrix product. So two neighbouring places of a group are one unit of work,
// given to a pair of CTAs (a cluster of two, on two SMs that work on one
// tcgen05 product): CTA r has query r, its 64 heads being its rows of both
// products, M = 128 over the pair:
//   S [64 heads x 256 rows]  = Q [64 x 512] KV^T          N = 256, K = 512
//   O [64 heads x 512 dims] += P [64 x 256] KV            N = 256 twice, K = 256
// Of the second operand each CTA brings half of N: of a tile's 256 rows, 128
// whole ones for S, and all 256 in half of their dims for O. Both halves
// stream through one ring of 16 KB slots in the order in which the products
// use them. Tensor memory holds O (256 columns) and two S (128 each), so that
// the next tile's scores come while this one's weights are formed.
//
// Tile: 256 rows of the unit's list, which are groups of 64 aligned positions:
// those that both queries see, then those that only the first sees, then the
// second's. Products of a group that one query does not see leave that query's
// CTA's lanes of O alone (disable-output-lane), so that a NaN in a row reaches
// only the queries that see it.
//
// What bounds it. A tile's products run 4,352 cycles at best (36 of N = 256 and
// K = 16 for S, rope residual included, 32 for O, 64 cycles each; all operations
// would take 4,096). Tiles take 2.7 us in a unit of many, some 5,250 cycles: 64
// queries over 32K common bf16 rows 166 to 170 us, 1.67 PFLOP/s, where
// csa2_attend_paged takes 332; run for seconds 187, 1.48 PFLOP/s, as the card's
// power limit then holds the clock at 1.63 GHz instead of 2.07 (csa2_attend_paged
// stays below it). The ring's seven slots are 1,900 cycles of products and just cover a
// copy's 1,100 to 1,500 and the barriers around it (without copies and weights a
// tile takes 4,700): what was between the products at first (copies looked up behind the wait for
// a slot, arrivals with a cluster-wide release, a barrier not looked at ahead: 9,800
// cycles a tile) is off that path. fp8 and fp4 rows: their conversion, 14,000
// cycles a tile: the pair converts every element twice, as a key and as a value,
// and for one query as for two; a query alone in its unit takes half as
// long again as with csa2_attend_paged, in bf16 a tenth. Short calls: plan 2.2
// us, Q 2, a tile's scores, first weights and products 4.5, partial 2 (128 KB a
// CTA, 32 bytes a clock), join 5: four queries over 2K rows 18.1 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <type_traits>

#include "launchers.cuh"
#include "tile_pipe.cuh"

namespace csa2 {

namespace {

constexpr int kGroupRows = 64;   // aligned positions of a row group
constexpr int kTileGroups = 4;   // row groups of a tile
constexpr int kRing = 7;         // slots
constexpr uint32_t kSlotBytes = 16384;
constexpr int kMaxCtaPairs = 80;   // pairs of CTAs, at most
constexpr int kPlanThreads = 1024;

// Two places of a group (or its last one alone), one of which has a query.
struct alignas(16) SharedUnit {
  int32_t q[2];       // the queries; -1: none
  int32_t seq[2];     // their sequences
  int32_t end[2];     // one past the last position that each sees, inside the table; 0: sees nothing
  int32_t head_seq;   // positions below len are read through its table row
  int32_t len;
  int32_t common;     // positions below it are seen by both (or by the only one that sees any)
  int32_t n[3];       // row groups: common, the first query's own, the second's
  int32_t tiles;
  int32_t pad[3];
  int64_t t[2];       // the queries' positions
};
static_assert(sizeof(SharedUnit) == 80, "SharedUnit");

struct alignas(16) SharedRun {
  int64_t tile;    // number of its first tile among all
  int32_t unit;    // its unit
  int32_t first;   // number of that tile in its unit
};
// What a pair of CTAs starts from: its run, the number of its tiles and its
// first unit, in one place (each step through memory is 0.6 us of a short call).
struct alignas(16) SharedStart {
  int64_t tiles;
  int32_t unit, first;
  SharedUnit u;
};

struct SharedParams {
  CUtensorMap q_map;   // Q: [64 n_query heads][512], boxes of 64 heads x 64 channels
  CUtensorMap kv_map;  // bf16 pages: [n_pages][page_size][512], boxes of one piece x 64 channels
  CUtensorMap v_map;   // the same as [n_pages][8 blocks][page_size][64], boxes of two blocks of 64 rows (pages of 64 rows and more)
  CUtensorMap code_map;  // fp8, fp4 codes: [n_pages][page_size][row bytes], boxes of one piece x 64 channels
  const uint16_t* q;
  const int64_t* q_pos;
  const int32_t* seq_of_q;
  const int32_t* order;
  const int32_t* head;
  const int64_t* shared;
  const float* sink;
  uint16_t* out;
  float* lse;
  uint32_t* flags;
  PagedView kv;
  RopeParams rp;
  float scale_log2;
  int n_query;
  int pairs;  // of CTAs
  int planned;  // whether a launch of its own has made the plan (units, starts, joins)
  SharedUnit* units;
  SharedStart* starts;  // [pairs]
  int4* joins;       // [min(n_query, pairs)]: of a split unit its queries, first and last run; third -1: none. The index is
                     // the unit, or with as many queries as pairs or more the run that begins it and does not end it
  float* part_o;     // [2 pairs slots][2][512 / 4][64 heads][4]
  float2* part_ml;   // [2 pairs slots][2][64]: reference and sum
};

// Slots of the partials: run c leaves at most two, as in csa2_attend_paged.
__device__ __forceinline__ int64_t shared_slot(int c, bool begins, int rank) { return 2 * (2 * (int64_t)c + (begins ? 1 : 0)) + rank; }

// rows of a piece: what one copy takes of a page
__host__ __device__ __forceinline__ int piece_shift(int page_shift) { return page_shift < 6 ? page_shift : 6; }

}  // namespace

// ---------------------------------------------------------------------------
// The plan: places -> units, and the units' tiles cut into runs of equal cost, one
// a pair of CTAs. Of up to kPlanHere places every pair of CTAs makes it for itself,
// a thread a place (three round trips to the L2); of more, one CTA in a launch of
// its own, a thread a share of the places (a launch, and what it costs to hand
// the plan over, 3 us of a call).
//
// On a line where a tile is kTilePlace long and a unit starts with kUnitPlace, run
// c has the tiles that start in the c-th of R equal parts (a part inside a unit's
// start has none).
// ---------------------------------------------------------------------------
constexpr int kTilePlace = 4, kUnitPlace = 8;  // a unit: its Q, its first weights, its outputs
constexpr int kPlanHere = 96;                 // units that fit shared memory beside the tiles
struct RunLine {
  int64_t cost;
  int runs, start;
  __device__ __forceinline__ RunLine(int64_t tiles, int units, int pairs) {
    start = tiles > 2 * (int64_t)pairs ? kUnitPlace : 0;
    cost = kTilePlace * tiles + (int64_t)start * units;
    runs = (int)min((int64_t)pairs, tiles);
  }
  // where unit u begins, t tiles coming before it, runs-fold
  __device__ __forceinline__ int64_t at(int64_t t, int u) const { return runs * (kTilePlace * t + (int64_t)start * u); }
  // of unit u the first tile from cut c on
  __device__ __forceinline__ int64_t tile_from(int c, int64_t t, int u) const {
    const int64_t left = c * cost - at(t, u + 1), step = (int64_t)kTilePlace * runs;
    return left <= 0 ? 0 : quotient(left + step - 1, step);
  }
  // run of tile j of unit u
  __device__ __forceinline__ int run_of(int64_t t, int u, int j) const {
    return (int)quotient(at(t, u + 1) + (int64_t)kTilePlace * runs * j, cost);
  }
};

namespace {
struct PlanUnit {
  SharedUnit u;
  bool begins;
};
// A place as the plan sees it: its head, the next place's (kNoPlace behind the
// last) and the first place of the run of equal heads that it lies in, which is
// where its group begins.
constexpr int32_t kNoPlace = INT32_MIN;
struct PlanPlace {
  int32_t head, next, run;
};
// The unit that place k begins, if it does. bad: flags to record.
__device__ __forceinline__ PlanUnit unit_at(const SharedParams& p, int k, const PlanPlace& at, uint32_t& bad) {
  PlanUnit r;
  const int n = p.n_query, h = at.head;
  r.begins = false;
  if (h != at.run) {  // its group does not begin where its head says
    bad |= CSA2_FLAG_BAD_QUERY;
    return r;
  }
  r.begins = ((k - h) & 1) == 0;
  if (!r.begins) return r;
  const int32_t cap = p.kv.max_pages << p.kv.page_shift;  // at most 2^30
  SharedUnit& u = r.u;
  int64_t len = p.shared[h];
  auto query = [&](int place) {
    const int q = p.order[place];
    if (q < -1 || q >= n) bad |= CSA2_FLAG_BAD_QUERY;
    return q >= 0 && q < n ? q : -1;
  };
  const int qh = query(h);
  u.q[0] = query(k);
  u.q[1] = at.next == h ? query(k + 1) : -1;
  u.head_seq = qh >= 0 ? p.seq_of_q[qh] : -1;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    u.seq[x] = -1;
    u.end[x] = 0;
    u.t[x] = 0;
    if (u.q[x] < 0) continue;
    const int b = p.seq_of_q[u.q[x]];
    const int64_t t = p.q_pos[u.q[x]];
    u.t[x] = t;
    if (b == -1) {
      u.q[x] = -1;  // a padding query
      continue;
    }
    if (b < 0 || b >= p.kv.n_seq || t < -1) {
      bad |= CSA2_FLAG_BAD_QUERY;
      continue;
    }
    u.seq[x] = b;
    if (t >= cap) bad |= CSA2_FLAG_BAD_PAGE;
    u.end[x] = (int32_t)(t >= cap ? cap : t + 1);
  }
  if (u.q[0] < 0 && u.q[1] < 0) {  // nothing to write: padding takes no tile
    r.begins = false;
    return r;
  }
  if (u.head_seq < 0 || u.head_seq >= p.kv.n_seq) len = 0;
  len = len < 0 ? 0 : (len > cap ? cap : len);
  u.len = (int32_t)len & ~((1 << p.kv.page_shift) - 1);  // sequences share whole pages
  const bool a = u.end[0] > 0, b = u.end[1] > 0;
  u.n[1] = u.n[2] = 0;
  if (a && b) {
    u.common = min(u.end[0], u.end[1]);
    if (u.seq[0] != u.seq[1]) u.common = min(u.common, u.len);
    const int f = u.common >> 6;
    u.n[1] = u.end[0] > u.common ? ((u.end[0] + 63) >> 6) - f : 0;
    u.n[2] = u.end[1] > u.common ? ((u.end[1] + 63) >> 6) - f : 0;
  } else {
    u.common = max(u.end[0], u.end[1]);
  }
  u.n[0] = (u.common + 63) >> 6;
  u.tiles = max(1, (u.n[0] + u.n[1] + u.n[2] + kTileGroups - 1) / kTileGroups);
  u.pad[0] = u.pad[1] = u.pad[2] = 0;
  return r;
}
}  // namespace

__global__ void __launch_bounds__(kPlanThreads, 1) attend_shared_plan_kernel(const __grid_constant__ SharedParams p) {
  __shared__ int64_t sum_t[32], share_t[kPlanThreads];  // tiles, units before a thread's share
  __shared__ int sum_u[32], share_u[kPlanThreads];
  __shared__ int last_run[32];
  __shared__ SharedRun runs[kMaxCtaPairs + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const int per = (p.n_query + kPlanThreads - 1) / kPlanThreads;
  const int lo = min(p.n_query, tid * per), hi = min(p.n_query, lo + per);
  // where the run of equal heads begins that goes on into the share
  int run = -1;
  for (int k = lo; k < hi; ++k) {
    if (k == 0 || p.head[k] != p.head[k - 1]) run = k;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) run = max(run, __shfl_up_sync(0xffffffffu, run, o));
  if (lane == 31) last_run[warp] = run;
  __syncthreads();
  run = __shfl_up_sync(0xffffffffu, run, 1);
  if (lane == 0) run = -1;
  for (int w = 0; w < warp; ++w) run = max(run, last_run[w]);
  // the units of the share in turn
  auto each_unit = [&](uint32_t& bad, auto&& take) {
    PlanPlace at{kNoPlace, lo < hi ? p.head[lo] : kNoPlace, run};
    int32_t before = lo > 0 && lo < hi ? p.head[lo - 1] : kNoPlace;
    for (int k = lo; k < hi; ++k) {
      at.head = at.next;
      at.next = k + 1 < p.n_query ? p.head[k + 1] : kNoPlace;
      if (k == 0 || at.head != before) at.run = k;
      before = at.head;
      const PlanUnit one = unit_at(p, k, at, bad);
      if (one.begins) take(one.u);
    }
  };
  int64_t tiles = 0;
  int units = 0;
  uint32_t bad = 0, unused = 0;
  SharedUnit only;  // of a share of one place
  each_unit(bad, [&](const SharedUnit& u) {
    tiles += u.tiles;
    ++units;
    only = u;
  });
  if (bad) set_flag(p.flags, bad);
  // exclusive scan over the threads
  int64_t it = tiles;
  int iu = units;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xffffffffu, it, o);
    const int b = __shfl_up_sync(0xffffffffu, iu, o);
    if (lane >= o) it += a, iu += b;
  }
  if (lane == 31) sum_t[warp] = it, sum_u[warp] = iu;
  __syncthreads();
  // (every warp scans the warps' sums for itself)
  int64_t at = sum_t[lane];
  int au = sum_u[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, at, o);
    const int y = __shfl_up_sync(0xffffffffu, au, o);
    if (lane >= o) at += x, au += y;
  }
  const int64_t T = __shfl_sync(0xffffffffu, at, 31);
  const int U = __shfl_sync(0xffffffffu, au, 31);
  const int64_t bt = __shfl_sync(0xffffffffu, at, max(warp, 1) - 1);
  const int bu = __shfl_sync(0xffffffffu, au, max(warp, 1) - 1);
  share_t[tid] = it - tiles + (warp > 0 ? bt : 0);
  share_u[tid] = iu - units + (warp > 0 ? bu : 0);
  int u0 = share_u[tid];
  if (per > 1) each_unit(unused, [&](const SharedUnit& u) { p.units[u0++] = u; });
  else if (units > 0) p.units[u0] = only;
  __syncthreads();
  const RunLine line(T, U, p.pairs);
  // thread c finds the first tile from the c-th cut on
  if (tid <= p.pairs) {
    SharedRun r{T, U, 0};
    if (tid < line.runs) {
      const int64_t y = tid * line.cost;
      int i = 0, end = kPlanThreads;  // the last share that begins at or before y
      while (end - i > 1) {
        const int mid = (i + end) >> 1;
        if (line.at(share_t[mid], share_u[mid]) <= y) i = mid;
        else end = mid;
      }
      int64_t t = share_t[i];
      for (int u = share_u[i]; u < U; ++u) {
        const int n = p.units[u].tiles;
        const int64_t j = line.tile_from(tid, t, u);
        if (j < n) {
          r = SharedRun{t + j, u, (int32_t)j};
          break;
        }
        t += n;
      }
    }
    runs[tid] = r;
  }
  __syncthreads();
  if (tid < p.pairs) {
    int4 jn = make_int4(-1, -1, -1, 0);
    // a unit that begins in run c and goes on
    const SharedRun next = runs[tid + 1];
    if (next.first > 0 && (runs[tid].unit < next.unit || runs[tid].first == 0)) {
      const SharedUnit& u = p.units[next.unit];
      jn = make_int4(u.q[0], u.q[1], tid, line.run_of(next.tile - next.first, next.unit, u.tiles - 1));
    }
    p.joins[tid] = jn;
  }
  // (four starts a warp)
  const int first_c = warp * 4;
  for (int c = first_c; c < min(p.pairs, first_c + 4); ++c) {
    const SharedRun r = runs[c];
    const int64_t n = runs[c + 1].tile - r.tile;
    int4* dst = reinterpret_cast<int4*>(p.starts + c);
    if (lane == 0) dst[0] = make_int4((int)(uint32_t)n, (int)(n >> 32), r.unit, r.first);
    if (lane < 5 && n > 0) dst[1 + lane] = reinterpret_cast<const int4*>(p.units + r.unit)[lane];
  }
}

// ---------------------------------------------------------------------------
// The tile kernel. Roles of a CTA's warps:
//   0 .. 7   math: softmax, outputs
//   8 ..     producers: a slot of the ring each in turn
//   then 1 or 2  Q, its rope channels rotated
//   last     issues the pair's products (in CTA 0 of the pair)
// Waits are bounded; barriers that the issuer waits for lie in CTA 0, to which
// CTA 1 arrives over the cluster, and the issuer's commits arrive in both.
// ---------------------------------------------------------------------------
namespace {

constexpr int kMathWarps = 8;
// 15 or 16 warps: four on a scheduler, each with up to 128 registers (with a
// seventeenth they would have 96, and the conversion of fp8 rows spill 900 bytes).
// A warp's slots come kProducers apart, no more than the ring's: its next
// slot but one of the ring must come after slots that it has waited for, or its
// wait could take the parity of the use before the last.
template <bool TMA>
struct SharedRoles {
  static constexpr int kProducers = TMA ? 4 : 6;  // threads copy, or convert, with more warps
  static constexpr int kQWarps = TMA ? 2 : 1;
  static constexpr int kQ = kMathWarps + kProducers;
  static constexpr int kIssuer = kQ + kQWarps;
  static constexpr int kThreads = 32 * (kIssuer + 1);
  static_assert(kProducers <= kRing && kThreads <= 512);
};

constexpr uint32_t S_Q = 0;                           // [9 blocks][64 heads][128 B]; block 8: rope residual
constexpr uint32_t S_P = S_Q + 9 * 8192;              // [4 row groups][64 heads][128 B]
constexpr uint32_t S_RING = S_P + 4 * 8192;           // [kRing][16 KB]
constexpr uint32_t S_BAR = S_RING + kRing * kSlotBytes;
constexpr uint32_t S_RED = S_BAR + 256;               // float [4 row groups][64 heads]
constexpr uint32_t S_ROPE = S_RED + 1024;             // float2 [2 halves of the heads][32]
constexpr uint32_t S_QROPE = S_ROPE + 512;            // float2 [32]
constexpr uint32_t S_MISC = S_QROPE + 256;
constexpr uint32_t S_UNITS = S_MISC + 64;              // SharedUnit [kPlanHere]
constexpr uint32_t S_SUMS = S_UNITS + kPlanHere * (uint32_t)sizeof(SharedUnit);  // int64 [4], int [4], SharedRun [2]
constexpr uint32_t kSharedSmemBytes = S_SUMS + 96 + 1024;
static_assert(kSharedSmemBytes <= 232448, "shared memory");

enum SBar : uint32_t { bFull = 0, bEmpty = 7, bQFull = 14, bQEmpty = 15, bScores = 16, bWeights = 18, bPFree = 19, bOFree = 20, bDrained = 21, bEdge = 22, kSBars = 28 };

constexpr uint32_t kIdescS = idesc_bf16(128, 256, 0, 0);
constexpr uint32_t kIdescO = idesc_bf16(128, 256, 0, 1);

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the address of the same place in CTA 0 of the pair
__device__ __forceinline__ uint32_t in_leader(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
// An arrival in CTA 0 for what this CTA's warps left in their own shared memory
// (made visible to the tensor core by a proxy fence before) or read from their
// own tensor memory, for products that CTA 0 issues. What has to be released at
// the scope of the pair is shared memory alone, and a fence for no more than that
// costs little (fp8 136.5 -> 137.9 us, bf16 as without it): an arrival that
// releases at cluster scope itself waits for all of the warp's accesses to global
// memory too, 1,500 cycles (64 x 32K 169 -> 185 us, fp8 152).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile(
      "fence.release.sync_restrict::shared::cta.cluster;\n"
      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void warp_arrive_cluster(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive_cluster(bar);
}
// (relaxed: there is nothing before it to be seen behind it, and a release waits
// for the warp's loads and stores, some 1,000 cycles)
__device__ __forceinline__ void expect_cluster_one(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %2, 0;\n@e mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;\n}" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}
// wait_phase for arrivals from the other CTA too: its warps', its copies', and the
// issuer's commits, which arrive in both. The acquiring side of the above.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t phase, uint32_t* flags) {
#pragma unroll 1
  for (int i = 0; i < 100000; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.relaxed.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
        "selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(phase), "r"(20000u)
        : "memory");
    if (ok != 0u) {
      asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
      return true;
    }
  }
  set_flag(flags, CSA2_FLAG_WAIT_TIMEOUT);
  return false;
}
__device__ __forceinline__ uint32_t done_cluster(uint32_t bar, uint32_t phase) {
  uint32_t ok;
  asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok)
               : "r"(bar), "r"(phase)
               : "memory");
  return ok;
}
__device__ __forceinline__ bool wait_cluster_all_lanes(uint32_t bar, uint32_t phase, uint32_t* flags) {
  return __all_sync(0xffffffffu, wait_cluster(bar, phase, flags)) != 0;
}
// by a warp's first lane
__device__ __forceinline__ bool warp_wait_cluster(uint32_t bar, uint32_t phase, uint32_t* flags) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_cluster(bar, phase, flags);
  return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
}
// copies into this CTA whose bytes are counted by a barrier of CTA 0
__device__ __forceinline__ void tma_pair_2d(uint32_t leader, uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %5, 0;\n"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];\n}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_pair_3d(uint32_t leader, uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                            uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %6, 0;\n"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4}], [%5];\n}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_pair_4d(uint32_t leader, uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\nsetp.ne.u32 e, %7, 0;\n"
      "@e cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, %4, %5}], [%6];\n}" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 e, %5, 0;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader)
      : "memory");
}
// off0, off1: all ones leave CTA 0's, CTA 1's lanes of D as they are
__device__ __forceinline__ void mma_pair_lanes(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc,
                                               uint32_t off0, uint32_t off1) {
  asm volatile(
      "{\n.reg .pred p, e;\nsetp.ne.u32 p, %4, 0;\nsetp.ne.u32 e, %5, 0;\n"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, {%6, %6, %6, %6, %7, %7, %7, %7}, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader), "r"(off0), "r"(off1)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n.reg .pred e;\n.reg .b16 m;\nmov.b16 m, 3;\nsetp.ne.u32 e, %1, 0;\n"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n}" ::"r"(bar), "r"(leader)
      : "memory");
}

// Where a row group of a unit's list lies: 64 positions from 64 * block on, of
// which [from, to) are its own; who: 0 both queries see them, 1 the first
// alone, 2 the second alone; seq: the sequence of positions at or past len.
struct RowGroup {
  bool present;
  int who, block, from, to, seq;
};
__device__ __forceinline__ RowGroup row_group(const SharedUnit& u, int j) {
  RowGroup g;
  g.present = j < u.n[0] + u.n[1] + u.n[2];
  const int f = u.common >> 6;
  if (j < u.n[0]) {
    g.who = 0;
    g.block = j;
    g.from = 0;
    g.to = u.common;
    g.seq = u.end[0] > 0 ? u.seq[0] : u.seq[1];
  } else if (j < u.n[0] + u.n[1]) {
    g.who = 1;
    g.block = f + j - u.n[0];
    g.from = u.common;
    g.to = u.end[0];
    g.seq = u.seq[0];
  } else {
    g.who = 2;
    g.block = f + j - u.n[0] - u.n[1];
    g.from = u.common;
    g.to = u.end[1];
    g.seq = u.seq[1];
  }
  return g;
}
__device__ __forceinline__ int row_groups(const SharedUnit& u, int tile) {
  return min(kTileGroups, u.n[0] + u.n[1] + u.n[2] - kTileGroups * tile);
}
// page of position p of a group (-1: none)
__device__ __forceinline__ int32_t group_page(const SharedParams& p, const SharedUnit& u, const RowGroup& g, int pos) {
  return g.present && pos >= g.from && pos < g.to ? page_of(p.kv, pos < u.len ? u.head_seq : g.seq, pos) : -1;
}

// (field by field: a struct filled through a cast lives in local memory)
__device__ __forceinline__ SharedUnit load_unit(const SharedUnit* at) {
  const int4* v = reinterpret_cast<const int4*>(at);
  const int4 a = v[0], b = v[1], c = v[2];
  SharedUnit u;
  u.q[0] = a.x;
  u.q[1] = a.y;
  u.seq[0] = a.z;
  u.seq[1] = a.w;
  u.end[0] = b.x;
  u.end[1] = b.y;
  u.head_seq = b.z;
  u.len = b.w;
  u.common = c.x;
  u.n[0] = c.y;
  u.n[1] = c.z;
  u.n[2] = c.w;
  u.tiles = v[3].x;
  const int4 t = v[4];
  u.t[0] = (int64_t)(uint32_t)t.x | (int64_t)t.y << 32;
  u.t[1] = (int64_t)(uint32_t)t.z | (int64_t)t.w << 32;
  return u;
}

// A pair's run: its units, and of each the tiles [first, last).
struct SharedWalk {
  int64_t left;  // tiles of the run that are left, this unit's included
  int unit, first, last;
  bool begins, ends;
  const SharedUnit* units;
  SharedUnit u;
  // from the plan in memory
  __device__ __forceinline__ void start(const SharedUnit* all, const SharedStart* at) {
    units = all;
    const int4 a = *reinterpret_cast<const int4*>(at);
    left = (int64_t)(uint32_t)a.x | (int64_t)a.y << 32;
    unit = uniform(a.z);
    first = uniform(a.w);
    if (left > 0) load(&at->u);
  }
  // from the CTA's own
  __device__ __forceinline__ void start(const SharedUnit* all, const SharedRun& r, int64_t tiles) {
    units = all;
    left = tiles;
    unit = uniform(r.unit);
    first = uniform(r.first);
    if (left > 0) load(units + unit);
  }
  __device__ __forceinline__ void load(const SharedUnit* at) {
    u = load_unit(at);
    begins = uniform(first == 0);
    last = uniform((int)min((int64_t)u.tiles, first + left));
    ends = uniform(last == u.tiles);
  }
  __device__ __forceinline__ bool next() {
    left -= last - first;
    ++unit;
    first = 0;
    if (left > 0) load(units + unit);
    return left > 0;
  }
};

// place in the ring
struct RingAt {
  uint32_t slot, phase;
  __device__ __forceinline__ void step(uint32_t n) {  // n <= 2 kRing - slot
    slot += n;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (slot >= (uint32_t)kRing) {
        slot -= kRing;
        phase ^= 1u;
      }
    }
  }
};

// The ring behind its last slot, `filled` of them before: the products' arrivals
// for all of them. Nothing is filled after these, but an arrival from the other CTA
// must find this one's shared memory still its own.
__device__ __forceinline__ void drain_ring(const SharedParams& p, uint32_t bars, const RingAt& end, uint32_t filled, bool live) {
#pragma unroll 1
  for (uint32_t i = 0; i < (uint32_t)kRing && live; ++i) {
    RingAt at = end;
    at.step(i);
    if (filled + i >= (uint32_t)kRing) live = wait_cluster_all_lanes(bars + 8 * (bEmpty + at.slot), at.phase ^ 1u, p.flags);
  }
}

// A slot's rows by the warp itself: pages of less than the eight rows of a copy's
// swizzle atom, row by row. K: channels 64 b .. of the 128 rows of the
// tile's groups 2 rank and 2 rank + 1; V: dims d0 .. d0 + 127 of group g's 64
// rows. Rows that are not the group's become zeros (in V: their weights are 0,
// but 0 times a NaN is not).
template <int KVF, bool IS_K>
__device__ __forceinline__ void fill_slot(const SharedParams& p, const SharedUnit& u, int tile, int g0, int d0, uint32_t dst_s,
                                          uint8_t* dst, int lane) {
  constexpr int kRows = IS_K ? 128 : 64;
  const int page_mask = (1 << p.kv.page_shift) - 1;
  if constexpr (KVF == 0) {
    constexpr int kChunks = IS_K ? 8 : 16;  // of 16 bytes, of a row
    const int c = lane % kChunks;
#pragma unroll 8
    for (int r = lane / kChunks; r < kRows; r += 32 / kChunks) {
      const RowGroup g = row_group(u, kTileGroups * tile + g0 + (r >> 6));
      const int pos = 64 * g.block + (r & 63);
      const int32_t page = group_page(p, u, g, pos);
      const uint8_t* src = page >= 0 ? p.kv.pages + page * p.kv.page_stride + (int64_t)(pos & page_mask) * 1024 + 2 * d0 + 16 * c
                                     : p.kv.pages;
      cp_async16(dst_s + (uint32_t)(c >> 3) * 8192u + (uint32_t)r * 128u + ((uint32_t)((c & 7) ^ (r & 7)) << 4), src, page >= 0 ? 16u : 0u);
    }
    cp_async_wait_all();
  } else {
    constexpr int kRowBytes = KVF == 1 ? 512 : 256, kScaleBytes = KVF == 1 ? 16 : 32;
    constexpr int kChunks = IS_K ? 4 : 8;  // of 16 channels, of a row
    constexpr int kBatch = 4;              // rows of a thread under way at once
    using Code = typename std::conditional<KVF == 1, uint4, uint2>::type;
    const int c = lane % kChunks, ch = d0 + 16 * c;
#pragma unroll 1
    for (int r0 = lane / kChunks; r0 < kRows; r0 += kBatch * (32 / kChunks)) {
      Code code[kBatch];
      uint8_t scale[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * (32 / kChunks);
        const RowGroup g = row_group(u, kTileGroups * tile + g0 + (r >> 6));
        const int pos = 64 * g.block + (r & 63);
        const int32_t page = group_page(p, u, g, pos);
        if constexpr (KVF == 1) code[i] = make_uint4(0u, 0u, 0u, 0u);
        else code[i] = make_uint2(0u, 0u);
        scale[i] = 0;
        if (page >= 0) {
          const uint8_t* src = p.kv.pages + page * p.kv.page_stride + (int64_t)(pos & page_mask) * kRowBytes;
          const uint8_t* sc = p.kv.scales + page * p.kv.scale_stride + (int64_t)(pos & page_mask) * kScaleBytes;
          if constexpr (KVF == 1) code[i] = ldg_stream16(src + ch);
          else code[i] = ldg_stream8(src + ch / 2);
          scale[i] = __ldg(sc + (KVF == 1 ? ch / 32 : ch / 16));
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = r0 + i * (32 / kChunks);
        uint32_t o[8];
        if constexpr (KVF == 1) fp8_to_bf16(code[i], scale[i], o);
        else fp4_to_bf16(code[i].x, code[i].y, scale[i], o);
        uint8_t* at = dst + (uint32_t)(c >> 2) * 8192u + (uint32_t)r * 128u;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(at + (((2 * (c & 3) + k) ^ (r & 7)) << 4)) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
  }
  fence_proxy_async_smem();
}

// What a tile's producers know of it: the number of its row groups; of lane
// 8 g + i the table's entry for piece i of group g (as it was read; -1: not
// wanted) and the row of that page where the piece begins; and which groups lie
// whole in the tile (bits 8 g). Read a tile before it is used, and not touched before
// that: 800 cycles of a round trip to the L2.
struct TileSource {
  int n;
  int32_t entry, row;
  uint32_t whole;
  // the page, past the end of the pages (where copies read zeros) for none
  __device__ __forceinline__ int32_t page(const SharedParams& p) const {
    return (uint32_t)entry < (uint32_t)p.kv.n_pages ? entry : p.kv.n_pages;
  }
};
__device__ __forceinline__ TileSource look_up(const SharedParams& p, const SharedUnit& u, int tile, int lane) {
  const int pc = piece_shift(p.kv.page_shift);
  TileSource src;
  src.n = uniform(row_groups(u, tile));
  const RowGroup g = row_group(u, kTileGroups * tile + (lane >> 3));
  const int pos = 64 * g.block + ((lane & 7) << pc), column = pos >> p.kv.page_shift;
  src.entry = -1;
  if ((lane & 7) < (kGroupRows >> pc) && g.present && pos < g.to && pos + (1 << pc) > g.from && column < p.kv.max_pages)
    src.entry = p.kv.table[(int64_t)(max(pos, g.from) < u.len ? u.head_seq : g.seq) * p.kv.table_ld + column];
  src.row = pos & ((1 << p.kv.page_shift) - 1);
  src.whole = __ballot_sync(0xffffffffu, (lane & 7) == 0 && g.present && g.from <= 64 * g.block && g.to >= 64 * g.block + 64);
  return src;
}
// A producer's way through its pair's run: keys(tile, source), values(tile,
// source) in the order of the products, look(tile) a tile ahead of both.
template <class Look, class Keys, class Values>
__device__ __forceinline__ void produce_tiles(SharedWalk& walk, Look&& look, Keys&& keys, Values&& values) {
  do {
    TileSource now = look(walk.first), ahead = now;
    if (walk.first + 1 < walk.last) ahead = look(walk.first + 1);
    keys(walk.first, now);
#pragma unroll 1
    for (int t = walk.first; t < walk.last; ++t) {
      TileSource next = ahead;
      if (t + 2 < walk.last) next = look(t + 2);
      if (t + 1 < walk.last) keys(t + 1, ahead);
      values(t, now);
      now = ahead;
      ahead = next;
    }
  } while (walk.next());
}

// fp8 and fp4 rows (pages of eight rows and more). A slot's codes, 128 runs of 64
// channels, are copied into the end of the slot itself and converted in place,
// from the front: 8 runs of bf16 take as much room as 16 (fp8) of codes leave, so
// that no code is overwritten before it has been read. A warp's next slot is on
// its way while it converts one (72 cycles a warp and 16 channels a lane, which
// is what bounds it: with the codes in registers, loaded four at a time, a slot
// took a warp 9,500 cycles, most of them waiting for the L2).
// Codes times their block's scale in bf16, exact: codes have at most 4 (e2m1: 2)
// significant bits, scales 1 (4), and the product is rounded like a float's.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t f16x2, __nv_bfloat162 sc) {
  const __half2_raw h{(unsigned short)(f16x2 & 0xFFFFu), (unsigned short)(f16x2 >> 16)};
  const __nv_bfloat162 v = __hmul2(__float22bfloat162_rn(__half22float2(__half2(h))), sc);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void scaled_e4m3(const uint4& codes, uint32_t scale, uint32_t (&o)[8]) {
  const __nv_bfloat162 sc = __float2bfloat162_rn(ue8m0_value(scale));
  const uint32_t cw[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[2 * k] = scaled_pair(e4m3x2_to_f16x2(cw[k] & 0xFFFFu), sc);
    o[2 * k + 1] = scaled_pair(e4m3x2_to_f16x2(cw[k] >> 16), sc);
  }
}
__device__ __forceinline__ void scaled_e2m1(const uint2& codes, uint32_t scale, uint32_t (&o)[8]) {
  const __nv_bfloat162 sc = __float2bfloat162_rn(e4m3_value(scale));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h[4];
    e2m1x8_to_f16x2x4_cvt(k == 0 ? codes.x : codes.y, h);
#pragma unroll
    for (int u = 0; u < 4; ++u) o[4 * k + u] = scaled_pair(h[u], sc);
  }
}

template <int KVF>
struct CodeProducer {
  static constexpr uint32_t NP = SharedRoles<false>::kProducers;
  static constexpr int kRowBytes = KVF == 1 ? 512 : 256, kScaleBytes = KVF == 1 ? 16 : 32;
  static constexpr uint32_t kRun = KVF == 1 ? 64u : 32u;  // code bytes of 64 channels
  using Code = typename std::conditional<KVF == 1, uint4, uint2>::type;
  const SharedParams& p;
  uint8_t* sm;
  uint32_t base_s, bars, full0, leader, here;
  int w, rank, lane, pc, pieces;
  SharedWalk& walk;
  RingAt base{0, 0};  // the next slot of all warps, and the slots before it
  uint32_t s = 0, asked = 0;
  bool live = true;
  // A slot whose codes are on their way: its place (bar 0: none); of runs 32 i +
  // lane their scales (two bytes, fp4: four), which nothing touches before the slot
  // is converted, and which runs are there (bits).
  struct Asked {
    uint32_t slot, bar, scales[4], there[4];
  };
  Asked on{0u, 0u, {0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}};

  // Runs 64 k .. of a slot, k < n: row group g0 + k's (K), or of one group its
  // dims d0 + 64 k .. (V).
  __device__ __forceinline__ void ask(const TileSource& src, int tile, bool is_k, int n, int g0, int d0, uint32_t slot, uint32_t bar) {
    on.slot = slot;
    on.bar = bar;
    const int32_t page = src.page(p);
    const uint32_t dst = base_s + slot + kSlotBytes - 128u * kRun;
    expect_one(leader, here, 64u * kRun * (uint32_t)n);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int g = is_k ? g0 + k : g0, ch = is_k ? d0 : d0 + 64 * k;
      if (k < n) {
#pragma unroll 1
        for (int i = 0; i < pieces; ++i)
          tma_3d_one(leader, dst + (64u * (uint32_t)k + (uint32_t)(i << pc)) * kRun, &p.code_map, ch * (int)kRun / 64,
                     uniform(src.row, 8 * g + i), uniform(page, 8 * g + i), here);
      }
      const RowGroup rg = row_group(walk.u, kTileGroups * tile + g);
      const int from = rg.from - 64 * rg.block, to = k < n && rg.present ? rg.to - 64 * rg.block : 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = 32 * i + lane;
        const int of = 8 * (g & 3) + (r >> pc);  // the lane that has the run's page
        const int32_t run_page = __shfl_sync(0xffffffffu, page, of), run_row = __shfl_sync(0xffffffffu, src.row, of);
        const bool there = run_page < p.kv.n_pages && r >= from && r < to;
        const uint8_t* sp = p.kv.scales + run_page * p.kv.scale_stride +
                            (uint32_t)((run_row + (r & ((1 << pc) - 1))) * kScaleBytes + ch / (KVF == 1 ? 32 : 16));
        uint32_t sc = 0u;
        if constexpr (KVF == 1) {
          if (there) sc = __ldg(reinterpret_cast<const uint16_t*>(sp));
        } else {
          if (there) sc = __ldg(reinterpret_cast<const uint32_t*>(sp));
        }
        on.scales[2 * k + i] = sc;
        on.there[2 * k + i] = __ballot_sync(0xffffffffu, there);
      }
    }
    ++asked;
  }
  // (asked for one after another on one barrier: each has landed before the next is counted)
  __device__ __forceinline__ void landed() { live = live && wait_all_lanes(here, (asked - 1u) & 1u, p.flags); }
  // A lane has channels 16 (lane & 3) .. of runs lane >> 2, + 8, ...
  __device__ __forceinline__ void convert(const Asked& a) const {
    const uint8_t* code_at = sm + a.slot + kSlotBytes - 128u * kRun + (kRun / 4u) * (uint32_t)lane;
    const int r = lane >> 2, c = lane & 3;
    uint8_t* out = sm + a.slot + 128u * (uint32_t)r;
#pragma unroll 1
    for (int j4 = 0; j4 < 4; ++j4) {
      Code code[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) code[i] = *reinterpret_cast<const Code*>(code_at + 8u * kRun * (uint32_t)(4 * j4 + i));
      __syncwarp();  // all lanes have read what the stores below may overwrite
      const uint32_t scales = j4 == 0 ? a.scales[0] : (j4 == 1 ? a.scales[1] : (j4 == 2 ? a.scales[2] : a.scales[3]));
      const uint32_t there = j4 == 0 ? a.there[0] : (j4 == 1 ? a.there[1] : (j4 == 2 ? a.there[2] : a.there[3]));
      uint32_t word[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) word[i] = __shfl_sync(0xffffffffu, scales, 8 * i + r);
      if (there != 0xFFFFFFFFu) {  // rows that are not the group's: zeros
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (((there >> (8 * i + r)) & 1u) != 0u) continue;
          if constexpr (KVF == 1) code[i] = make_uint4(0u, 0u, 0u, 0u);
          else code[i] = make_uint2(0u, 0u);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t sc = (word[i] >> (KVF == 1 ? 8 * (c >> 1) : 8 * c)) & 255u;
        uint32_t o[8];
        if constexpr (KVF == 1) scaled_e4m3(code[i], sc, o);
        else scaled_e2m1(code[i], sc, o);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<uint4*>(out + 1024u * (uint32_t)(4 * j4 + i) + (((2 * c + k) ^ r) << 4)) =
              make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      }
    }
    fence_proxy_async_smem();
    warp_arrive_cluster(a.bar);
  }
  __device__ __forceinline__ void flush() {
    if (on.bar == 0u) return;
    landed();
    convert(on);
    on.bar = 0u;
  }
  __device__ __forceinline__ void finish() {
    flush();
    if (w == 0) drain_ring(p, bars, base, s, live);
  }
  // this warp's slots of the next `count`
  __device__ __forceinline__ void slots(uint32_t count, int tile, const TileSource& src, bool is_k) {
    const int n = is_k ? min(2, max(0, src.n - 2 * rank)) : 2;
#pragma unroll 1
    for (uint32_t i = (w + NP - s % NP) % NP; i < count; i += NP) {
      RingAt at = base;
      at.step(i);
      const uint32_t empty = bars + 8 * (bEmpty + at.slot);
      if (s + i >= (uint32_t)kRing) {
        // (not free yet: the one on its way is converted meanwhile)
        if (!uniform(phase_done(empty, at.phase ^ 1u) != 0u)) flush();
        live = live && wait_cluster_all_lanes(empty, at.phase ^ 1u, p.flags);
      }
      if (on.bar != 0u) landed();
      const Asked last = on;
      ask(src, tile, is_k, n, is_k ? 2 * rank : (int)i >> 1, is_k ? 64 * (int)i : 256 * ((int)i & 1) + 128 * rank,
          S_RING + at.slot * kSlotBytes, full0 + 8 * at.slot);
      if (last.bar != 0u) convert(last);
    }
    base.step(count);
    s += count;
  }
};

template <int KVF>
__device__ __forceinline__ void produce_codes(const SharedParams& p, uint8_t* sm, uint32_t base_s, SharedWalk walk, int w, int rank) {
  if (walk.left <= 0) return;
  const uint32_t bars = base_s + S_BAR;
  const int pc = piece_shift(p.kv.page_shift);
  CodeProducer<KVF> c{p, sm, base_s, bars, in_leader(bars + 8 * bFull), elect_one(), bars + 8 * (bEdge + (uint32_t)w), w, rank,
                      (int)(threadIdx.x & 31), pc, kGroupRows >> pc, walk};
  produce_tiles(
      walk,
      [&](int tile) { return look_up(p, walk.u, tile, c.lane); },
      [&](int tile, const TileSource& src) {
        // codes on their way to the L2, half of the tile's rows by either CTA
        const int32_t page = src.page(p);
        if (w == 0 && (c.lane >> 4) == rank && page < p.kv.n_pages) {
          prefetch_l2(p.kv.pages + page * p.kv.page_stride + (int64_t)src.row * c.kRowBytes, (uint32_t)c.kRowBytes << pc);
          prefetch_l2(p.kv.scales + page * p.kv.scale_stride + (int64_t)src.row * c.kScaleBytes, (uint32_t)c.kScaleBytes << pc);
        }
        c.slots(8, tile, src, true);
      },
      [&](int tile, const TileSource& src) { c.slots(2u * (uint32_t)src.n, tile, src, false); });
  c.finish();
}

// Producer warp w of a CTA: every kProducers-th slot of the ring. What a tile's
// copies need is found once a tile, before the waits for its slots: with the look-up
// behind them the warps took 1,300 cycles to issue a slot's two copies.
template <int KVF, bool TMA>
__device__ __forceinline__ void produce_role(const SharedParams& p, uint8_t* sm, uint32_t base_s, SharedWalk walk, int w, int rank) {
  constexpr uint32_t NP = SharedRoles<TMA>::kProducers;
  const int lane = threadIdx.x & 31;
  const uint32_t bars = base_s + S_BAR, full0 = in_leader(bars + 8 * bFull);
  const uint32_t leader = elect_one();
  const int ps = p.kv.page_shift, pc = piece_shift(ps);
  const int pieces = kGroupRows >> pc;
  RingAt base{0, 0};  // the next slot of all warps, and the slots before it
  uint32_t s = 0, edges = 0;
  bool live = true;
  auto look = [&](int tile) {
    if (TMA) return look_up(p, walk.u, tile, lane);
    return TileSource{uniform(row_groups(walk.u, tile)), -1, 0, 0u};
  };
  // this warp's slots of the next `count`: fill(i, its place)
  auto each = [&](uint32_t count, auto&& fill) {
#pragma unroll 1
    for (uint32_t i = (w + NP - s % NP) % NP; i < count; i += NP) {
      RingAt at = base;
      at.step(i);
      if (s + i >= (uint32_t)kRing) live = live && wait_cluster_all_lanes(bars + 8 * (bEmpty + at.slot), at.phase ^ 1u, p.flags);
      if (live) fill((int)i, full0 + 8 * at.slot, at.slot * kSlotBytes + S_RING);
    }
    base.step(count);
    s += count;
  };
  auto keys = [&](int tile, const TileSource& src) {
    const int n = min(2, max(0, src.n - 2 * rank));  // row groups of this CTA's half
    const int32_t page = src.page(p);
    const int page0 = uniform(page, 16 * rank), page1 = uniform(page, 16 * rank + 8);
    const int row0 = uniform(src.row, 16 * rank), row1 = uniform(src.row, 16 * rank + 8);
    each(8, [&](int b, uint32_t bar, uint32_t slot) {
      const uint32_t dst = base_s + slot;
      if (!TMA) {
        if (n > 0) fill_slot<KVF, true>(p, walk.u, tile, 2 * rank, 64 * b, dst, sm + slot, lane);
        warp_arrive_cluster(bar);
        return;
      }
      expect_cluster_one(leader, bar, 8192u * (uint32_t)n);
      if (pieces == 1) {
        if (n > 0) tma_pair_3d(leader, dst, &p.kv_map, 64 * b, row0, page0, bar);
        if (n > 1) tma_pair_3d(leader, dst + 8192u, &p.kv_map, 64 * b, row1, page1, bar);
      } else {
#pragma unroll 1
        for (int g = 0; g < n; ++g) {
#pragma unroll 1
          for (int i = 0; i < pieces; ++i)
            tma_pair_3d(leader, dst + 8192u * (uint32_t)g + ((uint32_t)i << (7 + pc)), &p.kv_map, 64 * b, 0,
                        uniform(page, 8 * (2 * rank + g) + i), bar);
        }
      }
    });
  };
  auto values = [&](int tile, const TileSource& src) {
    const int32_t pages = src.page(p);
    each(2 * (uint32_t)src.n, [&](int i, uint32_t bar, uint32_t slot) {
      const int g = i >> 1, d0 = 256 * (i & 1) + 128 * rank;
      const uint32_t dst = base_s + slot;
      if (!TMA) {
        fill_slot<KVF, false>(p, walk.u, tile, g, d0, dst, sm + slot, lane);
        warp_arrive_cluster(bar);
        return;
      }
      if (((src.whole >> (8 * g)) & 1u) == 0u) {
        // A group that ends inside its 64 positions: the rows behind it hold
        // anything, and are cleared once they have landed (their weights are 0, but
        // 0 times a NaN is not). Copied by the warp itself such a slot took it
        // 2 us, and the ring with it.
        const RowGroup rg = row_group(walk.u, kTileGroups * tile + g);
        const uint32_t here = bars + 8 * (bEdge + (uint32_t)w);
        expect_one(leader, here, kSlotBytes);
        if (pieces == 1) {
          const int page = uniform(pages, 8 * g), row = uniform(src.row, 8 * g);
          tma_3d_one(leader, dst, &p.kv_map, d0, row, page, here);
          tma_3d_one(leader, dst + 8192u, &p.kv_map, d0 + 64, row, page, here);
        } else {
#pragma unroll 1
          for (int k = 0; k < pieces; ++k) {
            const int page = uniform(pages, 8 * g + k);
            tma_3d_one(leader, dst + ((uint32_t)k << (7 + pc)), &p.kv_map, d0, 0, page, here);
            tma_3d_one(leader, dst + 8192u + ((uint32_t)k << (7 + pc)), &p.kv_map, d0 + 64, 0, page, here);
          }
        }
        live = live && wait_all_lanes(here, edges & 1u, p.flags);
        ++edges;
        // lanes 0 .. 15 a row's 256 bytes, lanes 16 .. 31 the next one's
        const uint32_t chunk = dst + 8192u * ((lane >> 3) & 1) + 16u * (lane & 7);
        const int from = rg.from - 64 * rg.block, to = rg.to - 64 * rg.block;
#pragma unroll 4
        for (int r = lane >> 4; r < kGroupRows; r += 2) zero16_if(r < from || r >= to ? 1u : 0u, chunk + 128u * (uint32_t)r);
        fence_proxy_async_smem();
        warp_arrive_cluster(bar);
        return;
      }
      expect_cluster_one(leader, bar, kSlotBytes);
      if (pieces == 1) {
        tma_pair_4d(leader, dst, &p.v_map, 0, uniform(src.row, 8 * g), d0 / 64, uniform(pages, 8 * g), bar);
      } else {
#pragma unroll 1
        for (int k = 0; k < pieces; ++k) {
          const int page = uniform(pages, 8 * g + k);
          tma_pair_3d(leader, dst + ((uint32_t)k << (7 + pc)), &p.kv_map, d0, 0, page, bar);
          tma_pair_3d(leader, dst + 8192u + ((uint32_t)k << (7 + pc)), &p.kv_map, d0 + 64, 0, page, bar);
        }
      }
    });
  };
  if (walk.left <= 0) return;
  produce_tiles(walk, look, keys, values);
  if (w == 0) drain_ring(p, bars, base, s, live);
}

// Q of this CTA's query: plain blocks by TMA, the rope block rotated and split
// into bf16 hi + lo by the role's threads (see csa2_attend_paged).
template <int WARPS>
__device__ __forceinline__ void q_role(const SharedParams& p, uint8_t* sm, uint32_t base_s, SharedWalk walk, int t, int rank) {
  const uint32_t bars = base_s + S_BAR, bar = in_leader(bars + 8 * bQFull);
  const uint32_t leader = elect_one();
  const bool rope = p.rp.pairs > 0;
  const double freq = t < p.rp.pairs ? p.rp.freq[t & 31] : 0.0;
  bool live = true;
  if (walk.left <= 0) return;
  uint32_t seg = 0;
  do {
    const int qi = uniform(rank == 0 ? walk.u.q[0] : walk.u.q[1]);
    const int64_t t_q = rank == 0 ? walk.u.t[0] : walk.u.t[1];
    // (a wait that ran out is recorded; the barriers below are met all the same)
    if (seg > 0) live = live && wait_cluster_all_lanes(bars + 8 * bQEmpty, (seg & 1u) ^ 1u, p.flags);
    if (t < 32 && live) {
      const int plain = qi < 0 ? 0 : (rope ? 7 : 8);
      expect_cluster_one(leader, bar, 8192u * (uint32_t)plain);
#pragma unroll 1
      for (int b = 0; b < plain; ++b) tma_pair_2d(leader, base_s + S_Q + 8192u * (uint32_t)b, &p.q_map, 64 * b, kHeads * qi, bar);
    }
    if (rope && qi >= 0) {
      // thread: chunk 56 + (t & 7) of every 4 WARPS-th head: always the same four pairs
      constexpr int kStep = 4 * WARPS;
      float2* table = reinterpret_cast<float2*>(sm + S_QROPE);
      const uint16_t* q = p.q + (int64_t)qi * kHeads * kDim + 8 * (56 + (t & 7));
#pragma unroll 1
      for (int h0 = t >> 3; h0 < kHeads; h0 += 8 * kStep) {
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint4*>(q + (int64_t)(h0 + kStep * i) * kDim);
        if (h0 < kStep) {
          asm volatile("bar.sync 3, %0;" ::"n"(32 * WARPS) : "memory");  // the last query's table has been read
          if (t < 32) {
            float cs, sn;
            angle_cs((double)max(t_q, (int64_t)0) * freq, cs, sn);
            table[t] = make_float2(cs, sn);
          }
          asm volatile("bar.sync 3, %0;" ::"n"(32 * WARPS) : "memory");
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int h = h0 + kStep * i;
          uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, lo[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 cs = table[4 * (t & 7) + k];
            const float x0 = bf16lo(w[k]), x1 = bf16hi(w[k]);
            const float y0 = x0 * cs.x - x1 * cs.y, y1 = x0 * cs.y + x1 * cs.x;
            w[k] = pack_bf16(y0, y1);
            lo[k] = pack_bf16(y0 - bf16lo(w[k]), y1 - bf16hi(w[k]));
          }
          const uint32_t off = (uint32_t)h * 128u + ((uint32_t)((t & 7) ^ (h & 7)) << 4);
          *reinterpret_cast<uint4*>(sm + S_Q + 7u * 8192u + off) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(sm + S_Q + 8u * 8192u + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
    }
    if (live) warp_arrive_cluster(bar);
    ++seg;
  } while (walk.next());
  if (t < 32 && live) wait_cluster_all_lanes(bars + 8 * bQEmpty, (seg & 1u) ^ 1u, p.flags);  // (as drain_ring)
}

// The pair's products, by a warp of CTA 0.
__device__ __forceinline__ void issue_shared(const SharedParams& p, uint32_t base_s, uint32_t tmem_s, uint32_t tmem_o, SharedWalk walk) {
  const uint32_t bars = base_s + S_BAR, leader = elect_one();
  uint32_t* flags = p.flags;
  const bool rope = p.rp.pairs > 0;
  const uint64_t qd = sdesc_sw128(base_s + S_Q, 16u, 1024u), pd = sdesc_sw128(base_s + S_P, 16u, 1024u);
  const uint64_t kd = sdesc_sw128(base_s + S_RING, 16u, 1024u), vd = sdesc_sw128(base_s + S_RING, 8192u, 1024u);
  RingAt at{0, 0};
  uint32_t n = 0, done = 0, seg = 0;  // tiles scored, tiles whose outputs were issued, units
  bool live = true;
  // The slot whose turn it is, waited for. Its barrier was looked at while the
  // products of the slot before were issued: a look takes some 300 cycles from
  // the instruction to the branch, longer than a slot's products run. When a
  // wait has run out (live: false) nothing is waited for any more and the
  // products go on, on whatever lies there, so that every role comes to its end.
  uint32_t landed = 0;
  auto ready = [&]() {
    if (!uniform(landed != 0u)) live = live && wait_cluster_all_lanes(bars + 8 * (bFull + at.slot), at.phase, flags);
    tc_fence_after();
    RingAt next = at;
    next.step(1);
    landed = done_cluster(bars + 8 * (bFull + next.slot), next.phase);
  };
  auto scores = [&](bool last) {
    const uint32_t d = tmem_s + 128u * (n & 1u);
#pragma unroll 1
    for (uint32_t b = 0; b < 8; ++b, at.step(1)) {
      ready();
      const uint64_t k0 = sdesc_add(kd, (uint32_t)uniform((int)at.slot) * kSlotBytes);
#pragma unroll
      for (uint32_t k = 0; k < 4; ++k) mma_pair(leader, d, sdesc_add(qd, b * 8192u + 32u * k), sdesc_add(k0, 32u * k), kIdescS, b | k);
      if (rope && b == 7) {
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) mma_pair(leader, d, sdesc_add(qd, 8u * 8192u + 32u * k), sdesc_add(k0, 32u * k), kIdescS, 1u);
      }
      commit_pair(leader, bars + 8 * (bEmpty + at.slot));
    }
    commit_pair(leader, bars + 8 * (bScores + (n & 1u)));
    if (last) commit_pair(leader, bars + 8 * bQEmpty);
    ++n;
  };
  if (walk.left > 0) {
    do {
      live = live && wait_cluster_all_lanes(bars + 8 * bQFull, seg & 1u, flags);
      tc_fence_after();
      scores(walk.first + 1 == walk.last);
      uint32_t holds = 0;  // whose lanes of O hold a sum (bits)
#pragma unroll 1
      for (int t = walk.first; t < walk.last; ++t) {
        if (t + 1 < walk.last) scores(t + 2 == walk.last);
        const uint32_t formed = done_cluster(bars + 8 * bWeights, done & 1u);
        // who sees the tile's row groups, and (in the same places) whether their
        // lanes of O hold a sum already
        uint32_t whose = 0, begun = holds != 0u ? 0x55u : 0x54u;
        const uint32_t ng = (uint32_t)uniform(row_groups(walk.u, t));
        const bool common = uniform(kTileGroups * (t + 1) <= walk.u.n[0]);
        if (common) {
          holds = 3u;
        } else {
          begun = 0;
#pragma unroll 1
          for (int g = 0; g < (int)ng; ++g) {
            const uint32_t who = (uint32_t)row_group(walk.u, kTileGroups * t + g).who, lanes = who == 0u ? 3u : who;
            whose |= who << (2 * g);
            begun |= ((holds & lanes) != 0u ? 1u : 0u) << (2 * g);
            holds |= lanes;
          }
          whose = (uint32_t)uniform((int)whose);
        }
        begun = (uint32_t)uniform((int)begun);
        if (!uniform(formed != 0u)) live = live && wait_cluster_all_lanes(bars + 8 * bWeights, done & 1u, flags);
        if (t == walk.first && seg > 0) live = live && wait_cluster_all_lanes(bars + 8 * bOFree, (seg & 1u) ^ 1u, flags);
        tc_fence_after();
        // the products of a slot: half j of the dims, row group g
        auto slot_products = [&](uint32_t g, uint32_t j, uint32_t keep, uint32_t who) {
          ready();
          const uint64_t v0 = sdesc_add(vd, (uint32_t)uniform((int)at.slot) * kSlotBytes), p0 = sdesc_add(pd, 8192u * g);
          const uint32_t d = tmem_o + 128u * j;
          if (who == 0u) {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) mma_pair(leader, d, sdesc_add(p0, 32u * k), sdesc_add(v0, 2048u * k), kIdescO, k | keep);
          } else {
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k)
              mma_pair_lanes(leader, d, sdesc_add(p0, 32u * k), sdesc_add(v0, 2048u * k), kIdescO, k | keep, who == 1u ? 0u : ~0u,
                             who == 1u ? ~0u : 0u);
          }
          commit_pair(leader, bars + 8 * (bEmpty + at.slot));
          at.step(1);
        };
        if (common) {
#pragma unroll 1
          for (uint32_t g = 0; g < (uint32_t)kTileGroups; ++g) {
            slot_products(g, 0, g != 0u || begun == 0x55u ? 1u : 0u, 0u);
            slot_products(g, 1, g != 0u || begun == 0x55u ? 1u : 0u, 0u);
          }
        } else {
#pragma unroll 1
          for (uint32_t i = 0; i < 2u * ng; ++i) slot_products(i >> 1, i & 1u, (begun >> (i & ~1u)) & 1u, (whose >> (i & ~1u)) & 3u);
        }
        commit_pair(leader, bars + 8 * bPFree);
        ++done;
      }
      ++seg;
    } while (walk.next());
  }
  if (!live) {  // products still in flight land before tensor memory is freed
    commit_pair(leader, bars + 8 * bDrained);
    wait_phase(bars + 8 * bDrained, 0u, flags);
  }
}

// Softmax of a tile and, at a unit's end, its output or partial. Warp w: TMEM
// lanes 32 (w & 3) .., which hold heads 32 (w & 1) .. + 31, of S its columns
// 128 ((w >> 1) & 1) .. (the upper lanes hold the second half of N), of which
// the warp takes 64 (w >> 2) ..: a thread has one head and the 64 rows of row
// group 2 ((w >> 1) & 1) + (w >> 2). Four threads share a head, the four warps of
// its half of the heads a barrier.
__device__ __forceinline__ void math_shared(const SharedParams& p, uint8_t* sm, uint32_t base_s, uint32_t tmem_s, uint32_t tmem_o,
                                            SharedWalk walk, int c, int warp, int rank) {
  const uint32_t bars = base_s + S_BAR;
  const uint32_t weights = in_leader(bars + 8 * bWeights), o_free = in_leader(bars + 8 * bOFree);
  const int lane = threadIdx.x & 31, hb = warp & 1, upper = (warp >> 1) & 1, cols = warp >> 2;
  const int head = 32 * hb + lane, group = 2 * upper + cols;
  const uint32_t lane_base = (uint32_t)(32 * (warp & 3)) << 16;
  float* red = reinterpret_cast<float*>(sm + S_RED);
  float2* rope_tab = reinterpret_cast<float2*>(sm + S_ROPE) + 32 * hb;
  const float scale = p.scale_log2;
  auto sync_half = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + hb) : "memory"); };
  auto any_half = [&](bool v) {
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %1, 0;\nbar.red.or.pred q, %2, 128, p;\nselp.u32 %0, 1, 0, q;\n}"
                 : "=r"(r)
                 : "r"((uint32_t)v), "r"(1 + hb)
                 : "memory");
    return r != 0;
  };
  if (walk.left <= 0) return;
  bool live = true;  // a wait that ran out is recorded; the loop then only runs out
  uint32_t n = 0;
  do {
    const SharedUnit& u = walk.u;
    const int qi = rank == 0 ? u.q[0] : u.q[1];
    const int64_t t_q = rank == 0 ? u.t[0] : u.t[1];
    if (upper + cols == 0 && lane < p.rp.pairs) {
      float cs, sn;
      rope_cs(p.rp, lane, max(t_q, (int64_t)0), cs, sn);
      rope_tab[lane] = make_float2(cs, sn);  // read behind the barriers of the unit's end
    }
    float m_run = -INFINITY, m_use = kNoRef, lsum = 0.f;
#pragma unroll 1
    for (int t = walk.first; t < walk.last; ++t, ++n) {
      // the rows that this query sees of the warp's group
      uint32_t mask[2];
      {
        const RowGroup g = row_group(u, kTileGroups * t + group);
        const bool mine = g.present && (g.who == 0 || g.who == rank + 1) && (rank == 0 ? u.end[0] : u.end[1]) > 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int pos = 64 * g.block + 32 * i + lane;
          const bool seen = mine && pos >= g.from && pos < g.to;
          const bool there = seen && group_page(p, u, g, pos) >= 0;
          if (seen && !there) set_flag(p.flags, CSA2_FLAG_BAD_PAGE);
          mask[i] = __ballot_sync(0xffffffffu, there);
        }
      }
      live = live && warp_wait_cluster(bars + 8 * (bScores + (n & 1u)), (n >> 1) & 1u, p.flags);
      tc_fence_after();
      const uint32_t s_at = tmem_s + 128u * (n & 1u) + lane_base + 64u * cols;
      const bool first = t == walk.first;
      bool move = first;
      uint32_t packed[32];
      float add = 0.f;
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        if (move) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t r[32];
            tmem_ld32(s_at + 32u * i, r);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) top = fmaxf(top, (mask[i] >> k) & 1u ? __uint_as_float(r[k]) * scale : -INFINITY);
          }
          red[64 * group + head] = top;
          sync_half();
          top = fmaxf(fmaxf(red[head], red[64 + head]), fmaxf(red[128 + head], red[192 + head]));
          const float mn = (m_run == -INFINITY || top > m_run + kRefSlack) ? fmaxf(m_run, top) : m_run;
          const float al = m_run == -INFINITY ? 1.f : exp2f(m_run - mn);
          m_run = mn;
          m_use = mn == -INFINITY ? kNoRef : mn;
          if (any_half(al != 1.f)) {
            lsum *= al;
            // the products of the tile before are complete
            if (!first) live = live && warp_wait_cluster(bars + 8 * bPFree, (n & 1u) ^ 1u, p.flags);
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              const uint32_t a = tmem_o + lane_base + 128u * cols + 32u * i;
              uint32_t r[32];
              tmem_ld32(a, r);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * al);
              tmem_st32(a, r);
            }
            tmem_wait_st();
          }
        }
        float over = -INFINITY;
        add = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t r[32];
          tmem_ld32(s_at + 32u * i, r);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            float x0 = fmaf(__uint_as_float(r[k]), scale, -m_use), x1 = fmaf(__uint_as_float(r[k + 1]), scale, -m_use);
            if (!((mask[i] >> k) & 1u)) x0 = -INFINITY;
            if (!((mask[i] >> (k + 1)) & 1u)) x1 = -INFINITY;
            over = fmaxf(over, fmaxf(x0, x1));
            x0 = exp2_approx(x0);
            x1 = exp2_approx(x1);
            add += x0 + x1;
            packed[16 * i + k / 2] = pack_bf16(x0, x1);
          }
        }
        move = any_half(over > kRefSlack);
        if (!move) break;
      }
      lsum += add;
      // the products of the tile before have read its weights
      if (n > 0) live = live && warp_wait_cluster(bars + 8 * bPFree, (n & 1u) ^ 1u, p.flags);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        *reinterpret_cast<uint4*>(sm + S_P + 8192u * (uint32_t)group + 128u * (uint32_t)head + (uint32_t)((k ^ (head & 7)) << 4)) =
            make_uint4(packed[4 * k], packed[4 * k + 1], packed[4 * k + 2], packed[4 * k + 3]);
      fence_proxy_async_smem();
      tc_fence_before();
      warp_arrive_cluster(weights);
    }
    // ---- the unit's end: the four threads' sums of a head, then O
    red[64 * group + head] = lsum;
    sync_half();
    const float l = red[head] + red[64 + head] + red[128 + head] + red[192 + head];
    const bool none = m_run == -INFINITY && l == l;  // no row seen (scores that are all NaN set no reference either)
    live = live && warp_wait_cluster(bars + 8 * bPFree, (n & 1u) ^ 1u, p.flags);
    tc_fence_after();
    const bool whole = walk.begins && walk.ends;
    // dims of the warp's columns: N runs over CTA 0's 128 dims of a half, then CTA 1's
    const int dim0 = 256 * cols + 128 * upper;
    if (whole) {
      const float sk = p.sink != nullptr ? p.sink[head] : -INFINITY, sk2 = sk * 1.4426950408889634f;
      const float M = fmaxf(m_run, sk2);
      float fo = 0.f, lse = sk;
      if (!none) {
        const float em = exp2f(m_run - M);
        const float den = l * em + exp2f(sk2 - M);
        fo = em / den;
        lse = (M + log2f(den)) * 0.6931471805599453f;
      }
      if (qi >= 0 && group == 0 && p.lse != nullptr) p.lse[(int64_t)qi * kHeads + head] = lse;
      const int first_rope = kDim - 2 * p.rp.pairs;
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        uint32_t r[32];
        tmem_ld32(tmem_o + lane_base + 128u * cols + 32u * i, r);
        tmem_wait_ld();
        const int d = dim0 + 32 * i;
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          float x0 = none ? 0.f : __uint_as_float(r[k]) * fo, x1 = none ? 0.f : __uint_as_float(r[k + 1]) * fo;
          if (d >= first_rope) {  // rotated back by -t
            const float2 cs = rope_tab[(d + k - first_rope) >> 1];
            const float y = x0 * cs.x + x1 * cs.y;
            x1 = x1 * cs.x - x0 * cs.y;
            x0 = y;
          }
          r[k / 2] = pack_bf16(x0, x1);
        }
        if (qi >= 0) {
          uint4* dst = reinterpret_cast<uint4*>(p.out + ((int64_t)qi * kHeads + head) * kDim + d);
#pragma unroll
          for (int k = 0; k < 4; ++k) dst[k] = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
        }
      }
    } else {
      const int64_t slot = shared_slot(c, walk.begins, rank);
      if (group == 0) {
        p.part_ml[slot * kHeads + head] = make_float2(m_run, l);
      }
      float4* po = reinterpret_cast<float4*>(p.part_o) + slot * (kDim / 4) * kHeads;
#pragma unroll 2
      for (int i = 0; i < 4; ++i) {
        uint32_t r[32];
        tmem_ld32(tmem_o + lane_base + 128u * cols + 32u * i, r);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          float4 v = make_float4(__uint_as_float(r[4 * k]), __uint_as_float(r[4 * k + 1]), __uint_as_float(r[4 * k + 2]),
                                 __uint_as_float(r[4 * k + 3]));
          if (none) v = make_float4(0.f, 0.f, 0.f, 0.f);  // nothing was summed into these lanes
          po[(dim0 / 4 + 8 * i + k) * kHeads + head] = v;
        }
      }
    }
    tc_fence_before();  // O has been read
    warp_arrive_cluster(o_free);
    sync_half();  // red and the rope table are free for the next unit
  } while (walk.next());
}

// The plan of up to kPlanHere places by the CTA's own threads, and this pair's run.
__device__ __forceinline__ void plan_here(const SharedParams& p, uint8_t* sm, SharedWalk& walk, int c, int rank) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kWarps = kPlanHere / 32;
  SharedUnit* units = reinterpret_cast<SharedUnit*>(sm + S_UNITS);
  int64_t* sum_t = reinterpret_cast<int64_t*>(sm + S_SUMS);
  int* sum_u = reinterpret_cast<int*>(sm + S_SUMS + 32);
  SharedRun* cut = reinterpret_cast<SharedRun*>(sm + S_SUMS + 48);
  PlanUnit one;
  one.begins = false;
  uint32_t bad = 0;
  int64_t it = 0;
  int iu = 0;
  if (warp < kWarps) {
    // every warp looks at all places' heads: where runs of equal ones begin (bits)
    int32_t head[kWarps];
    uint32_t begins[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) head[w] = 32 * w + lane < p.n_query ? p.head[32 * w + lane] : kNoPlace;
    PlanPlace at{kNoPlace, kNoPlace, 0};
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const int32_t up = __shfl_up_sync(0xffffffffu, head[w], 1), last = __shfl_sync(0xffffffffu, head[max(w, 1) - 1], 31);
      const int32_t down = __shfl_down_sync(0xffffffffu, head[w], 1), first = __shfl_sync(0xffffffffu, head[min(w + 1, kWarps - 1)], 0);
      begins[w] = __ballot_sync(0xffffffffu, lane == 0 ? w == 0 || head[w] != last : head[w] != up);
      if (w == warp) {
        at.head = head[w];
        at.next = lane < 31 ? down : (w + 1 < kWarps ? first : kNoPlace);
      }
    }
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t till = w < warp ? begins[w] : (w == warp ? begins[w] & (0xFFFFFFFFu >> (31 - lane)) : 0u);
      if (till != 0u) at.run = 32 * w + 31 - __clz((int)till);
    }
    if (tid < p.n_query) one = unit_at(p, tid, at, bad);
    if (bad && blockIdx.x == 0) set_flag(p.flags, bad);
    it = one.begins ? one.u.tiles : 0;
    iu = one.begins ? 1 : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t a = __shfl_up_sync(0xffffffffu, it, o);
      const int b = __shfl_up_sync(0xffffffffu, iu, o);
      if (lane >= o) it += a, iu += b;
    }
    if (lane == 31) sum_t[warp] = it, sum_u[warp] = iu;
  }
  __syncthreads();
  int64_t T = 0, t0 = it - (one.begins ? one.u.tiles : 0);
  int U = 0, u0 = iu - (one.begins ? 1 : 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) t0 += sum_t[w], u0 += sum_u[w];
    T += sum_t[w];
    U += sum_u[w];
  }
  const RunLine line(T, U, p.pairs);
  if (tid == 0) {
    if (c >= line.runs) cut[0] = SharedRun{T, U, 0};
    if (c + 1 >= line.runs) cut[1] = SharedRun{T, U, 0};
  }
  if (one.begins) {
    units[u0] = one.u;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int64_t y = (c + e) * line.cost;
      if (c + e < line.runs && y >= line.at(t0, u0) && y < line.at(t0 + one.u.tiles, u0 + 1)) {
        const int64_t j = line.tile_from(c + e, t0, u0);
        cut[e] = j < one.u.tiles ? SharedRun{t0 + j, u0, (int32_t)j} : SharedRun{t0 + one.u.tiles, u0 + 1, 0};
      }
    }
  }
  __syncthreads();
  const SharedRun from = cut[0], to = cut[1];
  // a unit that begins in this run and goes on
  const bool goes_on = one.begins && t0 >= from.tile && t0 < to.tile && t0 + one.u.tiles > to.tile;
  const int4 jn = goes_on ? make_int4(one.u.q[0], one.u.q[1], c, line.run_of(t0, u0, one.u.tiles - 1)) : make_int4(-1, -1, -1, 0);
  if (p.n_query >= p.pairs) {
    const bool any = __syncthreads_or(goes_on) != 0;
    if (rank == 0 && (goes_on || (!any && tid == 0))) p.joins[c] = jn;
  } else if (rank == 0) {
    if (one.begins && t0 >= from.tile && t0 < to.tile) p.joins[u0] = jn;
    if (c == 0 && tid >= U && tid < p.n_query) p.joins[tid] = make_int4(-1, -1, -1, 0);
  }
  walk.start(units, from, to.tile - from.tile);
}

template <int KVF, bool TMA>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(SharedRoles<TMA>::kThreads, 1)
    attend_shared_kernel(const __grid_constant__ SharedParams p) {
  extern __shared__ uint8_t smem_raw[];
  using Roles = SharedRoles<TMA>;
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (base_s - raw_s);
  const uint32_t bars = base_s + S_BAR;
  const int tid = threadIdx.x;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rank = (int)cluster_rank(), c = (int)blockIdx.x >> 1;
  pdl_trigger();
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(base_s + S_MISC) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 32 * kMathWarps) {
    for (uint32_t b = 0; b < kSBars; ++b) {
      uint32_t count = 1;
      if (b < bEmpty) count = 2;                                      // each CTA once
      else if (b == bQFull) count = 2 * (1 + Roles::kQWarps);                // the copies, and the warps
      else if (b == bWeights || b == bOFree) count = 2 * kMathWarps;
      mbar_init(bars + 8 * b, count);
    }
    fence_mbar_init();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*reinterpret_cast<uint32_t*>(sm + S_MISC));
  const uint32_t tmem_o = tmem, tmem_s = tmem + 256;
  pdl_wait();
  SharedWalk walk;
  if (p.planned) walk.start(p.units, p.starts + c);
  else plan_here(p, sm, walk, c, rank);
  if (warp < kMathWarps) {
    math_shared(p, sm, base_s, tmem_s, tmem_o, walk, c, warp, rank);
  } else if (warp < Roles::kQ) {
    if (KVF != 0 && p.kv.page_shift >= 3) produce_codes<KVF>(p, sm, base_s, walk, warp - kMathWarps, rank);
    else produce_role<KVF, TMA>(p, sm, base_s, walk, warp - kMathWarps, rank);
  } else if (warp < Roles::kIssuer) {
    q_role<Roles::kQWarps>(p, sm, base_s, walk, tid - 32 * Roles::kQ, rank);
  } else if (rank == 0) {
    issue_shared(p, base_s, tmem_s, tmem_o, walk);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA's memory goes while the other may use it
  if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Join of a split unit's partials, the formula of csa2_attend_paged's join. A
// thread has one head and 16 dims (a sector of the output; the parts' values lie
// next to each other over the heads). GROUPS 1: a CTA has 64 dims. GROUPS 4:
// it has 16, and its quarters take every fourth part, for the few queries that
// have many parts. What a thread waits for is one round trip for PARTS parts: four,
// or for many queries with two or three parts each two, which leaves room for
// twice the CTAs. Whole calls over 8K common rows, <4, 4>, <1, 4> and <1, 2>: 4
// queries 22.3 and 29.8 us, 8 28.9, 32.8, 39.6, 10 27.8 and 29.0, 12 28.7 and 28.6,
// 16 31.7, 30.7, 34.1, 19 35.6, 33.1, 35.8, 32 45.3, 39.5, 41.2, 38 49.9, 43.9, 44.2, 40
// 52.6, 46.9, 46.5, 64 70.4, 59.8, 58.2; over 2K, 30K and in pairs, fours or without
// common rows the same within 1 us, but that over 500 rows <4, 4> loses from 10 on.
constexpr int kJoinDims = 16;
template <int GROUPS, int PARTS>
__global__ void __launch_bounds__(256, 8 / PARTS) attend_shared_join_kernel(const __grid_constant__ SharedParams p) {
  __shared__ float2 weight[kMaxCtaPairs][kHeads];  // reference and sum, then the weight
  __shared__ float red[2][4][kHeads];
  __shared__ float2 turn[32];
  const int head = threadIdx.x & 63, quarter = threadIdx.x >> 6, rank = (int)blockIdx.z, group = GROUPS == 1 ? 0 : quarter;
  const int d0 = kJoinDims * (GROUPS == 1 ? (int)blockIdx.y * 4 + quarter : (int)blockIdx.y), first_rope = kDim - 2 * p.rp.pairs;
  const bool rope = GROUPS == 1 ? 64 * ((int)blockIdx.y + 1) > first_rope : d0 + kJoinDims > first_rope;  // of the CTA
  const double freq = rope && threadIdx.x < (unsigned)p.rp.pairs ? p.rp.freq[threadIdx.x] : 0.0;
  pdl_wait();
  const int4 jn = p.joins[blockIdx.x];
  const int qi = rank == 0 ? jn.x : jn.y;
  if (jn.z < 0 || qi < 0) return;
  const int n = jn.w - jn.z + 1;
  auto slot = [&](int k) { return shared_slot(jn.z + k, k == 0, rank); };
  const float4* parts = reinterpret_cast<const float4*>(p.part_o) + (int64_t)(d0 / 4) * kHeads + head;
  float4 v[PARTS][kJoinDims / 4];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int u = 0; u < PARTS; ++u) {
      const int k = k0 + u * GROUPS;
#pragma unroll
      for (int i = 0; i < kJoinDims / 4; ++i)
        v[u][i] = k < n ? parts[(slot(k) * (kDim / 4) + i) * kHeads] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  fetch(group);
  const float sk = p.sink != nullptr ? p.sink[head] : -INFINITY, sk2 = sk * 1.4426950408889634f;
  const int64_t t = rope && threadIdx.x < 32 ? p.q_pos[qi] : 0;
  // the largest reference, each quarter over its share of the parts
  float M = -INFINITY;
#pragma unroll 4
  for (int k = quarter; k < n; k += 4) {
    const float2 ml = p.part_ml[slot(k) * kHeads + head];
    weight[k][head] = ml;
    M = fmaxf(M, ml.x);
  }
  red[0][quarter][head] = M;
  if (threadIdx.x < 32 && rope) {
    float cs, sn;
    angle_cs((double)t * freq, cs, sn);
    turn[threadIdx.x] = make_float2(cs, sn);
  }
  __syncthreads();
  M = fmaxf(fmaxf(red[0][0][head], red[0][1][head]), fmaxf(red[0][2][head], red[0][3][head]));
  const bool none = M == -INFINITY;
  M = fmaxf(M, sk2);
  float den = 0.f;
  for (int k = quarter; k < n; k += 4) {
    const float2 ml = weight[k][head];
    const float e = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
    den += e * ml.y;  // 0 times NaN stays
    weight[k][head].x = e;
  }
  red[1][quarter][head] = den;
  __syncthreads();
  den = (red[1][0][head] + red[1][1][head]) + (red[1][2][head] + red[1][3][head]);
  const bool empty = none && den == 0.f;  // no row in any part
  if (!none) den += exp2f(sk2 - M);
  else if (empty) den = 1.f;
  const float inv = empty ? 0.f : 1.f / den;
  if (d0 == 0 && group == 0 && p.lse != nullptr)
    p.lse[(int64_t)qi * kHeads + head] = empty ? sk : (M + log2f(den)) * 0.6931471805599453f;
  float o[kJoinDims];
#pragma unroll
  for (int i = 0; i < kJoinDims; ++i) o[i] = 0.f;
  for (int k0 = group; k0 < n; k0 += PARTS * GROUPS) {
    if (k0 > group) fetch(k0);
#pragma unroll
    for (int u = 0; u < PARTS; ++u) {
      const float e = k0 + u * GROUPS < n ? weight[k0 + u * GROUPS][head].x : 0.f;
#pragma unroll
      for (int i = 0; i < kJoinDims / 4; ++i) {
        o[4 * i] = fmaf(e, v[u][i].x, o[4 * i]);
        o[4 * i + 1] = fmaf(e, v[u][i].y, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(e, v[u][i].z, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(e, v[u][i].w, o[4 * i + 3]);
      }
    }
  }
  if constexpr (GROUPS > 1) {
    float(*acc)[kJoinDims][kHeads] = reinterpret_cast<float(*)[kJoinDims][kHeads]>(&weight[0][0]);
    static_assert(sizeof(float) * (GROUPS - 1) * kJoinDims * kHeads <= sizeof(weight));
    __syncthreads();  // the weights have been read
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < kJoinDims; ++i) acc[group - 1][i][head] = o[i];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 0; g < GROUPS - 1; ++g) {
#pragma unroll
      for (int i = 0; i < kJoinDims; ++i) o[i] += acc[g][i][head];
    }
  }
  uint32_t w[kJoinDims / 2];
#pragma unroll
  for (int i = 0; i < kJoinDims; i += 2) {
    float x0 = o[i] * inv, x1 = o[i + 1] * inv;
    if (d0 + i >= first_rope) {
      const float2 cs = turn[(d0 + i - first_rope) >> 1];
      const float y = x0 * cs.x + x1 * cs.y;
      x1 = x1 * cs.x - x0 * cs.y;
      x0 = y;
    }
    w[i / 2] = pack_bf16(x0, x1);
  }
  uint4* dst = reinterpret_cast<uint4*>(p.out + ((int64_t)qi * kHeads + head) * kDim + d0);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

constexpr size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
}  // namespace

static int attend_shared_pairs(int num_sms) { return std::min(num_sms / 2, kMaxCtaPairs); }

size_t attend_shared_workspace_bytes(int num_sms, int n_query) {
  const size_t pairs = (size_t)attend_shared_pairs(num_sms), slots = 4 * pairs;
  return al256(slots * kHeads * kDim * 4) + al256(slots * kHeads * 8) + al256(pairs * sizeof(SharedStart)) +
         al256(pairs * sizeof(int4)) + al256((size_t)n_query * sizeof(SharedUnit));
}

cudaError_t launch_attend_shared(cudaStream_t st, int num_sms, int kv_fmt, const AttendParams& a, const PagedView& kv,
                                 const int32_t* order, const int32_t* head, const int64_t* shared, void* ws, int* n_launch) {
  SharedParams p{};
  p.pairs = attend_shared_pairs(num_sms);
  const size_t slots = 4 * (size_t)p.pairs;
  uint8_t* w = static_cast<uint8_t*>(ws);
  auto part = [&](size_t bytes) {
    uint8_t* at = w;
    w += al256(bytes);
    return at;
  };
  p.part_o = reinterpret_cast<float*>(part(slots * kHeads * kDim * 4));
  p.part_ml = reinterpret_cast<float2*>(part(slots * kHeads * 8));
  p.starts = reinterpret_cast<SharedStart*>(part(p.pairs * sizeof(SharedStart)));
  p.joins = reinterpret_cast<int4*>(part(p.pairs * sizeof(int4)));
  p.units = reinterpret_cast<SharedUnit*>(part((size_t)a.n_query * sizeof(SharedUnit)));
  p.q = a.q;
  p.q_pos = a.q_pos;
  p.seq_of_q = a.seq_of_q;
  p.order = order;
  p.head = head;
  p.shared = shared;
  p.sink = a.sink;
  p.out = a.out;
  p.lse = a.lse;
  p.flags = a.flags;
  p.kv = kv;
  p.rp = a.rp;
  p.scale_log2 = a.scale_log2;
  p.n_query = a.n_query;
  const int piece = 1 << piece_shift(kv.page_shift);
  const uint64_t q_dims[2] = {(uint64_t)kDim, (uint64_t)kHeads * a.n_query}, q_strides[1] = {2u * kDim};
  const uint32_t q_box[2] = {64u, (uint32_t)kHeads};
  const uint64_t kv_dims[3] = {(uint64_t)kDim, 1ull << kv.page_shift, (uint64_t)kv.n_pages};
  const uint64_t kv_strides[2] = {2u * kDim, (uint64_t)kv.page_stride};
  const uint32_t kv_box[3] = {64u, (uint32_t)piece, 1u};
  cudaError_t e = encode_bf16_map(&p.q_map, 2, a.q, q_dims, q_strides, q_box);
  if (e == cudaSuccess && kv_fmt == 0) e = encode_bf16_map(&p.kv_map, 3, kv.pages, kv_dims, kv_strides, kv_box);
  if (e == cudaSuccess && kv_fmt == 0 && piece == kGroupRows) {
    const uint64_t v_dims[4] = {64u, 1ull << kv.page_shift, (uint64_t)kDim / 64, (uint64_t)kv.n_pages};
    const uint64_t v_strides[3] = {2u * kDim, 128u, (uint64_t)kv.page_stride};
    const uint32_t v_box[4] = {64u, (uint32_t)kGroupRows, 2u, 1u};
    e = encode_bf16_map(&p.v_map, 4, kv.pages, v_dims, v_strides, v_box);
  }
  if (e == cudaSuccess && kv_fmt != 0 && piece >= 8) {
    const uint32_t run = kv_fmt == 1 ? 64u : 32u;
    const uint64_t c_dims[3] = {8u * run, 1ull << kv.page_shift, (uint64_t)kv.n_pages};
    const uint64_t c_strides[2] = {8u * run, (uint64_t)kv.page_stride};
    const uint32_t c_box[3] = {run, (uint32_t)piece, 1u};
    e = encode_byte_map(&p.code_map, 3, kv.pages, c_dims, c_strides, c_box);
  }
  if (e != cudaSuccess) return e;
  p.planned = a.n_query > kPlanHere;  // (then there are as many queries as pairs: kPlanHere is more than those)
  static_assert(kPlanHere >= kMaxCtaPairs);
  if (p.planned) {
    e = launch_ex(attend_shared_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, true, 0, p);
    if (e != cudaSuccess) return e;
  }
#define CSA2_SHARED(F, T)                                                                                               \
  do {                                                                                                                 \
    e = cudaFuncSetAttribute(attend_shared_kernel<F, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSharedSmemBytes); \
    if (e == cudaSuccess)                                                                                              \
      e = launch_ex(attend_shared_kernel<F, T>, dim3(2 * p.pairs), dim3(SharedRoles<T>::kThreads), kSharedSmemBytes, st, true, 0, p); \
  } while (0)
  // (TMA: pieces of at least the 8 rows of a swizzle atom)
  if (kv_fmt == 0 && piece >= 8) CSA2_SHARED(0, true);
  else if (kv_fmt == 0) CSA2_SHARED(0, false);
  else if (kv_fmt == 1) CSA2_SHARED(1, false);
  else CSA2_SHARED(2, false);
#undef CSA2_SHARED
  if (e != cudaSuccess) return e;
  // few queries: many parts a unit, few units to be joined (CTAs without one cost
  // their start, 1.6 ns each). The borders are where the variants meet: 10 to 12
  // queries and 38 to 40 on 76 pairs.
  const unsigned joins = (unsigned)std::min(p.pairs, p.n_query);
  const dim3 by_quarter(joins, kDim / kJoinDims, 2), by_dims(joins, kDim / kJoinDims / 4, 2);
  if (7 * joins <= (unsigned)p.pairs) e = launch_ex(attend_shared_join_kernel<4, 4>, by_quarter, dim3(256), 0, st, true, 0, p);
  else if (2 * joins <= (unsigned)p.pairs) e = launch_ex(attend_shared_join_kernel<1, 4>, by_dims, dim3(256), 0, st, true, 0, p);
  else e = launch_ex(attend_shared_join_kernel<1, 2>, by_dims, dim3(256), 0, st, true, 0, p);
  if (e != cudaSuccess) return e;
  *n_launch += p.planned ? 3 : 2;
  return cudaGetLastError();
}

}  // namespace csa2

// Rotary positions as an operator of its own (csa2_rope), and the append that
// rotates new rows and stores them in a paged cache (csa2_append_paged).
#include <cmath>

#include "launchers.cuh"
#include "paged.cuh"
#include "row_store.cuh"

namespace csa2 {

namespace {

// ---------------------------------------------------------------------------
// csa2_rope: y = amplitude * R(pos f) x on rope_dim channels of every head,
// the others copied. Pair k of the interleaved layout is (o + 2k, o + 2k + 1),
// of the half layout (o + k, o + k + rope_dim / 2); (u, v) -> (u cos - v sin,
// u sin + v cos). Memory-bound: 2 x the elements' bytes. A CTA takes a few
// tokens and some of their heads: it issues its first loads, forms the tokens'
// (cos, sin) once in shared memory while they are under way, and then rotates
// in registers. The angle is pos * (f / 2 pi) modulo one turn, which 64-bit
// integers give exactly where double precision, at two operations a clock and
// SM, costs more than the rotation: 8,191 tokens of 64 heads x 128 in bf16
// take 49 us (5.5 TB/s, 81% of a copy) and took 56 us with double angles,
// 64 us with the table's rows in order (see table_at) and a division a row.
// Left: loads and stores of a CTA alternate; more CTAs an SM, more or fewer
// loads a thread, and more tokens a CTA change nothing or spill.
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256;
constexpr int kRopeTable = 1024;  // (cos, sin) entries a CTA holds: 8 KB
constexpr int kRopeTokens = 32;   // tokens a CTA takes at most

struct RopeArgs {
  const uint8_t* x;
  uint8_t* out;
  const int64_t* pos;
  int64_t x_tok, x_head, o_tok, o_head;  // strides in elements
  int64_t n_tok;
  int32_t n_heads, head_dim;
  int32_t tok_per_cta, heads_per_cta;
  int32_t units_rope, units_pass;  // vector units of a head: rotated ones, then copied ones
  int32_t rope_dim, offset, layout;
  float amplitude;
  uint64_t turns[CSA2_ROPE_MAX_PAIRS];  // a position's turn of pair k, in 2^-64 of a full one
};

// f / 2 pi modulo 1 in units of 2^-64, rounded: the turn that one position
// adds. |f| < 2^32. The 53 bits of f times the first 128 of 1 / 2 pi are exact
// in three words; the cut tail of 1 / 2 pi is below f 2^-64 units.
uint64_t turn_of(double f) {
  using u128 = unsigned __int128;
  int e = 0;
  const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(f), &e), 53);
  e -= 53;                                                // |f| = m 2^e
  const u128 lo = (u128)m * 0x7f09d5f47d4d3770ull;        // 1 / 2 pi = 0x.28be60db9391054a7f09d5f47d4d3770..
  const u128 top = (u128)m * 0x28be60db9391054aull + (uint64_t)(lo >> 64);
  // |f| / 2 pi = (top 2^64 + low word) 2^(e - 128): its units of 2^-64 start at bit -e of top
  const int shift = -e;                                   // 21 and more
  const u128 units = shift > 120 ? 0 : (((top >> (shift - 1)) + 1) >> 1);
  return f < 0 ? (uint64_t)0 - (uint64_t)units : (uint64_t)units;
}

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Place of pair k in a token's table. Threads of neighbouring units read two
// pairs (16 bytes) at once, eight pairs apart: the four 16-byte pieces of a
// group of eight pairs are turned by the group, so that they fall into
// different banks (in order, four of eight threads shared them).
__device__ __forceinline__ int table_at(int k) { return (k & ~7) | ((k ^ ((k >> 3) & 6)) & 7); }

template <typename T, int N, int ALIGN>
struct alignas(ALIGN) Vec {
  T e[N];
};

// VEC elements a unit. A rotated unit of the half layout is two vectors (the
// pairs' first and second members); of the interleaved layout one vector of
// VEC >= 2 elements. HALF: the layout; ALIGN: bytes that every vector's start
// is a multiple of.
template <typename T, int VEC, bool HALF, int ALIGN>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ __align__(16) float2 tab[kRopeTable];
  __shared__ bool live[kRopeTokens];
  using V = Vec<T, VEC, ALIGN>;
  constexpr int kUnroll = HALF ? 2 : 4;  // 64 bytes a thread under way
  const int tid = threadIdx.x;
  const int64_t tok0 = (int64_t)blockIdx.x * a.tok_per_cta;
  const int n_tok = (int)min((int64_t)a.tok_per_cta, a.n_tok - tok0);
  const int h0 = blockIdx.y * a.heads_per_cta;
  const int n_heads = min(a.heads_per_cta, a.n_heads - h0);
  const int units = a.units_rope + a.units_pass;
  const int pairs = a.rope_dim >> 1, off = a.offset;
  const int table_row = (pairs + 7) & ~7;  // a token's entries, whole groups of eight
  // thread = (unit, row of the pass); rows are (token, head)
  const int rows_per_pass = max(1, kRopeThreads / units);
  const int unit0 = tid % units, row0 = tid / units;
  const T* x = reinterpret_cast<const T*>(a.x);
  T* out = reinterpret_cast<T*>(a.out);

  // first element of a unit in its head
  auto channel = [&](int unit) -> int {
    if (unit < a.units_rope) return off + unit * VEC;
    const int p = (unit - a.units_rope) * VEC;  // channel among the copied ones
    if (p < off) return p;
    return p + (HALF ? 2 * pairs : a.units_rope * VEC);
  };
  // a thread's rows: (token, head) pairs rows_per_pass apart
  const int step_tok = rows_per_pass / n_heads, step_head = rows_per_pass - step_tok * n_heads;
  struct Row {
    int tk, h;
  };
  auto next = [&](Row r) {
    r.tk += step_tok;
    r.h += step_head;
    if (r.h >= n_heads) {
      r.h -= n_heads;
      ++r.tk;
    }
    return r;
  };
  auto load = [&](Row r, int ch, bool turn, V& v, V& w) {
    const T* src = x + (tok0 + r.tk) * a.x_tok + (int64_t)(h0 + r.h) * a.x_head + ch;
    if constexpr (sizeof(V) == 16) {
      // x is read once: its lines leave the L2 before out's, which the next
      // reader wants (8,191 tokens of 64 x 128: 51.9 -> 49.2 us)
      *reinterpret_cast<uint4*>(&v) = __ldcs(reinterpret_cast<const uint4*>(src));
      if (HALF && turn) *reinterpret_cast<uint4*>(&w) = __ldcs(reinterpret_cast<const uint4*>(src + pairs));
    } else {
      v = *reinterpret_cast<const V*>(src);
      if (HALF && turn) w = *reinterpret_cast<const V*>(src + pairs);
    }
  };
  auto store = [&](Row r, int unit, int ch, V v, V w) {
    if (!live[r.tk]) return;
    T* dst = out + (tok0 + r.tk) * a.o_tok + (int64_t)(h0 + r.h) * a.o_head + ch;
    if (unit < a.units_rope) {
      const float2* cs = tab + r.tk * table_row;
      if constexpr (HALF) {
#pragma unroll
        for (int e = 0; e < VEC; e += (VEC > 1 ? 2 : 1)) {
          const float4 t = VEC > 1 ? *reinterpret_cast<const float4*>(cs + table_at(unit * VEC + e))
                                   : make_float4(cs[unit].x, cs[unit].y, 0.f, 0.f);
          const float u0 = to_f32(v.e[e]), z0 = to_f32(w.e[e]);
          v.e[e] = from_f32<T>(u0 * t.x - z0 * t.y);
          w.e[e] = from_f32<T>(u0 * t.y + z0 * t.x);
          if constexpr (VEC > 1) {
            const float u1 = to_f32(v.e[e + 1]), z1 = to_f32(w.e[e + 1]);
            v.e[e + 1] = from_f32<T>(u1 * t.z - z1 * t.w);
            w.e[e + 1] = from_f32<T>(u1 * t.w + z1 * t.z);
          }
        }
        *reinterpret_cast<V*>(dst + pairs) = w;
      } else {
#pragma unroll
        for (int e = 0; e + 1 < VEC; e += 2) {
          const int k = (unit * VEC + e) >> 1;
          if (k < pairs) {  // the last unit may reach past the rotated channels
            const float2 t = cs[VEC > 2 ? table_at(k) : k];
            const float u = to_f32(v.e[e]), z = to_f32(v.e[e + 1]);
            v.e[e] = from_f32<T>(u * t.x - z * t.y);
            v.e[e + 1] = from_f32<T>(u * t.y + z * t.x);
          }
        }
      }
    }
    *reinterpret_cast<V*>(dst) = v;
  };

  V v[kUnroll], w[kUnroll];
  const bool active = row0 < rows_per_pass;
  const Row start{row0 / n_heads, row0 % n_heads};
  if (active) {
    Row r = start;
    const int ch = channel(unit0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (r.tk < n_tok) load(r, ch, unit0 < a.units_rope, v[u], w[u]);
      r = next(r);
    }
  }
  for (int i = tid; i < n_tok * pairs; i += kRopeThreads) {
    const int tk = i / pairs, k = i - tk * pairs;
    // pos turns modulo one: exact in 64-bit integers
    const int64_t turn = (int64_t)((uint64_t)a.pos[tok0 + tk] * a.turns[k]);
    float c, s;
    sincospif((float)turn * 0x1p-63f, &s, &c);
    tab[tk * table_row + (VEC > 2 ? table_at(k) : k)] = make_float2(a.amplitude * c, a.amplitude * s);
  }
  if (tid < n_tok) live[tid] = a.pos[tok0 + tid] >= 0;
  __syncthreads();
  if (!active) return;
  for (int unit = unit0; unit < units; unit += kRopeThreads) {
    const int ch = channel(unit);
    const bool turn = unit < a.units_rope;
    Row r = start;
    bool loaded = unit == unit0;
    while (r.tk < n_tok) {
      Row at[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        at[u] = r;
        if (!loaded && r.tk < n_tok) load(r, ch, turn, v[u], w[u]);
        r = next(r);
      }
      loaded = false;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (at[u].tk < n_tok) store(at[u], unit, ch, v[u], w[u]);
    }
  }
}

template <typename T, int VEC, bool HALF, int ALIGN>
cudaError_t launch_rope_t(cudaStream_t st, RopeArgs& a, int num_sms, bool in_place, int* n_launch) {
  const int r = a.rope_dim, D = a.head_dim;
  a.units_rope = HALF ? (r / 2) / VEC : (r + VEC - 1) / VEC;
  // in place the channels that stay need no copy
  a.units_pass = in_place ? 0 : (HALF ? (D - r) / VEC : D / VEC - a.units_rope);
  const int units = a.units_rope + a.units_pass;
  if (units == 0) return cudaSuccess;
  const int pairs = r / 2;
  // about eight units a thread, as many tokens as the table holds; a call of
  // few tokens splits their heads until every SM has two CTAs
  int64_t tt = 8 * kRopeThreads / ((int64_t)a.n_heads * units);
  tt = tt < 1 ? 1 : (tt > kRopeTokens ? kRopeTokens : tt);
  const int table_row = (pairs + 7) & ~7;
  if (pairs > 0 && tt > kRopeTable / table_row) tt = kRopeTable / table_row;
  while (tt > 1 && (a.n_tok + tt - 1) / tt < 2 * num_sms) tt = (tt + 1) / 2;
  const int64_t gx = (a.n_tok + tt - 1) / tt;
  int hpc = a.n_heads;
  while (hpc > 1 && gx * ((a.n_heads + hpc - 1) / hpc) < 2 * num_sms) hpc = (hpc + 1) / 2;
  a.tok_per_cta = (int)tt;
  a.heads_per_cta = hpc;
  if (gx > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)gx, (unsigned)((a.n_heads + hpc - 1) / hpc));
  rope_kernel<T, VEC, HALF, ALIGN><<<grid, kRopeThreads, 0, st>>>(a);
  *n_launch += 1;
  return cudaGetLastError();
}

// The widest unit that every row's start, the rotated range and the head's
// width allow: 16 bytes, else one pair (interleaved, as one access where pairs
// are aligned) or one element of each member (half).
template <typename T>
cudaError_t launch_rope_type(cudaStream_t st, RopeArgs& a, int num_sms, bool in_place, int* n_launch) {
  constexpr int W = 16 / (int)sizeof(T);
  const bool half = a.layout == CSA2_ROPE_HALF;
  auto fits = [&](int v) {
    const int64_t align = (int64_t)v * (int64_t)sizeof(T);
    auto mult = [&](int64_t e) { return e % v == 0; };
    return reinterpret_cast<uintptr_t>(a.x) % align == 0 && reinterpret_cast<uintptr_t>(a.out) % align == 0 &&
           mult(a.x_tok) && mult(a.x_head) && mult(a.o_tok) && mult(a.o_head) && mult(a.head_dim) &&
           mult(a.offset) && (!half || mult(a.rope_dim / 2));
  };
  constexpr int S = (int)sizeof(T);
  if (half)
    return fits(W) ? launch_rope_t<T, W, true, 16>(st, a, num_sms, in_place, n_launch)
                   : launch_rope_t<T, 1, true, S>(st, a, num_sms, in_place, n_launch);
  if (fits(W)) return launch_rope_t<T, W, false, 16>(st, a, num_sms, in_place, n_launch);
  return fits(2) ? launch_rope_t<T, 2, false, 2 * S>(st, a, num_sms, in_place, n_launch)
                 : launch_rope_t<T, 2, false, S>(st, a, num_sms, in_place, n_launch);
}

// ---------------------------------------------------------------------------
// csa2_append_paged: one warp per new row, lane l holding channels 16l ..;
// the row's page is looked up while its channels load, lane k forms the
// (cos, sin) of pair k (one angle a lane) and hands it to the lanes that hold
// the pair: the same double-precision steps as the packed store's, whose bits
// the rows have. Decode is bound by latency; prompts by the six double
// operations of an angle, two a clock and SM: about 14,800 bf16 rows take 12.3 us, 10.2
// without them, of which 4.5 are the bytes. Four rows a warp under one lookup
// (14.3 us) or two (13.8) leave too few warps to hide either.
// ---------------------------------------------------------------------------
template <typename T, int FMT>
__global__ void __launch_bounds__(256) append_paged_kernel(const T* __restrict__ rows, int64_t n_rows, int n_seq,
                                                           const int64_t* __restrict__ tok_off,
                                                           const int64_t* __restrict__ first_pos, const PagedView kv,
                                                           const RopeParams rp, uint32_t* flags) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= n_rows) return;
  float v[16];
  const T* src = rows + row * kDim + lane * 16;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 f = reinterpret_cast<const float4*>(src)[k];
      v[4 * k] = f.x; v[4 * k + 1] = f.y; v[4 * k + 2] = f.z; v[4 * k + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 f = reinterpret_cast<const uint4*>(src)[k];
      const uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        v[8 * k + 2 * u] = bf16lo(w[u]);
        v[8 * k + 2 * u + 1] = bf16hi(w[u]);
      }
    }
  }
  const int b = find_segment(tok_off, n_seq, row);
  const int64_t t0 = tok_off[b];
  if (row < t0 || row >= tok_off[b + 1]) return;  // past the last sequence: left as it was
  const int64_t p = first_pos[b] + (row - t0);
  const int32_t g = p >= 0 ? page_of(kv, b, p) : -1;
  if (g < 0) {
    if (lane == 0) set_flag(flags, CSA2_FLAG_BAD_PAGE);
    return;
  }
  if (rp.pairs > 0) {
    float c = 1.f, s = 0.f;
    if (lane < rp.pairs) rope_cs(rp, lane, p, c, s);
    const int first = kDim - 2 * rp.pairs;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int ch = lane * 16 + 2 * k;
      const int pair = ch >= first ? (ch - first) >> 1 : 0;
      const float pc = __shfl_sync(0xffffffffu, c, pair), ps = __shfl_sync(0xffffffffu, s, pair);
      if (ch >= first) {
        const float x0 = v[2 * k], x1 = v[2 * k + 1];
        v[2 * k] = x0 * pc - x1 * ps;
        v[2 * k + 1] = x0 * ps + x1 * pc;
      }
    }
  }
  const int64_t r = p & ((1 << kv.page_shift) - 1);
  store_row<kDim, FMT>(v, lane, kv.pages + g * kv.page_stride + r * row_code_bytes(kDim, FMT),
                       FMT == 0 ? nullptr : kv.scales + g * kv.scale_stride + r * row_scale_bytes(kDim, FMT));
}

}  // namespace

cudaError_t launch_rope(cudaStream_t st, int num_sms, const csa2_rope_table& tab, int dtype, const void* x, void* out,
                        const int64_t* pos, int64_t n_tok, int n_heads, int head_dim, int64_t x_tok, int64_t x_head,
                        int64_t o_tok, int64_t o_head, bool transpose, bool in_place, int* n_launch) {
  RopeArgs a{};
  a.x = static_cast<const uint8_t*>(x);
  a.out = static_cast<uint8_t*>(out);
  a.pos = pos;
  a.x_tok = x_tok;
  a.x_head = x_head;
  a.o_tok = o_tok;
  a.o_head = o_head;
  a.n_tok = n_tok;
  a.n_heads = n_heads;
  a.head_dim = head_dim;
  a.rope_dim = tab.rope_dim;
  a.offset = tab.offset;
  a.layout = tab.layout;
  a.amplitude = (float)tab.amplitude;
  for (int k = 0; k < tab.rope_dim / 2; ++k) a.turns[k] = turn_of(transpose ? -tab.freq[k] : tab.freq[k]);
  switch (dtype) {
    case CSA2_DTYPE_BF16: return launch_rope_type<__nv_bfloat16>(st, a, num_sms, in_place, n_launch);
    case CSA2_DTYPE_FP16: return launch_rope_type<__half>(st, a, num_sms, in_place, n_launch);
    case CSA2_DTYPE_FP32: return launch_rope_type<float>(st, a, num_sms, in_place, n_launch);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_append_paged(cudaStream_t st, int dtype, const void* rows, int64_t n_rows, int n_seq,
                                const int64_t* tok_off, const int64_t* first_pos, const PagedView& kv, int kv_fmt,
                                const RopeParams& rp, uint32_t* flags) {
  if ((n_rows + 7) / 8 > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((n_rows + 7) / 8));
#define CSA2_APPEND(T, F) \
  append_paged_kernel<T, F><<<grid, 256, 0, st>>>(static_cast<const T*>(rows), n_rows, n_seq, tok_off, first_pos, kv, rp, flags)
#define CSA2_APPEND_F(T)                \
  do {                                  \
    if (kv_fmt == 0) CSA2_APPEND(T, 0); \
    else if (kv_fmt == 1) CSA2_APPEND(T, 1); \
    else CSA2_APPEND(T, 2);             \
  } while (0)
  if (dtype == CSA2_DTYPE_FP32) CSA2_APPEND_F(float);
  else CSA2_APPEND_F(uint16_t);
#undef CSA2_APPEND_F
#undef CSA2_APPEND
  return cudaGetLastError();
}

}  // namespace csa2

// Pieces shared by the tile kernels over paged caches: bounded waits and
// warp-uniform issue of barrier, TMA and tensor-core instructions, prefetches,
// and the conversion of fp8 and fp4 rows to bf16.
#pragma once
#include <cuda.h>

#include "common.cuh"

namespace csa2 {

// Bounded wait on an mbarrier phase: 100,000 suspensions of up to 20 us, then
// CSA2_FLAG_WAIT_TIMEOUT and false. (mbar_wait with its clock is 40
// instructions at each of a dozen places.)
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

__device__ __forceinline__ void prefetch_l2_line(const void* ptr) { asm volatile("prefetch.global.L2 [%0];" ::"l"(ptr)); }
__device__ __forceinline__ void prefetch_l2(const void* ptr, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ptr), "r"(bytes) : "memory");
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

// a / b of values >= 0: 32-bit where they fit (a 64-bit division is several
// hundred cycles, before any row is asked for)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((uint64_t)(a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// 16 zero bytes into shared memory if hit != 0, without a branch
__device__ __forceinline__ void zero16_if(uint32_t hit, uint32_t dst) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %0, 0;\n@p st.shared.v4.u32 [%1], {%2, %2, %2, %2};\n}" ::"r"(hit), "r"(dst), "r"(0u)
               : "memory");
}

}  // namespace csa2

// One row of a cache stored by a warp, lane l holding its channels
// l * DIM / 32 .. in fp32: bf16, fp8 (e4m3 + ue8m0 per 32 channels), fp4
// (E2M1 + e4m3 per 16) or mxfp4 (E2M1 + ue8m0 per 32).
#pragma once
#include "common.cuh"

namespace csa2 {

__host__ __device__ constexpr int row_code_bytes(int dim, int fmt) {
  return fmt == 0 ? 2 * dim : (fmt == 1 ? dim : dim / 2);
}
__host__ __device__ constexpr int row_scale_bytes(int dim, int fmt) {
  return fmt == 0 ? 0 : (fmt == 2 ? dim / 16 : dim / 32);
}

// FMT: 0 bf16, 1 fp8, 2 fp4, 3 mxfp4; out / out_scale: this row's codes and scales
template <int DIM, int FMT>
__device__ __forceinline__ void store_row(const float (&v)[DIM / 32], int lane, uint8_t* __restrict__ out,
                                          uint8_t* __restrict__ out_scale) {
  constexpr int E = DIM / 32;  // channels per lane (4 or 16)
  if constexpr (FMT == 0) {
    uint32_t w[E / 2];
#pragma unroll
    for (int k = 0; k < E / 2; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
    uint2* dst = reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(out) + lane * E);
#pragma unroll
    for (int k = 0; k < E / 4; ++k) dst[k] = make_uint2(w[2 * k], w[2 * k + 1]);
  } else if constexpr (FMT == 1) {
    constexpr int LPB = 32 / E;  // lanes per 32-channel block
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) amax = fmaxf(amax, fabsf(v[k]));
#pragma unroll
    for (int o = 1; o < LPB; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const uint32_t eb = fp8_scale_byte(amax);
    const int sh = 127 - (int)eb;  // x / 2^(eb-127), exact
    uint8_t* dst = out + lane * E;
#pragma unroll
    for (int k = 0; k < E; k += 4) {
      uint32_t word = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) word |= (uint32_t)f32_to_e4m3(ldexpf(v[k + u], sh)) << (8 * u);
      *reinterpret_cast<uint32_t*>(dst + k) = word;
    }
    if ((lane % LPB) == 0) out_scale[lane / LPB] = (uint8_t)eb;
  } else {
    constexpr int BLK = (FMT == 2) ? 16 : 32;  // channels per scale
    constexpr int LPB = (BLK / E) > 0 ? BLK / E : 1;  // lanes per block
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < E; ++k) amax = fmaxf(amax, fabsf(v[k]));
#pragma unroll
    for (int o = 1; o < LPB; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float sc;
    uint32_t sbyte;
    if constexpr (FMT == 2) {
      sbyte = fp4_scale_e4m3(amax);
      sc = e4m3_value(sbyte);
    } else {
      sbyte = mxfp4_scale_byte(amax);
      sc = ue8m0_value(sbyte);
    }
    uint8_t* dst = out + lane * (E / 2);
#pragma unroll
    for (int k = 0; k < E; k += 2) dst[k / 2] = (uint8_t)(e2m1_code(v[k], sc) | (e2m1_code(v[k + 1], sc) << 4));
    if ((lane % LPB) == 0) out_scale[lane / LPB] = (uint8_t)sbyte;
  }
}

}  // namespace csa2

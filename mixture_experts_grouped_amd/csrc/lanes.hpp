// lanes.hpp -- reductions over the 16 lanes of a DPP row and small numeric
// helpers shared by the router, the optimisers and the 8- and 4-bit kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "engine.hpp"

namespace moelora {

// The value of the lane N places on in the same row of 16 lanes (DPP row
// rotate: one VALU operand modifier, no LDS).
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, true);
}
template <int N>
__device__ __forceinline__ float row_ror(float v) {
  return __uint_as_float(row_ror<N>(__float_as_uint(v)));
}

// All 16 lanes get the result; sums pair the same values in every lane, so
// the lanes agree bit for bit.
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, row_ror<8>(v));
  v = max(v, row_ror<4>(v));
  v = max(v, row_ror<2>(v));
  return max(v, row_ror<1>(v));
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  v = min(v, row_ror<8>(v));
  v = min(v, row_ror<4>(v));
  v = min(v, row_ror<2>(v));
  return min(v, row_ror<1>(v));
}
__device__ __forceinline__ float row_sum(float v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  return v + row_ror<1>(v);
}

// Sums over the wave, in every lane (whole waves only).
__device__ __forceinline__ int wave_sum(int v) {
  v += (int)row_ror<8>((uint32_t)v);
  v += (int)row_ror<4>((uint32_t)v);
  v += (int)row_ror<2>((uint32_t)v);
  v += (int)row_ror<1>((uint32_t)v);
  return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
         __builtin_amdgcn_readlane(v, 48);
}
template <int N>
__device__ __forceinline__ double row_ror(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)row_ror<N>((uint32_t)(b >> 32)) << 32 | row_ror<N>((uint32_t)b));
}
__device__ __forceinline__ double readlane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane), lo = (uint32_t)__builtin_amdgcn_readlane((int)b, lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_sum(double v) {
  v += row_ror<8>(v);
  v += row_ror<4>(v);
  v += row_ror<2>(v);
  v += row_ror<1>(v);
  return (readlane(v, 0) + readlane(v, 16)) + (readlane(v, 32) + readlane(v, 48));
}

// Magnitude bits of an fp32 value: as integers they order like the
// magnitudes, infinity above every finite value and NaN above infinity, so
// an integer maximum keeps a NaN that a floating one would drop.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Eight bf16 values of a 16-byte chunk.
__device__ __forceinline__ void widen8(u32x4 w, float (&v)[8]) {
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    v[2 * c] = bf2f(w[c] & 0xffffu);
    v[2 * c + 1] = bf2f(w[c] >> 16);
  }
}

// The normal distribution function to fp32's relative precision: a block in its
// lower tail is scaled by its own largest value, which norm_cdf's absolute error
// of 1e-7 would shift (1 % at -8).  Phi(g) = 1/2 exp(-z^2) f(z) at z = -g / sqrt 2
// >= 0, with f(z) = exp(z^2) erfc(z) = t P(t), t = 1 / (1 + 0.46 z): P of degree 7 is
// fitted for the smallest largest relative error over all z, 6.8e-7 (8.7e-7
// evaluated in fp32); here halved.  98,304 x 2048, same inputs: 200 us, 195 with
// norm_cdf, 302 with the math library's erfcf.
__device__ __forceinline__ float norm_cdf_rel(float g) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.46f * 0.70710678118654752f, fabsf(g), 1.0f));
  float q = 0.0338571894f;
  q = fmaf(q, t, -0.113314702f);
  q = fmaf(q, t, 0.084595587f);
  q = fmaf(q, t, 0.0263052463f);
  q = fmaf(q, t, 0.093423918f);
  q = fmaf(q, t, 0.115590938f);
  q = fmaf(q, t, 0.129778633f);
  q = fmaf(q, t, 0.12976353f);
  const float tail = q * t * __builtin_amdgcn_exp2f(-0.72134752044448170f * g * g);  // log2(e) / 2
  return g < 0.0f ? tail : 1.0f - tail;
}

}  // namespace moelora

// Rotary positions on the device: cos and sin of a pair's angle at a position.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace exq {

// gain * (cos, sin) of 2 pi frac(pos * step / 2^64), rounded once to fp32.
//
// pos * step wraps in 64-bit integers, which drops whole turns exactly; the
// turn is split into the nearest quarter q and a remainder |r| <= 1/8 turn,
// and cos, sin of x = 2 pi r, |x| <= pi/4, come from their Taylor polynomials
// in fp64: up to x^13 for sin and x^14 for cos, whose first dropped terms are
// at most 2^-44.9 and 2^-49 of the result. fp64 because the rounding to fp32 then
// agrees with the correctly rounded one but for about one angle in 2^20: the
// rotated values, and with them the KV codes, are the same bits wherever they
// are computed. The kernels evaluate each (token, pair) once per block, in
// shared memory: GB300 has few fp64 lanes.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t step, int32_t pos, double gain, bool grad) {
  const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
  const uint64_t q = (turn + (1ull << 61)) >> 62;
  const double r = static_cast<double>(static_cast<int64_t>(turn - (q << 62)));
  const double x = r * (6.283185307179586476925 * 0x1p-64);
  const double t = x * x;
  double s = 1.0 / 6227020800.0;
  s = fma(s, t, -1.0 / 39916800.0);
  s = fma(s, t, 1.0 / 362880.0);
  s = fma(s, t, -1.0 / 5040.0);
  s = fma(s, t, 1.0 / 120.0);
  s = fma(s, t, -1.0 / 6.0);
  s = fma(s * t, x, x);
  double c = -1.0 / 87178291200.0;
  c = fma(c, t, 1.0 / 479001600.0);
  c = fma(c, t, -1.0 / 3628800.0);
  c = fma(c, t, 1.0 / 40320.0);
  c = fma(c, t, -1.0 / 720.0);
  c = fma(c, t, 1.0 / 24.0);
  c = fma(c, t, -0.5);
  c = fma(c, t, 1.0);
  // quarter q: (c, s) -> (c, s), (-s, c), (-c, -s), (s, -c)
  double co = (q & 1) ? s : c, si = (q & 1) ? c : s;
  if (q == 1 || q == 2) co = -co;
  if (q & 2) si = -si;
  if (grad) si = -si;
  return make_float2(static_cast<float>(co * gain), static_cast<float>(si * gain));
}

__device__ __forceinline__ float half_bits_to_float(uint32_t h) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
}
__device__ __forceinline__ uint32_t float_to_half_bits(float f) {
  return __half_as_ushort(__float2half_rn(f));
}

// the two values of a pair: products and sums each rounded (no contraction)
__device__ __forceinline__ float rope_first(float x1, float x2, float2 cs) {
  return __fsub_rn(__fmul_rn(x1, cs.x), __fmul_rn(x2, cs.y));
}
__device__ __forceinline__ float rope_second(float x1, float x2, float2 cs) {
  return __fadd_rn(__fmul_rn(x2, cs.x), __fmul_rn(x1, cs.y));
}

}  // namespace exq

// Scales and codes of the 8-bit formats, for the kernels that make operands of the FP8 product.
#pragma once
#include <cuda_fp8.h>

#include "dense.h"

namespace moe {

// A block's scale is its largest magnitude over the largest code (448 or 57344); 1 for a block of
// zeros, at least 2^-126 so that it is a normal number, and with pow2 rounded up to a power of two.  A
// code is the quotient x / scale rounded to nearest even.  (A division for each value made the kernel
// arithmetic-bound: 18.9 us for 4096 x 4096 bf16.)  With the scale's reciprocal r, correctly rounded, q = x r is
// off by a last place at most, its remainder q s - x is exact in one multiply-add, and q - r (q s - x) is the
// correctly rounded quotient, with the sign of a zero (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990); of values below 2^-100, whose remainders may lie below f32's range, q
// may stay as it is.  4096 x 4096 bf16 takes 12.3 us, 11.9 with q alone, which gave 3 to 6 of 10^4 bf16 values
// another code.  The magnitudes are compared as integers, so that a NaN counts as the largest and makes the
// scale NaN.

__device__ __forceinline__ float block_scale(uint32_t amax, bool e5m2, bool pow2) {
  if (amax == 0u) return 1.f;
  float s = __fdiv_rn(__uint_as_float(amax), e5m2 ? 57344.f : 448.f);
  if (s < 1.17549435e-38f) s = 1.17549435e-38f;
  const uint32_t u = __float_as_uint(s);
  if (pow2 && (u & 0x7FFFFFu) && u < 0x7F800000u) s = __uint_as_float((u & 0x7F800000u) + 0x800000u);
  return s;
}

// The same with the format known at compile time and, for magnitudes of 2^-90 to infinity, the quotient by the largest
// code from its reciprocal (as `quotient` below): a division's instructions are a tenth of what a row's values take.
template <bool E5M2>
__device__ __forceinline__ float block_scale(uint32_t amax, bool pow2) {
  constexpr float kMost = E5M2 ? 57344.f : 448.f, kInverse = 1.f / kMost;
  if (amax - 0x12800000u >= 0x6D000000u) return block_scale(amax, E5M2, pow2);
  const float x = __uint_as_float(amax), q = x * kInverse;
  const float s = fmaf(fmaf(q, kMost, -x), -kInverse, q);
  const uint32_t u = __float_as_uint(s);
  return pow2 && u & 0x7FFFFFu ? __uint_as_float((u & 0x7F800000u) + 0x800000u) : s;
}

struct Divisor {
  float r, s;
};
// (an infinite scale: every finite value's quotient is 0)
__device__ __forceinline__ Divisor divisor(float scale) {
  return Divisor{__frcp_rn(scale), __float_as_uint(scale) == 0x7F800000u ? 0.f : scale};
}
// x over the scale in f32, rounded to nearest even
__device__ __forceinline__ float quotient(float x, const Divisor &d) {
  const float q = x * d.r;
  return fmaf(fmaf(q, d.s, -x), -d.r, q);
}
__device__ __forceinline__ uint32_t codes2(float a, float b, const Divisor &d, bool e5m2) {
  const float2 q = __fmul2_rn(make_float2(a, b), make_float2(d.r, d.r));
  const float2 rest = __ffma2_rn(q, make_float2(d.s, d.s), make_float2(-a, -b));
  return __nv_cvt_float2_to_fp8x2(__ffma2_rn(rest, make_float2(-d.r, -d.r), q), __NV_SATFINITE,
                                  e5m2 ? __NV_E5M2 : __NV_E4M3);
}
__device__ __forceinline__ uint32_t codes4(const float *v, const Divisor &d, bool e5m2) {
  return codes2(v[0], v[1], d, e5m2) | codes2(v[2], v[3], d, e5m2) << 16;
}

template <bool E5M2>
__device__ __forceinline__ uint32_t codes4(const float *v, const Divisor &d) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = make_float2(v[2 * i], v[2 * i + 1]), q = __fmul2_rn(x, make_float2(d.r, d.r));
    const float2 rest = __ffma2_rn(q, make_float2(d.s, d.s), make_float2(-x.x, -x.y));
    o[i] = __nv_cvt_float2_to_fp8x2(__ffma2_rn(rest, make_float2(-d.r, -d.r), q), __NV_SATFINITE, E5M2 ? __NV_E5M2 : __NV_E4M3);
  }
  return o[0] | o[1] << 16;
}
__device__ __forceinline__ uint32_t largest(const float (&v)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return m;
}

}  // namespace moe

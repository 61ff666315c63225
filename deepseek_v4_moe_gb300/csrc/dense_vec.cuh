// Loads and stores of eight values of a row, as floats, for the dense sublayer's streaming kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "dense.h"

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// two floats rounded to a pair of T, the first in the low half
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const T x = from_f32<T>(a), y = from_f32<T>(b);
  return (uint32_t)*reinterpret_cast<const uint16_t *>(&x) | (uint32_t)*reinterpret_cast<const uint16_t *>(&y) << 16;
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b, const __nv_bfloat16 *) {
  a = bf_lo(w);
  b = bf_hi(w);
}
__device__ __forceinline__ void unpack2(uint32_t w, float &a, float &b, const __half *) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
  a = f.x;
  b = f.y;
}

// Eight values of one row that belong to thread t of a group of `n` threads.  VEC: columns 8t .. 8t+7
// as one access (the row aligned to eight values, hidden a multiple of 8).  Otherwise columns t, t + n,
// t + 2n, ...: single accesses that neighbouring threads make side by side.  Columns from `hidden`
// on read as zero and are not written.
template <typename T, bool VEC>
struct Eight {
  T v[8];
  __device__ __forceinline__ void load(const T *row, int t, int n, int hidden) {
    const T *q = row + t;
    if (7 * n + t < hidden) {  // most threads' columns all exist
#pragma unroll
      for (int e = 0; e < 8; ++e, q += n) v[e] = *q;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = e * n + t;
        v[e] = c < hidden ? row[c] : from_f32<T>(0.f);
      }
    }
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = to_f32(v[e]);
  }
  static __device__ __forceinline__ void store(T *row, int t, int n, int hidden, const float (&o)[8]) {
    T *q = row + t;
    if (7 * n + t < hidden) {
#pragma unroll
      for (int e = 0; e < 8; ++e, q += n) *q = from_f32<T>(o[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = e * n + t;
        if (c < hidden) row[c] = from_f32<T>(o[e]);
      }
    }
  }
};

template <typename T>
struct Eight<T, true> {
  uint4 w;
  __device__ __forceinline__ void load(const T *row, int t, int, int hidden) {
    w = 8 * t < hidden ? *reinterpret_cast<const uint4 *>(row + 8 * t) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    const T *tag = nullptr;
    unpack2(w.x, o[0], o[1], tag);
    unpack2(w.y, o[2], o[3], tag);
    unpack2(w.z, o[4], o[5], tag);
    unpack2(w.w, o[6], o[7], tag);
  }
  static __device__ __forceinline__ void store(T *row, int t, int, int hidden, const float (&o)[8]) {
    if (8 * t < hidden)
      *reinterpret_cast<uint4 *>(row + 8 * t) =
          make_uint4(pack2<T>(o[0], o[1]), pack2<T>(o[2], o[3]), pack2<T>(o[4], o[5]), pack2<T>(o[6], o[7]));
  }
};

// f32: one 32-byte access (the row 32-byte aligned); two of 16 bytes each would use half of every sector
// they touch
template <>
struct Eight<float, true> {
  float v[8];
  __device__ __forceinline__ void load(const float *row, int t, int, int hidden) {
    if (8 * t < hidden) {
      asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                   : "l"(row + 8 * t));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = v[e];
  }
  static __device__ __forceinline__ void store(float *row, int t, int, int hidden, const float (&o)[8]) {
    if (8 * t < hidden)
      asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(row + 8 * t), "f"(o[0]), "f"(o[1]),
                   "f"(o[2]), "f"(o[3]), "f"(o[4]), "f"(o[5]), "f"(o[6]), "f"(o[7])
                   : "memory");
  }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_eight(const T *row, int t, int n, int hidden, float (&o)[8]) {
  Eight<T, VEC> e;
  e.load(row, t, n, hidden);
  e.get(o);
}

// A block's sum is multiplied by its two scales a and b.  Their product serves where it is a normal f32 value
// (or 0, as one of them is); elsewhere it has lost bits, or is 0 or infinite, where the sum times both need not
// be.  Then the sum is multiplied by one after the other, first by the one that leads away from the end of the
// range at which the product lies: no step is less exact than the result.
__device__ __forceinline__ bool normal_f32(float x) {
  return (__float_as_uint(x) & 0x7FFFFFFFu) - 0x00800000u < 0x7F000000u;
}
__device__ __forceinline__ bool scales_multiply(float a, float b, float product) {
  return normal_f32(product) || a == 0.f || b == 0.f;
}
struct ScalePair {
  float first, then;
};
__device__ __forceinline__ ScalePair scales_apart(float a, float b) {
  const float product = a * b;
  if (scales_multiply(a, b, product)) return ScalePair{1.f, product};
  return (fabsf(a) < fabsf(b)) == (fabsf(product) > 1.f) ? ScalePair{a, b} : ScalePair{b, a};
}

// 1 / (1 + exp(-x)) by the approximate base-2 exponential and reciprocal: a few units of 2^-22, and |x| 2^-23
// more where it is small, as the exponent's rounding counts (2^-17 at -80); well below the 16-bit types that what is
// made of it is rounded to; 0 and 1 far out, where exp(-x) overflows or vanishes.  (With subnormals, which change nothing here, each takes several instructions more.)
__device__ __forceinline__ float fast_sigmoid(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}

// act(g) and, for the backward pass, its derivative.  The tanh form of gelu is g * sigmoid(2 z) with
// z = sqrt(2 / pi) (g + 0.044715 g^3), as (1 + tanh(z)) / 2 = sigmoid(2 z).
constexpr float kGelu2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
__device__ __forceinline__ float act_value(int act, float g) {
  return g * fast_sigmoid(act == kSilu ? g : kGelu2 * fmaf(0.044715f * g * g, g, g));
}
__device__ __forceinline__ void act_both(int act, float g, float &a, float &da) {
  const float s = fast_sigmoid(act == kSilu ? g : kGelu2 * fmaf(0.044715f * g * g, g, g));
  // (finite: past 4e19, where its square leaves f32, what it is multiplied by is 0)
  const float slope = act == kSilu ? 1.f : fminf(kGelu2 * fmaf(3.f * 0.044715f * g, g, 1.f), 3e38f);
  a = g * s;
  da = fmaf(a * (1.f - s), slope, s);
}

}  // namespace moe

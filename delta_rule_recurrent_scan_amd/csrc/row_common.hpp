// Device helpers of the row-wise kernels (short convolution, norms): groups
// of 8 consecutive elements per thread, as one 16-byte (bf16) or two 16-byte
// (fp32) accesses where the row is aligned, else element by element.
#pragma once

#include "device_common.hpp"

namespace osdn {

// n valid elements (n >= 8: all) of 8 at p into v; the rest are zero.
template <bool ALN>
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[8]) {
  if constexpr (ALN) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
template <bool ALN>
__device__ __forceinline__ void load8(const __bf16* p, int n, float (&v)[8]) {
  if constexpr (ALN) {
    const bf16x8 a = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)a[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? (float)p[i] : 0.f;
  }
}
template <bool ALN>
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if constexpr (ALN) {
    f32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) { a[i] = v[i]; b[i] = v[4 + i]; }
    *reinterpret_cast<f32x4*>(p) = a;
    *reinterpret_cast<f32x4*>(p + 4) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
template <bool ALN>
__device__ __forceinline__ void store8(__bf16* p, int n, const float (&v)[8]) {
  if constexpr (ALN) {
    bf16x8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (__bf16)v[i];
    *reinterpret_cast<bf16x8*>(p) = a;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (__bf16)v[i];
  }
}

// Sum over aligned groups of L lanes, L a run-time 4, 8 or 16 (the lanes of a
// 32-, 64- or 128-element head).
__device__ __forceinline__ float head_sum(float x, int L) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  if (L >= 8) x += dpp_f<0x141>(x);
  if (L >= 16) x += dpp_f<0x140>(x);
  return x;
}

// 1 / (1 + e^-x) through the hardware exp2 and reciprocal (1 ulp each): for
// x -> -inf e^-x overflows to inf and the result is 0, never NaN.
__device__ __forceinline__ float sigmoid_f(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}

}  // namespace osdn

// Device helpers of the row-wise kernels (short convolution, norms): groups
// of consecutive elements per thread.
#pragma once

#include "device_common.hpp"
#include "pack_common.hpp"

namespace osdn {

// V (4 or 8) consecutive elements as they lie in memory: 16 bytes or less a
// lane in one or two accesses. Rows that start off 16 bytes use the same
// accesses (global memory takes any alignment); a row's ragged end goes
// element by element.
template <typename T, int V>
struct Raw {
  static constexpr int W = V * (int)sizeof(T) / 4;  // 32-bit words
  unsigned u[W];
  // n valid elements (n >= V: all); the rest are zero
  template <bool ALN>
  __device__ __forceinline__ void load(const T* p, int n) {
    if (ALN || n >= V) {
      __builtin_memcpy(u, ALN ? __builtin_assume_aligned(p, V * sizeof(T) < 16 ? V * sizeof(T)
                                                                                : 16)
                              : p,
                       sizeof(u));
    } else {
      T t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] = i < n ? p[i] : from_f32<T>(0.f);
      __builtin_memcpy(u, t, sizeof(u));
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < W; ++i) u[i] = 0;
  }
  __device__ __forceinline__ void widen(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(u[i]);
      } else {
        v[i] = __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
      }
    }
  }
  template <bool ALN>
  __device__ __forceinline__ void store(T* p, int n) const {
    if (ALN || n >= V) {
      __builtin_memcpy(ALN ? __builtin_assume_aligned(p, V * sizeof(T) < 16 ? V * sizeof(T) : 16)
                           : p,
                       u, sizeof(u));
    } else {
      T t[V];
      __builtin_memcpy(t, u, sizeof(u));
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) p[i] = t[i];
    }
  }
  __device__ __forceinline__ void narrow(const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    }
  }
};

template <bool ALN, int V, typename T>
__device__ __forceinline__ void load_v(const T* p, int n, float (&v)[V]) {
  Raw<T, V> r;
  r.template load<ALN>(p, n);
  r.widen(v);
}
template <bool ALN, int V, typename T>
__device__ __forceinline__ void store_v(T* p, int n, const float (&v)[V]) {
  Raw<T, V> r;
  r.narrow(v);
  r.template store<ALN>(p, n);
}

// Sum over aligned groups of L lanes, L a run-time 4, 8, 16 or 32 (the lanes of
// a 32-, 64- or 128-element head).
__device__ __forceinline__ float head_sum(float x, int L) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  if (L >= 8) x += dpp_f<0x141>(x);
  if (L >= 16) x += dpp_f<0x140>(x);
  if (L >= 32) x = add_swap16(x);
  return x;
}

// 1 / (1 + e^-x) through the hardware exp2 and reciprocal (1 ulp each): for
// x -> -inf e^-x overflows to inf and the result is 0, never NaN.
__device__ __forceinline__ float sigmoid_f(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}

}  // namespace osdn

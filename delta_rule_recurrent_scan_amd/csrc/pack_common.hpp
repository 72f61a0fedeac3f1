// bf16 pairs in 32-bit words.
#pragma once

#include "device_common.hpp"

namespace osdn {

// Two values rounded to bf16 by one packed conversion, and back.
__device__ __forceinline__ unsigned pack_bf16(float x, float y) {
  typedef __attribute__((ext_vector_type(2))) float f32x2;
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  return __builtin_bit_cast(unsigned, __builtin_convertvector((f32x2{x, y}), bf16x2));
}
__device__ __forceinline__ float low_bf16(unsigned u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high_bf16(unsigned u) {
  return __uint_as_float(u & 0xffff0000u);
}

}  // namespace osdn

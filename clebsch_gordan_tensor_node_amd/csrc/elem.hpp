// Element types of the training operators: 32-bit float, bfloat16 and IEEE half, all
// computed with in 32 bits and rounded to nearest (ties to even) where they are stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace cgtp {

struct Bf16 {
  __bf16 v;
};
struct F16 {
  _Float16 v;
};

__device__ inline float to_f32(float v) { return v; }
__device__ inline float to_f32(Bf16 v) { return float(v.v); }
__device__ inline float to_f32(F16 v) { return float(v.v); }

template <typename T>
__device__ inline T from_f32(float v);
template <>
__device__ inline float from_f32<float>(float v) {
  return v;
}
template <>
__device__ inline Bf16 from_f32<Bf16>(float v) {
  return Bf16{__bf16(v)};
}
template <>
__device__ inline F16 from_f32<F16>(float v) {
  return F16{_Float16(v)};
}

// Element i of an array that is fp32 or, where f32 is 0, of type T.
template <typename T>
__device__ inline float load_either(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : to_f32(static_cast<const T*>(p)[i]);
}
template <typename T>
__device__ inline void store_either(void* p, int f32, int64_t i, float v) {
  if (f32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<T*>(p)[i] = from_f32<T>(v);
}

}  // namespace cgtp

// Vectors of up to 16 bytes at any element's address, and sums over neighbouring lanes, as
// the training operators' kernels use them.
#pragma once

#include "elem.hpp"

namespace cgtp {

constexpr int kWave = 64;

template <typename T, int V>
struct Vec {
  typedef uint32_t Bits __attribute__((ext_vector_type(sizeof(T) * V / 4), aligned(sizeof(T)), may_alias));
  T v[V];
};
template <>
struct Vec<Bf16, 1> {
  typedef uint16_t Bits __attribute__((may_alias));
  Bf16 v[1];
};
template <>
struct Vec<F16, 1> {
  typedef uint16_t Bits __attribute__((may_alias));
  F16 v[1];
};
// 16 bytes (or one element) at any element's address.  Stream: the access does not keep
// the line in the caches.
template <bool Stream, typename T, int V>
__device__ inline Vec<T, V> load_vec(const T* p) {
  typedef typename Vec<T, V>::Bits Bits;
  const Bits* b = reinterpret_cast<const Bits*>(p);
  return __builtin_bit_cast(Vec<T, V>, Stream ? __builtin_nontemporal_load(b) : *b);
}
template <bool Stream, typename T, int V>
__device__ inline void store_vec(T* p, const Vec<T, V>& r) {
  typedef typename Vec<T, V>::Bits Bits;
  Bits* b = reinterpret_cast<Bits*>(p);
  if constexpr (Stream)
    __builtin_nontemporal_store(__builtin_bit_cast(Bits, r), b);
  else
    *b = __builtin_bit_cast(Bits, r);
}

template <int Ctrl>
__device__ inline float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), Ctrl, 0xf, 0xf, true));
}
// Sum over G neighbouring lanes (4 to 64), to each of them.
template <int G>
__device__ inline float lanes_sum(float v) {
  v += dpp<0xB1>(v);                          // quad_perm 1 0 3 2
  v += dpp<0x4E>(v);                          // quad_perm 2 3 0 1
  if constexpr (G >= 8) v += dpp<0x141>(v);   // row_half_mirror
  if constexpr (G >= 16) v += dpp<0x140>(v);  // row_mirror
  if constexpr (G >= 32) v += __shfl_xor(v, 16);
  if constexpr (G >= 64) v += __shfl_xor(v, 32);
  return v;
}

}  // namespace cgtp

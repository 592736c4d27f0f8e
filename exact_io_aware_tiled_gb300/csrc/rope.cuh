// rope.cuh -- the rotation's angle and the vector moves of a row, shared by the
// kernels that rotate by position (rope.cu, norm_rope.cu).
#pragma once
#include <cstring>
#include <type_traits>

#include "common.cuh"

namespace fa {
namespace {

// V consecutive elements, moved as one load or store.
template <typename T, int V> struct __align__(sizeof(T) * V) RVec { T e[V]; };

template <typename T, int V> __device__ __forceinline__ void unpack(const RVec<T, V>& v, float (&f)[V]) {
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = v.e[i];
  } else if constexpr (V == 1) {
    f[0] = Cvt<T>::to_f(v.e[0]);
  } else {
    uint32_t w[V / 2];
    memcpy(w, &v, sizeof(w));
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = Cvt<T>::lo(w[i]);
      f[2 * i + 1] = Cvt<T>::hi(w[i]);
    }
  }
}
template <typename T, int V> __device__ __forceinline__ RVec<T, V> pack(const float (&f)[V]) {
  RVec<T, V> v;
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < V; ++i) v.e[i] = f[i];
  } else if constexpr (V == 1) {
    v.e[0] = Cvt<T>::from_f(f[0]);
  } else {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = Cvt<T>::pack(f[2 * i], f[2 * i + 1]);
    memcpy(&v, w, sizeof(w));
  }
  return v;
}

// The turn f / 2 pi as a 64-bit binary fraction (whole turns dropped).
__device__ __forceinline__ unsigned long long turns_of(double f) {
  double t = f * 0.15915494309189533577;                    // 1 / (2 pi)
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}

// m cos and +-m sin of the angle p f, F the turn of f
__device__ __forceinline__ void turn(long long p, unsigned long long F, float m, float sm, float& c, float& s) {
  const long long frac = (long long)((unsigned long long)p * F);
  sincospif(__ll2float_rn(frac) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
  c *= m;
  s *= sm;
}

}  // namespace
}  // namespace fa

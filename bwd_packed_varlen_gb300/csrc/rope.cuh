// What the kernels that turn queries and keys share: angles, and groups of 16-bit elements.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "sm103_ptx.cuh"

namespace teattn {

// n / d with inv = ceil(2^32 / d), exact for n d < 2^32.
__device__ __forceinline__ int div_by(int n, uint32_t inv, int d) {
  return d == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), inv));
}

// The fraction of a turn per position of a frequency w, as a 64-bit fixed-point number.
__device__ __forceinline__ unsigned long long turn_per_position(double w) {
  const double turns = w * 0.15915494309189535;  // 1 / (2 pi)
  return static_cast<unsigned long long>((turns - floor(turns)) * 18446744073709551616.0);
}
// Sine and cosine at position pos: the product wraps to the fraction of a turn there, which
// alone is rounded to fp32.
__device__ __forceinline__ void sincos_at(long long pos, unsigned long long step, float* sn, float* cs) {
  const long long frac = static_cast<long long>(static_cast<unsigned long long>(pos) * step);
  sincospif(static_cast<float>(frac) * 1.0842021724855044e-19f, sn, cs);  // 2^-63: half turns
}

// V consecutive 16-bit elements.
template <int V>
struct Vec;
template <>
struct Vec<8> { using type = uint4; };
template <>
struct Vec<4> { using type = uint2; };
template <>
struct Vec<2> { using type = uint32_t; };
template <>
struct Vec<1> { using type = uint16_t; };

template <int V, bool kBF16>
__device__ __forceinline__ void widen(typename Vec<V>::type v, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = kBF16 ? __uint_as_float(static_cast<uint32_t>(v) << 16) : __half2float(__ushort_as_half(v));
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 x = unpack2<kBF16>(w[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
}

template <int V, bool kBF16>
__device__ __forceinline__ typename Vec<V>::type narrow(const float (&f)[V]) {
  typename Vec<V>::type v;
  if constexpr (V == 1) {
    v = kBF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(f[0])) : __half_as_ushort(__float2half_rn(f[0]));
  } else {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack2<kBF16>(f[2 * i], f[2 * i + 1]);
  }
  return v;
}

}  // namespace teattn

// Rotary positions: the angle of a position as a fraction of a turn, and the
// element types' pieces, shared by the kernels that turn rows.
#pragma once

#include <cuda_bf16.h>

#include "idx_common.cuh"

namespace idx {
namespace {

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f(float x) { return x; }
template <>
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }

// Turns a position, modulo 1, in units of 2^-64: |freq| = m 2^-s times 2^64 / (2
// pi), whose first 128 bits are kHi and kLo, in whole numbers (64-bit floating
// point is slow here: 5.9 us against 5.3 for 512 tokens of 64 + 4 heads).
__device__ __forceinline__ unsigned long long step_of(double freq) {
  constexpr unsigned long long kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;
  const unsigned long long bits = (unsigned long long)__double_as_longlong(freq);
  const int e = (int)(bits >> 52) & 0x7FF, s = 1075 - max(e, 1);
  const unsigned long long m = (bits & 0xFFFFFFFFFFFFFull) | (e > 0 ? 1ull << 52 : 0ull);
  const unsigned long long carry = __umul64hi(m, kLo), low = m * kHi + carry;
  const unsigned long long high = __umul64hi(m, kHi) + (low < carry ? 1ull : 0ull);
  auto shifted = [&](int n) {  // bits n .. n + 63 of the product
    return n >= 128 ? 0ull : n >= 64 ? high >> (n - 64) : n > 0 ? low >> n | high << (64 - n) : n > -64 ? low << -n : 0ull;
  };
  const unsigned long long step = s > 0 ? shifted(s) + (shifted(s - 1) & 1ull) : shifted(s);
  return bits >> 63 ? 0ull - step : step;
}

// The cosine and sine of position * step, times m.
__device__ __forceinline__ float2 turn_of(int position, unsigned long long step, float m) {
  const unsigned long long phase = step * (unsigned long long)(long long)position;
  const float half_turns = (float)(long long)phase * 1.0842021724855044e-19f;  // 2^-63: signed, in half turns
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * m, s * m);
}

// Two values at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A piece as 32-bit words: elements 2i and 2i + 1, and their rounding back.
template <typename T>
struct Words;
template <>
struct Words<float> {
  static __device__ __forceinline__ float2 get(const uint32_t* w, int i) { return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1])); }
  static __device__ __forceinline__ void put(uint32_t* w, int i, float2 y, bool ok) {
    w[2 * i] = ok ? __float_as_uint(y.x) : w[2 * i], w[2 * i + 1] = ok ? __float_as_uint(y.y) : w[2 * i + 1];
  }
};
template <>
struct Words<__half> {
  static __device__ __forceinline__ float2 get(const uint32_t* w, int i) { return __half22float2(*reinterpret_cast<const __half2*>(w + i)); }
  static __device__ __forceinline__ void put(uint32_t* w, int i, float2 y, bool ok) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y.y), "f"(y.x));
    w[i] = ok ? r : w[i];
  }
};
template <>
struct Words<__nv_bfloat16> {
  static __device__ __forceinline__ float2 get(const uint32_t* w, int i) { return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)); }
  static __device__ __forceinline__ void put(uint32_t* w, int i, float2 y, bool ok) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y.y), "f"(y.x));
    w[i] = ok ? r : w[i];
  }
};
template <int N>
struct alignas(4 * N) Row {
  uint32_t w[N];
};

}  // namespace
}  // namespace idx

// The 8-bit cache's block: places, codes and conversions (device side).
#pragma once

#include "common.cuh"

#include <cuda_fp16.h>

namespace bc {

// One block: key codes [HD/64][16][64], value codes [HD/4][4][4][4], two f32
// scales and padding to whole 32-byte sectors.
__host__ __device__ constexpr int kv8_block_bytes(int hd) { return 2 * kPage * hd + 32; }

// byte of the key code of dims d .. d + 3 (d a multiple of 4) of token p
__device__ __forceinline__ int kv8_k_at(int p, int d) { return (d >> 6) * (kPage * 64) + p * 64 + (d & 63); }

template <int TYPE>
struct Kv8Code;   // TYPE: bc_kv8_type

// Floating point, 4 exponent and 3 mantissa bits.
template <>
struct Kv8Code<0> {
  static constexpr float kMax = 448.f;
  // four values already divided by the scale, rounded to nearest even
  static __device__ __forceinline__ uint32_t encode(float x0, float x1, float x2, float x3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  }
  // four codes as two f16 pairs (exact)
  static __device__ __forceinline__ void decode(uint32_t w, uint32_t& a, uint32_t& b) {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(w & 0xffffu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(w >> 16)));
  }
};

// Integers -127 .. 127.
template <>
struct Kv8Code<1> {
  static constexpr float kMax = 127.f;
  // 1.5 2^23 + x has the rounded x (ties to even) in its low bits; a value
  // divided by its scale is at most 127 (1 + 2^-23), so nothing to clamp
  static __device__ __forceinline__ uint32_t encode(float x0, float x1, float x2, float x3) {
    const uint32_t lo = __byte_perm(__float_as_uint(x0 + 12582912.f), __float_as_uint(x1 + 12582912.f), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(x2 + 12582912.f), __float_as_uint(x3 + 12582912.f), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  // a code c is the f16 number 0x6400 | (c + 128) = 1024 + (c + 128), less
  // 1152 (both exact)
  static __device__ __forceinline__ void decode(uint32_t w, uint32_t& a, uint32_t& b) {
    const uint32_t x = w ^ 0x80808080u;
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    uint32_t u = __byte_perm(x, 0x64646464u, 0x4140), v = __byte_perm(x, 0x64646464u, 0x4342);
    __half2 p = __hsub2(*reinterpret_cast<__half2*>(&u), off), q = __hsub2(*reinterpret_cast<__half2*>(&v), off);
    a = *reinterpret_cast<uint32_t*>(&p);
    b = *reinterpret_cast<uint32_t*>(&q);
  }
};

template <int TYPE>
__device__ __forceinline__ float4 kv8_decode4(uint32_t w) {
  uint32_t a, b;
  Kv8Code<TYPE>::decode(w, a, b);
  const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a)), y = __half22float2(*reinterpret_cast<__half2*>(&b));
  return make_float4(x.x, x.y, y.x, y.y);
}

// 4 x 4 bytes transposed: byte j of word i goes to byte i of word j.
__device__ __forceinline__ void transpose4x4(uint32_t& w0, uint32_t& w1, uint32_t& w2, uint32_t& w3) {
  const uint32_t a = __byte_perm(w0, w1, 0x5140), b = __byte_perm(w2, w3, 0x5140);   // w0.0 w1.0 w0.1 w1.1
  const uint32_t c = __byte_perm(w0, w1, 0x7362), d = __byte_perm(w2, w3, 0x7362);   // w0.2 w1.2 w0.3 w1.3
  w0 = __byte_perm(a, b, 0x5410);
  w1 = __byte_perm(a, b, 0x7632);
  w2 = __byte_perm(c, d, 0x5410);
  w3 = __byte_perm(c, d, 0x7632);
}

}  // namespace bc

// Eight channels at a time: loads, stores and conversions of bf16, fp32 and e4m3
// with power-of-two scales, shared by the norm and the 8-bit kernels.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "ptx.cuh"

namespace flce {

constexpr int kVec = 8;            // channels per thread and step: one 16-byte bf16 load

// ------------------------------------------------------------------ 8-channel loads and stores
struct Raw8 {
  uint4 a, b;  // bf16: a only
};

template <typename E>
__device__ __forceinline__ Raw8 load8(const E* p) {
  Raw8 r;
  r.a = *reinterpret_cast<const uint4*>(p);
  if constexpr (sizeof(E) == 4) r.b = *reinterpret_cast<const uint4*>(p + 4);
  return r;
}

template <typename E>
__device__ __forceinline__ void unpack8(const Raw8& r, float (&v)[kVec]) {
  if constexpr (sizeof(E) == 4) {
    v[0] = __uint_as_float(r.a.x), v[1] = __uint_as_float(r.a.y), v[2] = __uint_as_float(r.a.z);
    v[3] = __uint_as_float(r.a.w), v[4] = __uint_as_float(r.b.x), v[5] = __uint_as_float(r.b.y);
    v[6] = __uint_as_float(r.b.z), v[7] = __uint_as_float(r.b.w);
  } else {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

template <typename E>
__device__ __forceinline__ Raw8 pack8(const float (&v)[kVec]) {
  Raw8 r;
  if constexpr (sizeof(E) == 4) {
    r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    r.a = make_uint4(ptx::pack_bf16x2(v[0], v[1]), ptx::pack_bf16x2(v[2], v[3]), ptx::pack_bf16x2(v[4], v[5]),
                     ptx::pack_bf16x2(v[6], v[7]));
  }
  return r;
}

template <typename E>
__device__ __forceinline__ void store8(E* p, const Raw8& r) {
  *reinterpret_cast<uint4*>(p) = r.a;
  if constexpr (sizeof(E) == 4) *reinterpret_cast<uint4*>(p + 4) = r.b;
}

// ------------------------------------------------------------------ pairs
// Two fp32 numbers in a 64-bit register: one instruction multiplies or adds both.
using F2 = unsigned long long;

__device__ __forceinline__ F2 pair(uint32_t lo, uint32_t hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ F2 both(float v) { return pair(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ void split(F2 v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a), hi = __uint_as_float(b);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 fma2_zero(F2 a, F2 b, F2 c) {  // rounded towards zero
  F2 r;
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// a + b, and what it rounds off added to `off` (Knuth's two-sum).
__device__ __forceinline__ F2 add2(F2 a, F2 b, F2& off) {
  const F2 minus = both(-1.0f);
  const F2 s = add2(a, b), t = fma2(a, minus, s);
  off = add2(off, add2(fma2(fma2(t, minus, s), minus, a), fma2(t, minus, b)));
  return s;
}

constexpr int kPairs = kVec / 2;

template <typename E>
__device__ __forceinline__ void unpack_pairs(const Raw8& r, F2 (&v)[kPairs]) {
  if constexpr (sizeof(E) == 4) {
    v[0] = pair(r.a.x, r.a.y), v[1] = pair(r.a.z, r.a.w), v[2] = pair(r.b.x, r.b.y), v[3] = pair(r.b.z, r.b.w);
  } else {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
    for (int i = 0; i < kPairs; ++i) v[i] = pair(w[i] << 16, w[i] & 0xffff0000u);
  }
}

template <typename E>
__device__ __forceinline__ Raw8 pack_pairs(const F2 (&v)[kPairs]) {
  float f[kVec];
#pragma unroll
  for (int i = 0; i < kPairs; ++i) split(v[i], f[2 * i], f[2 * i + 1]);
  return pack8<E>(f);
}

// ------------------------------------------------------------------ sums of twice 24 bits
// hi + lo: what an addition rounds off is kept.
struct Twofold {
  float hi, lo;
};
__device__ __forceinline__ Twofold operator+(Twofold a, Twofold b) {
  Twofold r;
  r.hi = a.hi + b.hi;
  const float t = r.hi - a.hi;
  r.lo = (a.hi - (r.hi - t)) + (b.hi - t) + (a.lo + b.lo);
  return r;
}
__device__ __forceinline__ Twofold warp_sum_twofold(Twofold t) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    t = t + Twofold{__shfl_xor_sync(0xffffffffu, t.hi, d), __shfl_xor_sync(0xffffffffu, t.lo, d)};
  return t;
}

// ------------------------------------------------------------------ e4m3 with a power-of-two scale
// E8M0 byte of the smallest 2^e with amax / 2^e <= 448 = 1.75 * 2^8, e >= -126.
// From amax's own exponent and mantissa (amax is finite and not negative).
__device__ __forceinline__ uint32_t e8m0_of(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 1));
}

// 2^-(e - 127) for an e8m0_of() byte (1 .. 248): exact.
__device__ __forceinline__ float inv_scale(uint32_t e8m0) { return __uint_as_float((254u - e8m0) << 23); }

// Eight floats to e4m3, round to nearest even, |v| > 448 to 448, NaN kept.
__device__ __forceinline__ uint2 to_e4m3x8(const float* v, float inv) {
  uint16_t h[4];
  const F2 by = both(inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    split(mul2(pair(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1])), by), lo, hi);
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(hi), "f"(lo));
  }
  return make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16));
}

}  // namespace flce

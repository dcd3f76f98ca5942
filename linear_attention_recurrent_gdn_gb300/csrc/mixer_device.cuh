// Element access shared by the mixer kernels: eight consecutive values of a
// type, moved as 16-byte vectors when VEC (the host checked alignment) and one
// by one otherwise, and held in 32 bits.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "mixer.h"

namespace dl {
namespace mx {

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <class T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }

template <class T> __device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b);
template <> __device__ __forceinline__ void unpack2<__nv_bfloat16>(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
template <> __device__ __forceinline__ void unpack2<__half>(uint32_t w, float& a, float& b) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x;
  b = f.y;
}
template <class T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 p = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Eight values of type T as they sit in memory.
template <class T> struct Vec8 { uint32_t w[sizeof(T) == 4 ? 8 : 4]; };

template <class T, bool VEC>
__device__ __forceinline__ Vec8<T> load8(const T* p, int valid) {
  Vec8<T> v;
  constexpr int NW = sizeof(T) == 4 ? 8 : 4;
  if (VEC) {
    if (valid > 0) {
#pragma unroll
      for (int k = 0; k < NW / 4; ++k) {
        const uint4 u = reinterpret_cast<const uint4*>(p)[k];
        v.w[4 * k] = u.x;
        v.w[4 * k + 1] = u.y;
        v.w[4 * k + 2] = u.z;
        v.w[4 * k + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < NW; ++k) v.w[k] = 0u;
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v.w[k] = k < valid ? reinterpret_cast<const uint32_t*>(p)[k] : 0u;
  } else {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = 2 * k < valid ? q[2 * k] : 0u, hi = 2 * k + 1 < valid ? q[2 * k + 1] : 0u;
      v.w[k] = lo | (hi << 16);
    }
  }
  return v;
}
template <class T, bool VEC>
__device__ __forceinline__ void store8(T* p, const Vec8<T>& v, int valid) {
  constexpr int NW = sizeof(T) == 4 ? 8 : 4;
  if (VEC) {
    if (valid > 0) {
#pragma unroll
      for (int k = 0; k < NW / 4; ++k)
        reinterpret_cast<uint4*>(p)[k] = make_uint4(v.w[4 * k], v.w[4 * k + 1], v.w[4 * k + 2], v.w[4 * k + 3]);
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < valid) reinterpret_cast<uint32_t*>(p)[k] = v.w[k];
  } else {
    uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < valid) q[k] = (uint16_t)(v.w[k >> 1] >> (16 * (k & 1)));
  }
}
template <class T> __device__ __forceinline__ void unpack8(const Vec8<T>& v, float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v.w[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack2<T>(v.w[k], f[2 * k], f[2 * k + 1]);
  }
}
template <class T> __device__ __forceinline__ Vec8<T> pack8(const float (&f)[8]) {
  Vec8<T> v;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v.w[k] = __float_as_uint(f[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v.w[k] = pack2<T>(f[2 * k], f[2 * k + 1]);
  }
  return v;
}
// Eight values as four pairs.
template <class T> __device__ __forceinline__ void pairs8(const Vec8<T>& v, unsigned long long (&f)[4]) {
  float t[8];
  unpack8<T>(v, t);
#pragma unroll
  for (int k = 0; k < 4; ++k) asm("mov.b64 %0, {%1, %2};" : "=l"(f[k]) : "f"(t[2 * k]), "f"(t[2 * k + 1]));
}
// Eight weights that are fp32 or of the activations' type.
template <class T, bool VEC>
__device__ __forceinline__ void weights8(const void* base, int64_t i, int valid, int f32, float (&f)[8]) {
  if (f32) {
    unpack8<float>(load8<float, VEC>(static_cast<const float*>(base) + i, valid), f);
  } else {
    unpack8<T>(load8<T, VEC>(static_cast<const T*>(base) + i, valid), f);
  }
}

// 1 / x within one step of the last place.
__device__ __forceinline__ float rcp_f(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Packed fp32 arithmetic: two values an instruction.
using f2 = unsigned long long;     // two fp32 values
__device__ __forceinline__ f2 mk2(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void un2(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ float ex2_f(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// silu (z / (1 + e^-z)) or sigmoid (1 / (1 + e^-z)) of a pair.  16-bit types:
// the fast e^x, within about 2^-20 relative, far below the type's own
// rounding, and one reciprocal for both, 1 / (p q); the exponentials are held
// at 2^62, so that the product is finite and a NaN stays its own value's, and
// silu's z at -43 (its value is -9e-18 or less in size either way).
template <class T, bool SILU>
__device__ __forceinline__ f2 act2(f2 z) {
  float a, b;
  if constexpr (sizeof(T) == 4) {
    un2(z, a, b);
    const float p = rcp_f(1.f + expf(-a)), q = rcp_f(1.f + expf(-b));
    return SILU ? mk2(a * p, b * q) : mk2(p, q);
  } else {
    un2(mul2(z, mk2(-1.4426950408889634f, -1.4426950408889634f)), a, b);
    float p, q;
    un2(add2(mk2(fminf(ex2_f(a), 0x1p62f), fminf(ex2_f(b), 0x1p62f)), mk2(1.f, 1.f)), p, q);
    const float r = rcp_f(p * q);
    const f2 s = mul2(mk2(q, p), mk2(r, r));
    un2(z, a, b);
    if (SILU) return mul2(mk2(max_nan(a, -43.f), max_nan(b, -43.f)), s);
    un2(s, p, q);
    return mk2(a != a ? a : p, b != b ? b : q);    // a NaN stays one
  }
}

// log(1 + e^x) without overflow or loss for either sign.
__device__ __forceinline__ float softplus_f(float x) { return fmaxf(x, 0.f) + log1pf(expf(-fabsf(x))); }

}  // namespace mx
}  // namespace dl

// Rows of bf16 or fp32 values in 16-byte units, exponentials in base 2, and two floats at a
// time: what the kernels over rows of logits or activations share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "epilogue.cuh"

namespace muon {
namespace {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// ex2.approx is low by 4.9e-8 in the mean over [-16, 0), measured against 64 bits (its
// terms of exactly 1 are not): a sequence's sum of log-probabilities adds that up, so the
// sum makes up for it.  Where many logits equal the largest, whose terms are exactly 1, the
// correction is the error: 4.9e-8 in log S, under half a unit of any |logp| >= 1.
constexpr float kExpLow = 4.9e-8f;

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;  // elements of 16 bytes
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  static constexpr uint32_t kLowest = 0xFF800000u;  // -inf in every element of a word
  static __device__ __forceinline__ uint4 mask_of(int e) {  // the bits of element e
    return make_uint4(e == 0 ? ~0u : 0u, e == 1 ? ~0u : 0u, e == 2 ? ~0u : 0u, e == 3 ? ~0u : 0u);
  }
  template <int G>
  static __device__ __forceinline__ float max(const uint4 (&w)[G]) {
    float m = -INFINITY;
#pragma unroll
    for (int g = 0; g < G; ++g)
      m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(w[g].x), __uint_as_float(w[g].y)),
                         fmaxf(__uint_as_float(w[g].z), __uint_as_float(w[g].w))));
    return m;
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
  static constexpr uint32_t kLowest = 0xFF80FF80u;
  static __device__ __forceinline__ uint4 mask_of(int e) {
    const uint32_t m = (e & 1) ? 0xFFFF0000u : 0x0000FFFFu;
    return make_uint4((e >> 1) == 0 ? m : 0u, (e >> 1) == 1 ? m : 0u, (e >> 1) == 2 ? m : 0u, (e >> 1) == 3 ? m : 0u);
  }
  template <int G>
  static __device__ __forceinline__ float max(const uint4 (&w)[G]) {
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&w[0].x);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t u[4] = {w[g].x, w[g].y, w[g].z, w[g].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&u[i]));
    }
    return fmaxf(__low2float(m), __high2float(m));
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

// Replaces the masked bits of a unit by those of -inf.
template <typename T>
__device__ __forceinline__ void drop(uint4& w, const uint4& m) {
  w.x = (w.x & ~m.x) | (Vec<T>::kLowest & m.x);
  w.y = (w.y & ~m.y) | (Vec<T>::kLowest & m.y);
  w.z = (w.z & ~m.z) | (Vec<T>::kLowest & m.z);
  w.w = (w.w & ~m.w) | (Vec<T>::kLowest & m.w);
}

// 16-byte accesses with an L2 policy.
__device__ __forceinline__ uint64_t l2_policy(bool evict_first) {
  uint64_t first, normal;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  return evict_first ? first : normal;
}
__device__ __forceinline__ uint4 load16(const uint4* p, uint64_t policy) {
  uint4 w;
  asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p), "l"(policy)
               : "memory");
  return w;
}
__device__ __forceinline__ void store16(uint4* p, const uint4& w, uint64_t policy) {
  asm volatile("st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %5;" ::"l"(p), "r"(w.x), "r"(w.y), "r"(w.z),
               "r"(w.w), "l"(policy)
               : "memory");
}

// Two floats at a time (one issue slot).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 make_f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

__device__ __forceinline__ float warp_max(float v) {  // of the numbers among them, like fmaxf
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

}  // namespace
}  // namespace muon

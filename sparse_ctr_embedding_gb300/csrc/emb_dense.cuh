// Device helpers shared by the dense-tower operators (emb_fp8.cu, emb_fp8_matmul.cu,
// emb_norm_fwd.cu, emb_norm_bwd.cu, emb_adamw.cu): typed loads and stores of eight
// elements, 8-bit codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "emb_internal.cuh"

namespace emb {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;  // keeps 448 / amax finite and amax / 448 normal for an all-zero block
constexpr float kFltMax = 3.402823466e+38f;

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) {
  return __half2float(v);
}
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __uint_as_float((unsigned)__bfloat16_as_ushort(v) << 16);
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Eight consecutive elements as they lie in memory: 32 bytes (f32) or 16.
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float v[8];
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
  }
  __device__ __forceinline__ void store(float* p) const {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ void set2(int i, float a, float b) {
    v[2 * i] = a;
    v[2 * i + 1] = b;
  }
};
template <typename T, typename T2>
struct Raw8Half {
  T2 v[4];
  __device__ __forceinline__ void load(const T* p) {
    unsigned* u = reinterpret_cast<unsigned*>(v);
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]) : "l"(p));
  }
  __device__ __forceinline__ void store(T* p) const {
    const unsigned* u = reinterpret_cast<const unsigned*>(v);
    asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]) : "memory");
  }
};
template <>
struct Raw8<__half> : Raw8Half<__half, __half2> {
  __device__ __forceinline__ float get(int i) const { return __half2float(i & 1 ? __high2half(v[i >> 1]) : __low2half(v[i >> 1])); }
  __device__ __forceinline__ void set2(int i, float a, float b) { v[i] = __floats2half2_rn(a, b); }
};
template <>
struct Raw8<__nv_bfloat16> : Raw8Half<__nv_bfloat16, __nv_bfloat162> {
  __device__ __forceinline__ float get(int i) const {  // a bf16 is the upper half of its float
    const unsigned u = *reinterpret_cast<const unsigned*>(&v[i >> 1]);
    return __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
  }
  __device__ __forceinline__ void set2(int i, float a, float b) { v[i] = __floats2bfloat162_rn(a, b); }
};

// Two floats as e4m3 codes (to nearest even; NaN stays NaN, larger magnitudes
// become 448): `lo` in the low byte.
__device__ __forceinline__ unsigned e4m3x2(float lo, float hi) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32(unsigned short c) {
  unsigned h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

__device__ __forceinline__ bool finite_f32(float x) { return fabsf(x) <= kFltMax; }
// |x| where it is finite, else 0: what counts towards a block's largest magnitude.
__device__ __forceinline__ float finite_abs(float x) { return finite_f32(x) ? fabsf(x) : 0.0f; }

// A block's multiplier and its scale, from its largest magnitude.
__device__ __forceinline__ float inv_of(float amax) { return __fmul_rn(__frcp_rn(amax), kE4m3Max); }
__device__ __forceinline__ float scale_of(float amax) { return __fmul_rn(amax, 1.0f / kE4m3Max); }

inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t ftype_bytes(int t) { return t == EMB_T_F32 ? 4 : 2; }
inline bool good_ftype(int t) { return t == EMB_T_F32 || t == EMB_T_BF16 || t == EMB_T_F16; }

}  // namespace emb

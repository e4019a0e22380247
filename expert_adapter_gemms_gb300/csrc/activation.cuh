// The gated activations and the 16-bit element types, shared by the 16-bit and the 4-bit
// feed-forward kernels.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace moe_lora {

// a(g) = g s(t) with s the logistic function and t = g (SiLU) or
// 2 sqrt(2/pi) (g + 0.044715 g^3) (GELU, tanh form: (1 + tanh z) / 2 = s(2z)); d = a'(g).
// The hardware exponential and reciprocal: a few fp32 ulps (up to |t| ulps for large |t|,
// where s or 1 - s is negligible), far below a 16-bit output's rounding; below t = -87 s is 0
// where the exact value is under 1e-37.
template <int kAct>
__device__ __forceinline__ void activation(float g, float& a, float& d) {
  float t = g, dt = 1.f;
  if (kAct == MOE_ACT_GELU) {
    constexpr float c = 1.5957691216057308f;
    t = c * g * (1.f + 0.044715f * g * g);
    dt = c * (1.f + 0.134145f * fminf(g * g, 1e30f));  // finite: far out it meets s or 1 - s of 0
  }
  const float s = __fdividef(1.f, 1.f + __expf(-t));
  a = g * s;
  d = s + a * (1.f - s) * dt;
}

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float f(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ float f(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 r(float v) { return __float2bfloat16_rn(v); }
  static __device__ __forceinline__ float2 f2(uint32_t v) { return make_float2(bf16_lo(v), bf16_hi(v)); }
  static __device__ __forceinline__ uint32_t r2(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <> struct Elem<__half> {
  static __device__ __forceinline__ float f(uint16_t v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ float f(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half r(float v) { return __float2half_rn(v); }
  static __device__ __forceinline__ float2 f2(uint32_t v) {
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  }
  static __device__ __forceinline__ uint32_t r2(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// D[16 x 8] += A[16 x 16] B[16 x 8], fp32 accumulators; mma16816_from: D = A B + C.
#define MOE_MMA16816(TYPE, PTX)                                                                                  \
  template <>                                                                                                    \
  __device__ __forceinline__ void mma16816<TYPE>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,           \
                                                 uint32_t a3, uint32_t b0, uint32_t b1) {                        \
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." PTX "." PTX                                            \
                 ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"                                    \
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                \
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));                                        \
  }                                                                                                              \
  template <>                                                                                                    \
  __device__ __forceinline__ void mma16816_from<TYPE>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,      \
                                                      uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1, \
                                                      float c2, float c3) {                                      \
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32." PTX "." PTX                                            \
                 ".f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"                                \
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])                                                \
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));    \
  }
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1);
template <typename T>
__device__ __forceinline__ void mma16816_from(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3);
MOE_MMA16816(__nv_bfloat16, "bf16")
MOE_MMA16816(__half, "f16")
#undef MOE_MMA16816

}  // namespace moe_lora

// Activations of the feed-forward operators and their derivatives, in fp32, and
// the conversions of 16-bit elements whose type (fp16 or bf16) is a template
// argument or a run-time flag.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "igc_ffn.h"

namespace igc {

// 2^x and 1/x to within 2^-22 and 2^-23 of their value (one instruction each: the forms
// that flush subnormals need no range handling, and a subnormal 2^x is 0 beside the 1 that
// it is added to here).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2 = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// 1 / (1 + 2^-t): the sigmoid of t / log2(e).  2^-t overflows to infinity for t < -128,
// and its reciprocal is then 0, as the sigmoid is to fp32's precision.
__device__ __forceinline__ float sigmoid2(float t) { return rcp_approx(1.0f + exp2_approx(-t)); }

// 2 log2(e) c (z + a z^3), c = sqrt(2 / pi): z (1 + tanh(u)) / 2 equals z sigmoid(2 u), which
// needs no tanh and keeps its relative accuracy where tanh(u) is near -1.
__device__ __forceinline__ float gelu_tanh_arg(float z, float z2) {
  return z * fmaf(2.0f * kLog2E * kGeluC * kGeluA, z2, 2.0f * kLog2E * kGeluC);
}

// act(z)
template <int kAct>
__device__ __forceinline__ float act_f32(float z) {
  if constexpr (kAct == IGC_ACT_RELU) return z > 0.0f ? z : (z != z ? z : 0.0f);
  if constexpr (kAct == IGC_ACT_GELU) return 0.5f * z * (1.0f + erff(z * kInvSqrt2));
  if constexpr (kAct == IGC_ACT_GELU_TANH) return z * sigmoid2(gelu_tanh_arg(z, z * z));
  if constexpr (kAct == IGC_ACT_SILU) return z * sigmoid2(kLog2E * z);
  return z;
}

// act(z) and act'(z) together (they share the exponential).
template <int kAct>
__device__ __forceinline__ void act_grad_f32(float z, float& f, float& d) {
  if constexpr (kAct == IGC_ACT_RELU) {
    f = z > 0.0f ? z : (z != z ? z : 0.0f);
    d = z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (kAct == IGC_ACT_GELU) {
    const float cdf = fmaf(0.5f, erff(z * kInvSqrt2), 0.5f);
    f = z * cdf;
    d = fmaf(z * kInvSqrt2Pi, exp2_approx((-0.5f * kLog2E) * z * z), cdf);
  } else if constexpr (kAct == IGC_ACT_GELU_TANH) {
    // s (1 - s) is 0 long before z^2 reaches the bound.  It meets z first and the polynomial
    // then: both products stay finite for every finite z (z times the polynomial would not
    // from 1.6e27 on, and infinity times 0 is NaN)
    const float z2 = fminf(z * z, 1e12f);
    const float s = sigmoid2(gelu_tanh_arg(z, z2));
    f = z * s;
    d = fmaf(z * fmaf(-s, s, s), fmaf(6.0f * kGeluC * kGeluA, z2, 2.0f * kGeluC), s);
  } else if constexpr (kAct == IGC_ACT_SILU) {
    const float s = sigmoid2(kLog2E * z);
    f = z * s;
    d = fmaf(f, 1.0f - s, s);
  } else {
    f = z;
    d = 1.0f;
  }
}

// Calls f(std::integral_constant<int, kAct>{}): the activation as a compile-time constant.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case IGC_ACT_RELU: f(std::integral_constant<int, IGC_ACT_RELU>{}); break;
    case IGC_ACT_GELU: f(std::integral_constant<int, IGC_ACT_GELU>{}); break;
    case IGC_ACT_GELU_TANH: f(std::integral_constant<int, IGC_ACT_GELU_TANH>{}); break;
    case IGC_ACT_SILU: f(std::integral_constant<int, IGC_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, IGC_ACT_NONE>{}); break;
  }
}

// The two 16-bit elements of a word, widened; two fp32 values rounded and packed.
__device__ __forceinline__ float2 unpack16(uint32_t w, bool bf16) {
  if (bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool bf16) {
  if (bf16) {
    __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float load16(const void* p, long long i, bool bf16) {
  return unpack16(static_cast<const uint16_t*>(p)[i], bf16).x;
}

__device__ __forceinline__ void store16(void* p, long long i, float v, bool bf16) {
  static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack16(v, 0.0f, bf16) & 0xffffu);
}

// Element i of a vector that is fp32 (f32) or of the operands' 16-bit type; 0 for no vector.
__device__ __forceinline__ float load_vec(const void* p, long long i, bool f32, bool bf16) {
  if (p == nullptr) return 0.0f;
  return f32 ? static_cast<const float*>(p)[i] : load16(p, i, bf16);
}

}  // namespace igc

// 16-bit (bf16 / f16) matrix-core helpers and the gated activations shared by
// the feed-forward and adapter kernels.
#pragma once

#include <type_traits>

#include "q8_device.h"

namespace q8 {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// v_mfma_f32_16x16x32: lane (g, r) = (lane / 16, lane % 16) holds K elements
// 8g .. 8g+7 of row r of either operand and receives D[4g .. 4g+3][r] (operand
// 0's rows by operand 1's).
template <bool BF>
__device__ __forceinline__ f32x4 mfma16(const i32x4& a, const i32x4& b, const f32x4& c) {
  if constexpr (BF)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0,
                                                  0);
}

// two float32 -> two 16-bit values in one register, round to nearest even
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2{(__bf16)a, (__bf16)b});
  } else {
    typedef _Float16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2{(_Float16)a, (_Float16)b});
  }
}

template <bool BF>
__device__ __forceinline__ float lo_f32(uint32_t w) {
  return out_bits_to_f32<BF>(w & 0xFFFFu);
}
template <bool BF>
__device__ __forceinline__ float hi_f32(uint32_t w) {
  return out_bits_to_f32<BF>(w >> 16);
}

// FP8 codes of v / s (true division, |v / s| <= 448 up to its rounding, which
// the clamp takes off)
__device__ __forceinline__ uint32_t fp8_codes4(f32x4 v, float s) {
  float y[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) y[r] = __builtin_amdgcn_fmed3f(v[r] / s, -448.0f, 448.0f);
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
}

// ---- activations ---------------------------------------------------------------
enum { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

// exp(x) with the rounding error of x * log2(e) put back as a first-order
// factor: within a few float32 roundings over the whole range (2^t alone is
// off by |x| 2^-24).
__device__ __forceinline__ float exp_f32(float x) {
  constexpr float kL2e = 1.44269504088896340736f, kL2eLo = 1.92596299112661746887e-8f, kLn2 = 0.69314718055994530942f;
  const float t = x * kL2e;
  const float e = __builtin_amdgcn_exp2f(t);
  const float lo = __builtin_fmaf(x, kL2eLo, __builtin_fmaf(x, kL2e, -t));
  // overflow and infinite x keep e (lo is then not a number)
  return __builtin_fabsf(t) < 126.0f ? __builtin_fmaf(e, lo * kLn2, e) : e;
}

__device__ __forceinline__ float sigmoid_f32(float x) { return __builtin_amdgcn_rcpf(1.0f + exp_f32(-x)); }

constexpr float kGeluC = 0.79788456080286535588f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// act(g). gelu: g Phi(g) with Phi(g) = erfc(-g / sqrt 2) / 2 (no cancellation
// for negative g); gelu_tanh: 0.5 (1 + tanh y) = sigmoid(2 y).
template <int ACT>
__device__ __forceinline__ float act_f32(float g) {
  if constexpr (ACT == kSilu) return g * sigmoid_f32(g);
  else if constexpr (ACT == kGelu) return 0.5f * g * erfcf(-0.70710678118654752440f * g);
  else return g * sigmoid_f32(2.0f * kGeluC * __builtin_fmaf(kGeluA * g * g, g, g));
}

// act'(g), with act(g) in a
template <int ACT>
__device__ __forceinline__ float act_grad_f32(float g, float& a) {
  if constexpr (ACT == kSilu) {
    const float s = sigmoid_f32(g);
    a = g * s;
    return __builtin_fmaf(a, 1.0f - s, s);
  } else if constexpr (ACT == kGelu) {
    const float phi = 0.5f * erfcf(-0.70710678118654752440f * g);
    a = g * phi;
    return __builtin_fmaf(g * 0.39894228040143267794f, exp_f32(-0.5f * g * g), phi);
  } else {
    // s = sigmoid(2y): s' = 2 s (1 - s) y'; y' is kept finite, as s (1 - s) = 0
    // where it would overflow
    const float y2 = 2.0f * kGeluC * __builtin_fmaf(kGeluA * g * g, g, g);
    const float s = sigmoid_f32(y2);
    a = g * s;
    const float dy = __builtin_fminf(__builtin_fmaf(3.0f * kGeluA * g, g, 1.0f), 1e38f);
    return __builtin_fmaf(a * (1.0f - s), 2.0f * kGeluC * dy, s);
  }
}

template <typename F>
__device__ __forceinline__ void act_switch(int act, F&& f) {
  if (act == kSilu) f(std::integral_constant<int, kSilu>{});
  else if (act == kGelu) f(std::integral_constant<int, kGelu>{});
  else f(std::integral_constant<int, kGeluTanh>{});
}

}  // namespace q8

// Activations of the dense and the gated linear layers, eight results at a time: values and
// slopes.  Internal to libpoetx.
#pragma once

#include "common.h"

namespace poetx {

namespace {

constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC = 0.79788456080286536f, kTanhA = 0.044715f;  // sqrt(2 / pi)

// The activations run on every result of a product's epilogue, where the matrix cores wait for
// them.  bf16: one hardware exp and one reciprocal each (relative errors of about 2^-22, and of
// 2^-24 of exp's argument, far below the rounding of the result), not the library's erf and tanh
// (whose epilogue took 31 us of a 130 us round of 256 x 256 tiles, k = 4096; 8192 tokens, 4096 ->
// 14336 with GELU and the kept pre-activation: 904 us then, 743 us now).  float32, whose products
// run at a tenth of the rate: the library's functions, a few units in the last place (2048 tokens,
// 1024 -> 4096 with GELU 159 us, 155 us with the forms for bf16).
template <typename T> struct Fn;
template <> struct Fn<bf16_t> {
  static __device__ inline float exp(float x) { return __expf(x); }
  static __device__ inline float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }
  // Phi(p) = erfc(-p / sqrt 2) / 2, with erfc(x) exp(x^2) / 2 for x >= 0 as a polynomial in t =
  // 1 / (1 + 0.51 x) without a constant term: a fit of least largest relative error over x <= 10,
  // 1.2e-6 in float32, so that far negative p keep their digits too; e: exp(-p^2 / 2).
  static __device__ inline float normal_cdf(float p, float e) {
    const float x = fabsf(p) * 0.70710678118654752f, t = __builtin_amdgcn_rcpf(fmaf(0.51f, x, 1.f));
    float q = fmaf(t, 0.0472500883f, -0.17956777f);
    q = fmaf(t, q, 0.179223239f);
    q = fmaf(t, q, 0.0275261737f);
    q = fmaf(t, q, 0.139533147f);
    q = fmaf(t, q, 0.14207615f);
    q = fmaf(t, q, 0.143958747f);
    q *= t * e;
    return p < 0.f ? q : 1.f - q;
  }
};
template <> struct Fn<float> {
  static __device__ inline float exp(float x) { return expf(x); }
  static __device__ inline float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }
  static __device__ inline float normal_cdf(float p, float) { return 0.5f * erfcf(-0.70710678118654752f * p); }
};

// v = act(v); one branch for the eight
template <typename T>
__device__ inline void act_values(float (&v)[8], int act) {
  switch (act) {
    case POETX_ACT_RELU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] < 0.f ? 0.f : v[e];  // a NaN stays NaN
      break;
    case POETX_ACT_GELU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= Fn<T>::normal_cdf(v[e], Fn<T>::exp(-0.5f * v[e] * v[e]));
      break;
    case POETX_ACT_GELU_TANH:  // (1 + tanh u) / 2 = sigmoid(2 u)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= Fn<T>::sigmoid(2.f * kTanhC * (v[e] + kTanhA * v[e] * v[e] * v[e]));
      break;
    case POETX_ACT_SILU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= Fn<T>::sigmoid(v[e]);
      break;
    default: break;
  }
}

// v *= act'(p)
template <typename T>
__device__ inline void act_slopes(float (&v)[8], const float (&p)[8], int act) {
  switch (act) {
    case POETX_ACT_RELU:
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= p[e] > 0.f ? 1.f : p[e] <= 0.f ? 0.f : p[e];  // 0 at 0; a NaN stays NaN
      break;
    case POETX_ACT_GELU:
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = Fn<T>::exp(-0.5f * p[e] * p[e]);
        v[e] *= Fn<T>::normal_cdf(p[e], d) + p[e] * kInvSqrt2Pi * d;
      }
      break;
    case POETX_ACT_GELU_TANH:
      // beyond |p| = 20 the slope is 0 or 1 to every float32 digit, while p^3 could overflow;
      // with g = sigmoid(2 u): d(p g) = g + p g (1 - g) 2 u'
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float q = p[e] < -20.f ? -20.f : p[e] > 20.f ? 20.f : p[e];
        const float g = Fn<T>::sigmoid(2.f * kTanhC * (q + kTanhA * q * q * q));
        v[e] *= g + q * g * (1.f - g) * 2.f * kTanhC * (1.f + 3.f * kTanhA * q * q);
      }
      break;
    case POETX_ACT_SILU:
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = Fn<T>::sigmoid(p[e]);
        v[e] *= g * (1.f + p[e] * (1.f - g));
      }
      break;
    default: break;
  }
}

}  // namespace

}  // namespace poetx

// The activations of the linear layer and their derivatives, in fp32.
#pragma once

namespace gb300 {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }

// sigmoid(v) and its derivative, from exp(-|v|): nothing cancels or overflows.
__device__ __forceinline__ void sigmoid_slope(float v, float& s, float& slope) {
  const float t = __expf(-fabsf(v)), big = __fdividef(1.f, 1.f + t);
  s = v >= 0.f ? big : t * big;
  slope = t * big * big;
}

// Standard normal distribution function and density at v, from one exponential:
// Abramowitz and Stegun, "Handbook of Mathematical Functions", 7.1.26,
//   erfc(x) = t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) exp(-x^2),  t = 1/(1 + p x),
// for x >= 0, absolute error at most 1.5e-7 (the size of an fp32 rounding of
// the result); cdf(v) = erfc(-v/sqrt 2)/2, by symmetry for either sign.
__device__ __forceinline__ void normal_cdf_pdf(float v, float& cdf, float& e) {
  const float x = fabsf(v) * 0.70710678f;
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  e = __expf(-x * x);                  // exp(-v^2 / 2)
  const float half_erfc = 0.5f * p * t * e;
  cdf = v >= 0.f ? 1.f - half_erfc : half_erfc;
}

// 2 sqrt(2/pi) (v + 0.044715 v^3): the tanh form of gelu is v sigmoid(this).
__device__ __forceinline__ float gelu_tanh_arg(float v) {
  return v * fmaf(0.0713548163f, v * v, 1.5957691216f);
}

template <int ACT>
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == ACT_RELU) return fmaxf(v, 0.f);
  if constexpr (ACT == ACT_GELU) {
    float cdf, e;
    normal_cdf_pdf(v, cdf, e);
    return v * cdf;
  }
  if constexpr (ACT == ACT_GELU_TANH) return v * sigmoid(gelu_tanh_arg(v));
  if constexpr (ACT == ACT_SILU) return v * sigmoid(v);
  return v;
}

// The derivative.  Past |v| = 80 it is 0 or 1 to the last bit of fp32; v is
// held there, so that no infinity meets a zero (a NaN stays one).
template <int ACT>
__device__ __forceinline__ float activate_grad(float v) {
  if constexpr (ACT == ACT_RELU) return v > 0.f ? 1.f : 0.f;
  v = fabsf(v) > 80.f ? copysignf(80.f, v) : v;
  if constexpr (ACT == ACT_GELU) {
    float cdf, e;
    normal_cdf_pdf(v, cdf, e);
    return fmaf(v * 0.3989422804f, e, cdf);
  }
  if constexpr (ACT == ACT_GELU_TANH) {
    float s, slope;
    sigmoid_slope(gelu_tanh_arg(v), s, slope);
    return fmaf(v * slope, fmaf(0.2140644489f, v * v, 1.5957691216f), s);
  }
  if constexpr (ACT == ACT_SILU) {
    float s, slope;
    sigmoid_slope(v, s, slope);
    return fmaf(v, slope, s);
  }
  return 1.f;
}

// f(integral constant) for the activation `act`, outside the element loops.
template <int V>
struct IntC { static constexpr int value = V; };
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  if (act == ACT_NONE) f(IntC<ACT_NONE>{});
  else if (act == ACT_RELU) f(IntC<ACT_RELU>{});
  else if (act == ACT_GELU) f(IntC<ACT_GELU>{});
  else if (act == ACT_GELU_TANH) f(IntC<ACT_GELU_TANH>{});
  else f(IntC<ACT_SILU>{});
}

}  // namespace gb300

// The activations of the linear layer and their derivatives, in fp32.
//
// Built on the hardware's 2^x and reciprocal (relative errors about 2^-22 and
// 2^-23, small arguments' results flushed to zero), written so that no infinity
// meets a zero in a derivative and a NaN stays one.
#pragma once

namespace gb300 {

enum : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// min(|x|, m), NaN where x is.
__device__ __forceinline__ float min_abs(float x, float m) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(fabsf(x)), "f"(m));
  return y;
}

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid(float v) {
  return rcp_fast(1.f + exp2_fast(-kLog2e * v));
}

// sigmoid(v) and its derivative, from exp(-|v|): nothing cancels.
__device__ __forceinline__ void sigmoid_slope(float v, float& s, float& slope) {
  const float t = exp2_fast(-kLog2e * fabsf(v)), big = rcp_fast(1.f + t), small = t * big;
  s = v >= 0.f ? big : small;
  slope = small * big;
}

// The standard normal distribution function at v, and exp(-v^2/2), from one
// exponential: Abramowitz and Stegun, "Handbook of Mathematical Functions",
// 7.1.26,
//   erfc(x) = t (a1 + t (a2 + t (a3 + t (a4 + t a5)))) exp(-x^2),  t = 1/(1 + p x),
// for x >= 0, absolute error at most 1.5e-7 (the size of an fp32 rounding of
// the result); cdf(v) = erfc(-v/sqrt 2)/2, by symmetry for either sign.  a =
// min(|v|, 20): there the exponential is zero.  (Coefficients halved, p over
// sqrt 2.)
__device__ __forceinline__ void normal_cdf_exp(float v, float a, float& cdf, float& e) {
  const float t = rcp_fast(fmaf(0.231641888f, a, 1.f));
  e = exp2_fast(a * a * (-0.5f * kLog2e));
  float p = fmaf(0.5307027145f, t, -0.7265760135f);
  p = fmaf(p, t, 0.7107068705f);
  p = fmaf(p, t, -0.142248368f);
  p = fmaf(p, t, 0.127414796f);
  cdf = 0.5f + copysignf(fmaf(p * t, -e, 0.5f), v);
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
    normal_cdf_exp(v, min_abs(v, 20.f), cdf, e);
    return v * cdf;
  }
  if constexpr (ACT == ACT_GELU_TANH) return v * sigmoid(gelu_tanh_arg(v));
  if constexpr (ACT == ACT_SILU) return v * sigmoid(v);
  return v;
}

// The derivative.  Far out (|v| = 20 for the gelus, 100 for silu) it is 0 or 1 to
// the last bit of fp32; the factors of v are held there.
template <int ACT>
__device__ __forceinline__ float activate_grad(float v) {
  if constexpr (ACT == ACT_RELU) return v > 0.f ? 1.f : 0.f;
  if constexpr (ACT == ACT_GELU) {
    const float a = min_abs(v, 20.f);
    float cdf, e;
    normal_cdf_exp(v, a, cdf, e);
    return fmaf(copysignf(a, v) * 0.3989422804f, e, cdf);
  }
  if constexpr (ACT == ACT_GELU_TANH) {
    const float c = copysignf(min_abs(v, 20.f), v);
    float s, slope;
    sigmoid_slope(gelu_tanh_arg(c), s, slope);
    return fmaf(c * slope, fmaf(0.2140644489f, c * c, 1.5957691216f), s);
  }
  if constexpr (ACT == ACT_SILU) {
    const float c = copysignf(min_abs(v, 100.f), v);
    float s, slope;
    sigmoid_slope(c, s, slope);
    return fmaf(c, slope, s);
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

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
// max(x, 0), NaN where x is (fmaxf would drop it).
__device__ __forceinline__ float max_zero(float x) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
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
  if constexpr (ACT == ACT_RELU) return max_zero(v);
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
  if constexpr (ACT == ACT_RELU) return v > 0.f ? 1.f : v <= 0.f ? 0.f : v;
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

// Two elements at once: the packed fp32 operations of sm_100 and later (one issue
// slot for two lanes' worth) carry the polynomial of the normal distribution and
// the products; roundings are those of the single forms.
struct Pair {
  unsigned long long v;
};
__device__ __forceinline__ Pair pair(float lo, float hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(Pair p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p.v));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Pair both(float x) { return pair(x, x); }

// normal_cdf_exp of two elements; a0, a1 as a.
__device__ __forceinline__ void normal_cdf_exp2(float v0, float v1, Pair a, Pair& cdf, Pair& e) {
  float x0, x1;
  unpair(fma2(a, both(0.231641888f), both(1.f)), x0, x1);
  const Pair t = pair(rcp_fast(x0), rcp_fast(x1));
  unpair(mul2(mul2(a, a), both(-0.5f * kLog2e)), x0, x1);
  const float e0 = exp2_fast(x0), e1 = exp2_fast(x1);
  e = pair(e0, e1);
  Pair p = fma2(both(0.5307027145f), t, both(-0.7265760135f));
  p = fma2(p, t, both(0.7107068705f));
  p = fma2(p, t, both(-0.142248368f));
  p = fma2(p, t, both(0.127414796f));
  unpair(fma2(mul2(p, t), pair(-e0, -e1), both(0.5f)), x0, x1);
  cdf = add2(both(0.5f), pair(copysignf(x0, v0), copysignf(x1, v1)));
}

template <int ACT>
__device__ __forceinline__ void activate2(float& v0, float& v1) {
  if constexpr (ACT == ACT_GELU) {
    Pair cdf, e;
    normal_cdf_exp2(v0, v1, pair(min_abs(v0, 20.f), min_abs(v1, 20.f)), cdf, e);
    unpair(mul2(pair(v0, v1), cdf), v0, v1);
  } else {
    v0 = activate<ACT>(v0);
    v1 = activate<ACT>(v1);
  }
}

// Derivatives at v0, v1.
template <int ACT>
__device__ __forceinline__ Pair activate_grad2(float v0, float v1) {
  if constexpr (ACT == ACT_GELU) {
    const float a0 = min_abs(v0, 20.f), a1 = min_abs(v1, 20.f);
    Pair cdf, e;
    normal_cdf_exp2(v0, v1, pair(a0, a1), cdf, e);
    return fma2(mul2(pair(copysignf(a0, v0), copysignf(a1, v1)), both(0.3989422804f)), e, cdf);
  } else {
    return pair(activate_grad<ACT>(v0), activate_grad<ACT>(v1));
  }
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

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
// -min(|x|, m), NaN where x is.
__device__ __forceinline__ float minus_min_abs(float x, float m) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(-fabsf(x)), "f"(-m));
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

// 2 sqrt(2/pi) (v + 0.044715 v^3): the tanh form of gelu is v sigmoid(this).
__device__ __forceinline__ float gelu_tanh_arg(float v) {
  return v * fmaf(0.0713548163f, v * v, 1.5957691216f);
}

// (gelu's other form: pairs only, below.)
template <int ACT>
__device__ __forceinline__ float activate(float v) {
  static_assert(ACT != ACT_GELU, "activate2");
  if constexpr (ACT == ACT_RELU) return max_zero(v);
  if constexpr (ACT == ACT_GELU_TANH) return v * sigmoid(gelu_tanh_arg(v));
  if constexpr (ACT == ACT_SILU) return v * sigmoid(v);
  return v;
}

// The derivative.  Far out (|v| = 20 for gelu's tanh form, 100 for silu) it is 0 or 1 to
// the last bit of fp32; the factors of v are held there.
template <int ACT>
__device__ __forceinline__ float activate_grad(float v) {
  static_assert(ACT != ACT_GELU, "activate_grad2");
  if constexpr (ACT == ACT_RELU) return v > 0.f ? 1.f : max_zero(v);
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
// slot for two lanes' worth) carry gelu's polynomial and the products.
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
__device__ __forceinline__ Pair both(float x) { return pair(x, x); }

// The normal distribution's left half at two places a = -n >= 0 (n = max(-|v|, -20): there
// the exponential is zero):  cdf(-a) = q t e,  e = exp(-a^2/2),  t = 1/(1 + 0.26 a), q a
// polynomial of degree 6 in t.  Its coefficients were fitted to cdf(-a)/e by
// reweighted least squares on [0, 13.2] (beyond it e is below fp32's normal numbers),
// the error's bound the smaller of 1e-7 of 1 and 5e-6 of cdf(-a); it keeps to 0.45 of
// both.  In fp32 cdf(-a) is off by at most 2^-22, and by 2^-16 of itself, most of that the
// rounding of a^2/2 far out.  (One degree less keeps to 1.4e-7 and 7.4e-5; the gradient of
// 4096 x 8192 then takes 33.3 us, 34.1 so, the 8192 x 8192 x 1024 layer 111.3, 112.9.)
__device__ __forceinline__ void normal_left2(Pair n, Pair& q, Pair& t, Pair& e) {
  float x0, x1;
  unpair(fma2(n, both(-0.26f), both(1.f)), x0, x1);
  t = pair(rcp_fast(x0), rcp_fast(x1));
  unpair(mul2(mul2(n, n), both(-0.5f * kLog2e)), x0, x1);
  e = pair(exp2_fast(x0), exp2_fast(x1));
  q = fma2(both(-0.07288757712f), t, both(0.2284436524f));
  q = fma2(q, t, both(-0.1052605882f));
  q = fma2(q, t, both(0.1652158797f));
  q = fma2(q, t, both(0.07392781973f));
  q = fma2(q, t, both(0.1070305929f));
  q = fma2(q, t, both(0.1035301834f));
}

// gelu(v) = max(v, 0) - a cdf(-a), its derivative d = cdf(-a) - a phi(a) for v < 0 and 1 - d
// else: the small side is never a difference from 1.
template <int ACT>
__device__ __forceinline__ void activate2(float& v0, float& v1) {
  if constexpr (ACT == ACT_GELU) {
    const Pair n = pair(minus_min_abs(v0, 20.f), minus_min_abs(v1, 20.f));
    Pair q, t, e;
    normal_left2(n, q, t, e);
    const Pair top = pair(max_zero(v0), max_zero(v1));
    unpair(fma2(mul2(q, t), mul2(e, n), top), v0, v1);
  } else {
    v0 = activate<ACT>(v0);
    v1 = activate<ACT>(v1);
  }
}

// Derivatives at v0, v1.
template <int ACT>
__device__ __forceinline__ Pair activate_grad2(float v0, float v1) {
  if constexpr (ACT == ACT_GELU) {
    const Pair n = pair(minus_min_abs(v0, 20.f), minus_min_abs(v1, 20.f));
    Pair q, t, e;
    normal_left2(n, q, t, e);
    float d0, d1;
    unpair(mul2(fma2(q, t, mul2(n, both(0.3989422804f))), e), d0, d1);
    return pair(v0 < 0.f ? d0 : 1.f - d0, v1 < 0.f ? d1 : 1.f - d1);
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

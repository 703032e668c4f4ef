// Activations and their slopes, for values of 32 bits and for results of 16.
#pragma once
#include "splat_internal.h"

__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }

// The normal distribution's tail T(|z|) = erfc(|z| / sqrt 2) / 2 and its density at z, for
// 16-bit images: T = t P(t) exp(-z^2 / 2), t = 1 / (1 + p |z|), P of degree 4. The
// exponential is the density up to a factor, which goes into the exponent, and its inverse
// into P: the passes with gelu are bound by these instructions.
__device__ __forceinline__ float normal_density(float z) {
  // log2 of exp(-z^2 / 2) / sqrt(2 pi)
  return __builtin_amdgcn_exp2f(__builtin_fmaf(z * -0.72134752f, z, -1.32574806f));
}
template <bool SLOPE>
__device__ __forceinline__ float normal_tail(float z, float density) {
  if constexpr (SLOPE) {
    // For gelu's slope, whose sums may be fp32: Abramowitz and Stegun 7.1.26 (absolute error
    // of erf below 1.5e-7); p and P for erfc(u) at u = |z| / sqrt 2, halved.
    const float t = fast_rcp(__builtin_fmaf(0.23164189f, fabsf(z), 1.0f));
    constexpr float F = 1.25331414f;                                       // sqrt(2 pi) / 2
    float p = __builtin_fmaf(1.061405429f * F, t, -1.453152027f * F);
    p = __builtin_fmaf(p, t, 1.421413741f * F);
    p = __builtin_fmaf(p, t, -0.284496736f * F);
    p = __builtin_fmaf(p, t, 0.254829592f * F);
    return p * (t * density);
  } else {
    // For gelu itself, small where the tail is: a least-maximum fit of the relative error,
    // 3.7e-5 up to 5.7, where fp16 ends, and 6e-4 up to 14, with an absolute error below
    // 1.9e-6: at most 0.08 steps of fp16 and 0.03 of bf16, where the fit above is off by 1.3
    // and 3.7 steps far below zero.
    const float t = fast_rcp(__builtin_fmaf(0.36f, fabsf(z), 1.0f));
    float p = __builtin_fmaf(-0.235040769f, t, 0.601457357f);
    p = __builtin_fmaf(p, t, 0.129469812f);
    p = __builtin_fmaf(p, t, 0.400783777f);
    p = __builtin_fmaf(p, t, 0.356639355f);
    return p * (t * density);
  }
}

// The normal distribution's integral F(z) and its density, to fp32: for fp32 images.
// F = 1/2 + z R(z^2) up to |z| = 1.25, R of degree 5; beyond, the tail t Q(t) exp(-z^2 / 2),
// t = 1 / (1 + 0.3 |z|), Q of degree 8. R and Q are least-maximum fits of the relative
// error of (F - 1/2) / z (9.6e-9) and of exp(z^2 / 2) (1 - F) / t (1.9e-8). Weighted by the
// normal density, gelu's and its slope's error is 3.7e-8 and 3.9e-8 of them, that of
// 0.5 z (1 + erf(z / sqrt 2)) in fp32 3.7e-8 and 4.0e-8, and with 7.1.26
// 8.6e-8 and 1.0e-7; the negative tail, lost to 1 + erf, is kept. Forward and
// backward of 1024x1024x32 fp32: 189 us, 185 with 7.1.26.
__device__ __forceinline__ void normal_f32(float z, float &integral, float &density) {
  const float v = z * z, e = __builtin_amdgcn_exp2f(v * -0.72134752f);
  const float t = fast_rcp(__builtin_fmaf(0.3f, fabsf(z), 1.0f));
  float q = __builtin_fmaf(0.0279918741f, t, -0.0799800679f);
  q = __builtin_fmaf(q, t, 0.045739051f);
  q = __builtin_fmaf(q, t, 0.00935356319f);
  q = __builtin_fmaf(q, t, 0.0617027469f);
  q = __builtin_fmaf(q, t, 0.0869150087f);
  q = __builtin_fmaf(q, t, 0.108938545f);
  q = __builtin_fmaf(q, t, 0.119682059f);
  q = __builtin_fmaf(q, t, 0.119682685f);
  const float tail = q * t * e;
  float r = __builtin_fmaf(-6.80949188e-06f, v, 0.000111041125f);
  r = __builtin_fmaf(r, v, -0.00118383719f);
  r = __builtin_fmaf(r, v, 0.00997228269f);
  r = __builtin_fmaf(r, v, -0.0664902106f);
  r = __builtin_fmaf(r, v, 0.398942262f);
  const float beyond = z < 0.0f ? tail : 1.0f - tail;
  integral = fabsf(z) < 1.25f ? __builtin_fmaf(z, r, 0.5f) : beyond;
  density = e * 0.39894228f;
}

// 1 / (1 + exp(-z)) and its complement to fp32: for results of 32 bits. The exponential of
// -|z| cannot overflow; the rest of its argument's product goes in as a factor, and the
// reciprocal gets a Newton step. Without either, silu at z = -20 is off by 11 roundings and
// at -80 by 40. The complement is 1 - s, whose error offsets that of s in the slope, until
// s is too near one. Forward and backward of 1024x1024x32 fp32: 187 us, 183 without.
__device__ __forceinline__ void logistic_f32(float z, float &s, float &rest) {
  constexpr float L = 1.44269502f, L2 = 1.92596303e-08f;                   // log2(e), and what L lacks
  const float a = fminf(fabsf(z), 150.0f);                                 // the exponential is 0 from 104
  const float hi = a * -L, lo = __builtin_fmaf(a, -L, -hi) - a * L2, e = __builtin_amdgcn_exp2f(hi);
  const float t = __builtin_fmaf(e * lo, 0.693147182f, e), x = 1.0f + t;
  float r = fast_rcp(x);
  r = __builtin_fmaf(__builtin_fmaf(-x, r, 1.0f), r, r);
  const float tr = t * r;
  s = z < 0.0f ? tr : r;
  rest = z > 2.0f ? tr : 1.0f - s;
}

// EXACT: for fp32 images.
template <int ACT, bool EXACT>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (ACT == SPLAT_ACT_RELU) return z < 0.0f ? 0.0f : z;
  if constexpr (ACT == SPLAT_ACT_SILU) {
    if constexpr (EXACT) {
      float t, rest;
      logistic_f32(z, t, rest);
      return z * t;
    }
    return z * fast_rcp(1.0f + __expf(-z));
  }
  if constexpr (ACT == SPLAT_ACT_GELU) {
    if constexpr (EXACT) {
      float a, density;
      normal_f32(z, a, density);
      return z * a;
    }
    const float tail = normal_tail<false>(z, normal_density(z));
    return z * (z < 0.0f ? tail : 1.0f - tail);
  }
  return z;
}

// LIMIT: an infinite z gets the slope's limit, 0 or 1, where the formula is 0 times infinity (a z
// read back from 16 bits may have become infinite there). The factor is held to a range beyond
// which the other one is zero, in one instruction that keeps a finite z's result; a NaN stays one
// by the other factor.
template <bool LIMIT>
__device__ __forceinline__ float slope_factor(float z) {
  return LIMIT ? __builtin_amdgcn_fmed3f(z, -150.0f, 150.0f) : z;
}
template <int ACT, bool EXACT, bool LIMIT = false>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == SPLAT_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == SPLAT_ACT_SILU) {
    if constexpr (EXACT) {
      float t, rest;
      logistic_f32(z, t, rest);
      return t * __builtin_fmaf(slope_factor<LIMIT>(z), rest, 1.0f);
    }
    const float t = fast_rcp(1.0f + __expf(-z));
    return t * __builtin_fmaf(slope_factor<LIMIT>(z), 1.0f - t, 1.0f);
  }
  if constexpr (ACT == SPLAT_ACT_GELU) {
    float a, density;
    if constexpr (EXACT) {
      normal_f32(z, a, density);
      return __builtin_fmaf(slope_factor<LIMIT>(z), density, a);
    }
    density = normal_density(z);
    a = normal_tail<true>(z, density);
    return __builtin_fmaf(slope_factor<LIMIT>(z), density, z < 0.0f ? a : 1.0f - a);
  }
  return 1.0f;
}

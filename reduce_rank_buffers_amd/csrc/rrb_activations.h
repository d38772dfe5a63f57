// The experts' activations and their slopes, in fp32.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/rrb.h"

namespace rrb {

// The sigmoid is v_rcp_f32 of 1 + v_exp_f32: about 2 ulp of fp32, where every
// result is rounded to bf16 (2^16 ulp of fp32) afterwards.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.f + __expf(-x)); }

// Argument of the tanh form's sigmoid: gelu_tanh(x) = x sigmoid(2u),
// u = sqrt(2/pi) (x + 0.044715 x^3).
__device__ __forceinline__ float gelu_2u(float x) {
  return 1.5957691216057308f * (x + 0.044715f * x * x * x);
}

// Phi(x) = erfc(-x / sqrt 2) / 2 with erfc(z) = t P(t) e^(-z^2), t = 1 / (1 +
// 0.38 z), z >= 0: P of degree 6, fitted to the smallest relative error of
// e^(z^2) erfc(z) on 0 <= z <= 10.5, 1.1e-6.  Relative, because x Phi(x) is
// rounded relative to itself however far out x is: with z^2 rounded to fp32
// before the exponential Phi stays within 2^-14 down to x = -13, below which it
// leaves fp32's normal range (a fit of the absolute error, 1.5e-7, was 0.4% off
// at -6 and 1% at -8).  About 17 instructions where the library's erfc takes
// some 100 (it was an eighth of a 4096-deep product's time).
// e receives e^(-x^2 / 2), of which the density is made.
__device__ __forceinline__ float normal_cdf(float x, float &e) {
  const float z = 0.70710678118654752f * fabsf(x);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.38f, z, 1.f));
  float q = __builtin_fmaf(-0.12530328f, t, 0.33559692f);
  q = __builtin_fmaf(q, t, -0.069232336f);
  q = __builtin_fmaf(q, t, 0.24729234f);
  q = __builtin_fmaf(q, t, 0.18082708f);
  q = __builtin_fmaf(q, t, 0.21652655f);
  q = __builtin_fmaf(q, t, 0.21429171f);
  e = __expf(-z * z);
  const float half = 0.5f * q * t * e;
  return x < 0.f ? half : 1.f - half;
}

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if (ACT == RRB_ACT_SILU) return x * sigmoid(x);
  if (ACT == RRB_ACT_GELU) {
    float e;
    return x * normal_cdf(x, e);
  }
  if (ACT == RRB_ACT_GELU_TANH) return x * sigmoid(gelu_2u(x));
  if (ACT == RRB_ACT_RELU) return x < 0.f ? 0.f : x;
  return x;
}

// act(x) and act'(x).
template <int ACT>
__device__ __forceinline__ void activate_grad(float x, float &f, float &df) {
  if (ACT == RRB_ACT_SILU) {
    const float s = sigmoid(x);
    f = x * s;
    df = s * (1.f + x * (1.f - s));
  } else if (ACT == RRB_ACT_GELU) {
    float e;
    const float c = normal_cdf(x, e);
    f = x * c;
    df = c + x * (0.3989422804014327f * e);
  } else if (ACT == RRB_ACT_GELU_TANH) {
    const float s = sigmoid(gelu_2u(x));
    const float t = s * (1.f - s);
    f = x * s;
    // Where the sigmoid is flat the slope's term is 0, also where x^2
    // overflows.
    df = t == 0.f ? s : s + x * t * 1.5957691216057308f * (1.f + 0.134145f * x * x);
  } else if (ACT == RRB_ACT_RELU) {
    f = x < 0.f ? 0.f : x;
    df = x > 0.f ? 1.f : 0.f;
  } else {
    f = x;
    df = 1.f;
  }
}

}  // namespace rrb

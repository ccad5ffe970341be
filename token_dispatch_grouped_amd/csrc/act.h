// The activations of the dense product and their derivatives, in fp32.
//   relu       max(z, 0)
//   gelu       z Phi(z), Phi the normal distribution's
//   gelu_tanh  z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
//   silu       z / (1 + e^-z)
// With 1 + tanh(u) = 2 sigmoid(2u), gelu_tanh and silu are both z sigmoid(z
// (k1 + k2 z^2)). For z < 0, Phi is e^(-z^2 / 2)
// times a polynomial in t = 1 / (1 + 0.307 |z|), for z > 0 one less that: the form
// of Abramowitz and Stegun's 7.1.26 with one term more, whose coefficients were
// fitted to the least relative error on |z| <= 13 (beyond, e^(-z^2 / 2) is no
// normal number): 4e-6, in fp32 with the exponential's own rounding 1e-5 in the tail's
// last decades; their own coefficients, made for the absolute error, are off by
// 1.6e-3 at z = -5 and by more than half a step of bf16 from z = -6.5 on. A
// reciprocal, an exponential and six fused multiply-adds; the derivative shares
// the exponential.
#pragma once

#include "common.h"
#include "moe.h"

namespace moe {

// Calls f with the activation as a constant, so that the choice is made once
// for many values.
template <typename F>
MOE_DEVICE void with_act(int act, F f) {
  switch (act) {
    case MOE_ACT_RELU: f(std::integral_constant<int, MOE_ACT_RELU>{}); break;
    case MOE_ACT_GELU: f(std::integral_constant<int, MOE_ACT_GELU>{}); break;
    case MOE_ACT_GELU_TANH:
    case MOE_ACT_SILU: f(std::integral_constant<int, MOE_ACT_SILU>{}); break;
    default: break;
  }
}

// k1 and k2 of the two sigmoid forms.
struct ActSigmoid {
  float k1, k2;
};
MOE_DEVICE ActSigmoid act_sigmoid(int act) {
  return act == MOE_ACT_GELU_TANH ? ActSigmoid{1.5957691216f, 0.0713548163f} : ActSigmoid{1.f, 0.f};
}

// Phi(z), and e = exp(-z^2 / 2).
MOE_DEVICE float normal_cdf(float z, float &e) {
  e = __builtin_amdgcn_exp2f(z * z * -0.72134752f);  // log2(e) / 2
  const float t = __builtin_amdgcn_rcpf(fmaf(0.30744407f, fabsf(z), 1.f));
  float q = fmaf(t, -0.075989746f, 0.19262688f);
  q = fmaf(t, q, 0.00437243f);
  q = fmaf(t, q, 0.13769136f);
  q = fmaf(t, q, 0.11837258f);
  q = fmaf(t, q, 0.12292468f);
  q *= t * e;
  return z < 0.f ? q : 1.f - q;
}

template <int ACT>
MOE_DEVICE float act_value(float z, const ActSigmoid &s) {
  if constexpr (ACT == MOE_ACT_RELU) {
    return z < 0.f ? 0.f : z;
  } else if constexpr (ACT == MOE_ACT_GELU) {
    float e;
    return z * normal_cdf(z, e);
  } else {
    const float z2 = fminf(z * z, 0x1p127f);  // 0 * inf is no number
    return z * sigmoid_f(z * fmaf(s.k2, z2, s.k1));
  }
}

template <int ACT>
MOE_DEVICE float act_slope(float z, const ActSigmoid &s) {
  if constexpr (ACT == MOE_ACT_RELU) {
    return z > 0.f ? 1.f : 0.f;
  } else if constexpr (ACT == MOE_ACT_GELU) {
    float e;
    const float c = normal_cdf(z, e);
    return fmaf(z * e, 0.39894228f, c);
  } else {
    // sigma + z sigma (1 - sigma) (k1 + 3 k2 z^2)
    const float z2 = fminf(z * z, 0x1p60f);
    const float sg = sigmoid_f(z * fmaf(s.k2, z2, s.k1));
    return fmaf(z * sg * (1.f - sg), fmaf(3.f * s.k2, z2, s.k1), sg);
  }
}

}  // namespace moe

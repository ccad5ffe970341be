// The activations of the dense product and their derivatives, in fp32.
//   relu       max(z, 0)
//   gelu       z Phi(z), Phi the normal distribution's
//   gelu_tanh  z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3)))
//   silu       z / (1 + e^-z)
// With 1 + tanh(u) = 2 sigmoid(2u), gelu_tanh and silu are both z sigmoid(z
// (k1 + k2 z^2)). Phi comes from Abramowitz and Stegun's 7.1.26, erfc(x) =
// (a1 t + ... + a5 t^5) e^(-x^2) with t = 1 / (1 + p x), off by at most 1.5e-7: a
// reciprocal, an exponential and seven fused multiply-adds, whose exponential
// the derivative shares. The results are rounded to bf16 (2^-8), except that
// Phi's own tail, where the formula's error shrinks with e^(-x^2) as well, is
// held to 2e-4 of itself down to z = -5.
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
  e = __expf(-0.5f * z * z);
  const float t = __builtin_amdgcn_rcpf(fmaf(0.23164189f, fabsf(z), 1.f));  // p / sqrt(2)
  float q = fmaf(t, 1.061405429f, -1.453152027f);
  q = fmaf(t, q, 1.421413741f);
  q = fmaf(t, q, -0.284496736f);
  q = fmaf(t, q, 0.254829592f);
  q *= 0.5f * t * e;
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

// act.cuh -- the activations of the linear operators and their derivatives.
//
//   relu       max(z, 0)
//   gelu       z Phi(z),  Phi(z) = (1 + erf(z / sqrt 2)) / 2
//   gelu_tanh  z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2
//            = z sigma(2 sqrt(2/pi) (z + 0.044715 z^3)),  as (1 + tanh u) / 2 = sigma(2 u)
//   silu       z sigma(z)
//
// Two forms of each.  PRECISE (fp32 storage) calls CUDA's functions.  The other
// one (16-bit storage) takes e^x and 1/x from the special-function unit, a few
// fp32 ulp, and Phi from Abramowitz and Stegun, Handbook of Mathematical
// Functions, 7.1.26: erfc(w) = (a1 t + ... + a5 t^5) e^(-w^2), t = 1/(1 + p w),
// whose error in erf is at most 1.5e-7, below 2^-13 of half a step of either
// 16-bit type around 1.  With w = |z| / sqrt 2 its exponential is e^(-z^2/2),
// which is also what Phi' needs, so the derivative costs two products more.
//
// Values that are not numbers pass through every function.  Infinities give
// what the formulas give (minus infinity times 0 is NaN in gelu, gelu_tanh and
// silu); the derivatives take their limits there, 1 and 0.
#pragma once

#include "../csrc/tc_gemm.cuh"

namespace swiglu {

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

template <bool PRECISE>
struct ActMath {
  static __device__ __forceinline__ float sigmoid(float x) {
    if constexpr (PRECISE) {
      const float t = expf(-fabsf(x));
      return x >= 0.0f ? 1.0f / (1.0f + t) : t / (1.0f + t);
    } else {
      return sigmoid_f32(x);
    }
  }
  // Phi(z), and e = e^(-z^2 / 2)
  static __device__ __forceinline__ float phi(float z, float& e) {
    if constexpr (PRECISE) {
      e = expf(-0.5f * z * z);
      return normcdff(z);
    } else {
      float t;
      asm("rcp.approx.f32 %0, %1;" : "=f"(t) : "f"(fmaf(fabsf(z), 0.3275911f * 0.70710678f, 1.0f)));
      e = exp_nonpos_f32(-0.5f * z * z);
      const float p =
          t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f),
                                   0.5f * 1.421413741f), 0.5f * -0.284496736f), 0.5f * 0.254829592f);
      const float q = p * e;  // Phi(-|z|)
      return z >= 0.0f ? 1.0f - q : q;
    }
  }
  static constexpr float TANH_K = 1.5957691216057308f;  // 2 sqrt(2/pi)

  template <int A>
  static __device__ __forceinline__ float value(float z) {
    if constexpr (A == ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (A == ACT_GELU) {
      float e;
      return z * phi(z, e);
    }
    if constexpr (A == ACT_GELU_TANH)
      return z * sigmoid(TANH_K * z * fmaf(0.044715f * z, z, 1.0f));
    if constexpr (A == ACT_SILU) return z * sigmoid(z);
    return z;
  }
  // the derivative; past |z| = 128 its last term is 0 in fp32, and is left out
  // so that no infinity meets that 0
  template <int A>
  static __device__ __forceinline__ float slope(float z) {
    if constexpr (A == ACT_RELU) return z <= 0.0f ? 0.0f : 1.0f;
    const bool in = fabsf(z) < 128.0f;
    if constexpr (A == ACT_GELU) {
      float e;
      const float p = phi(z, e);
      return in ? fmaf(z * e, 0.3989422804014327f, p) : p;
    }
    if constexpr (A == ACT_GELU_TANH) {
      const float p = sigmoid(TANH_K * z * fmaf(0.044715f * z, z, 1.0f));
      return in ? fmaf(z * p * (1.0f - p), TANH_K * fmaf(0.134145f * z, z, 1.0f), p) : p;
    }
    if constexpr (A == ACT_SILU) {
      const float p = sigmoid(z);
      return in ? fmaf(z * p, 1.0f - p, p) : p;
    }
    return 1.0f;
  }
};

// f(std::integral_constant) for the activation chosen at run time: one branch
// around a loop over values instead of one kernel per activation.
template <int A>
struct ActTag {
  static constexpr int value = A;
};
template <class F>
__device__ __forceinline__ void act_switch(int act, F f) {
  switch (act) {
    case ACT_RELU: f(ActTag<ACT_RELU>{}); break;
    case ACT_GELU: f(ActTag<ACT_GELU>{}); break;
    case ACT_GELU_TANH: f(ActTag<ACT_GELU_TANH>{}); break;
    case ACT_SILU: f(ActTag<ACT_SILU>{}); break;
    default: f(ActTag<ACT_NONE>{}); break;
  }
}

}  // namespace swiglu

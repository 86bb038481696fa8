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
// fp32 ulp, and Phi from its tail on either side,
//   Phi(-w) = e^(-w^2/2) (c1 t + ... + c6 t^6),  t = 1 / (1 + 0.412 w),
// the sum being the polynomial in t of the least largest error against
// e^(w^2/2) erfc(w / sqrt 2) / 2 under these bounds (a linear programme over 3000
// points; fp32 evaluation by itself costs about 2e-7): 8e-8 absolutely and 8e-6 of
// the value up to w = 6, where the tail is below any fp16 step, and 8e-4 of the
// value beyond, a fifth of half a bf16 step.  The value z Phi(z) is a product, so
// that what is left of Phi far left stays exact to so many digits; 1 - Phi(-w)
// takes its place right of 0 only.  The exponential is also what Phi' needs, so the
// derivative costs two products more.
// Values go in pairs through fma.rn.f32x2 and the like, as the epilogues that
// apply them are bound by the instructions they issue; for the same reason gelu
// and gelu_tanh let exponentials below 2^-126 become 0 (the forms that keep them
// take four instructions more each, and took the pass over 16384 x 2816 from 54 to
// 68 us).
//
// Values that are not numbers pass through every function but relu's derivative,
// which is 1 for them.  Infinities give
// what the formulas give (minus infinity times 0 is NaN in gelu, gelu_tanh and
// silu); the derivatives take their limits there, 1 and 0.
#pragma once

#include "../csrc/tc_gemm.cuh"

namespace swiglu {

enum Act : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// two fp32 values in one register pair
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
  __device__ __forceinline__ explicit F2(float a) : F2(a, a) {}
  __device__ __forceinline__ explicit F2(uint64_t p) : v(p) {}
  __device__ __forceinline__ void get(float& a, float& b) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
  }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a.v), "l"(b.v), "l"(c.v));
  return F2(r);
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return F2(r);
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a.v), "l"(b.v));
  return F2(r);
}
__device__ __forceinline__ float ex2_ftz(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_ftz(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float ACT_TANH_K = 1.5957691216057308f;  // 2 sqrt(2/pi)

// e = e^(-z^2 / 2) and p0, p1 = Phi(z), for both
__device__ __forceinline__ void phi2(F2 z, float z0, float z1, F2& e, float& p0, float& p1) {
  float a0, a1, q0, q1, r0, r1;
  mul2(mul2(z, z), F2(-0.72134752044448170f)).get(a0, a1);
  e = F2(ex2_ftz(a0), ex2_ftz(a1));
  const F2 t(rcp_ftz(fmaf(fabsf(z0), 0.412f, 1.0f)), rcp_ftz(fmaf(fabsf(z1), 0.412f, 1.0f)));
  // minus the sum
  F2 p = fma2(t, F2(-0.057465021f), F2(0.24332555f));
  p = fma2(t, p, F2(-0.29056361f));
  p = fma2(t, p, F2(-0.050197825f));
  p = fma2(t, p, F2(-0.18221125f));
  p = mul2(fma2(t, p, F2(-0.16288793f)), t);
  mul2(p, e).get(q0, q1);
  fma2(p, e, F2(1.0f)).get(r0, r1);
  p0 = z0 > 0.0f ? r0 : -q0;
  p1 = z1 > 0.0f ? r1 : -q1;
}
// sigma(2 sqrt(2/pi) (z + 0.044715 z^3)); far left 1 / (1 + infinity)
__device__ __forceinline__ F2 sigma_tanh2(F2 z, F2 zz) {
  float u0, u1, d0, d1;
  mul2(mul2(z, F2(-ACT_TANH_K * 1.4426950408889634f)), fma2(zz, F2(0.044715f), F2(1.0f))).get(u0, u1);
  add2(F2(ex2_ftz(u0), ex2_ftz(u1)), F2(1.0f)).get(d0, d1);
  return F2(rcp_ftz(d0), rcp_ftz(d1));
}

// 16-bit storage
template <int A>
__device__ __forceinline__ void act_value2(float& a, float& b) {
  if constexpr (A == ACT_RELU) {
    a = a < 0.0f ? 0.0f : a;
    b = b < 0.0f ? 0.0f : b;
  } else if constexpr (A == ACT_GELU) {
    const F2 z(a, b);
    F2 e(0.0f);
    float p0, p1;
    phi2(z, a, b, e, p0, p1);
    mul2(z, F2(p0, p1)).get(a, b);
  } else if constexpr (A == ACT_GELU_TANH) {
    const F2 z(a, b);
    mul2(z, sigma_tanh2(z, mul2(z, z))).get(a, b);
  } else if constexpr (A == ACT_SILU) {
    a = silu_f32(a);
    b = silu_f32(b);
  }
}
// the derivatives; past |z| = 128 their last term is 0 in fp32, and is left out so
// that no infinity meets that 0
template <int A>
__device__ __forceinline__ void act_slope2(float& a, float& b) {
  if constexpr (A == ACT_RELU) {
    a = a <= 0.0f ? 0.0f : 1.0f;
    b = b <= 0.0f ? 0.0f : 1.0f;
  } else if constexpr (A == ACT_GELU) {
    const F2 z(a, b);
    F2 e(0.0f);
    float p0, p1, f0, f1;
    phi2(z, a, b, e, p0, p1);
    mul2(mul2(z, e), F2(0.3989422804014327f)).get(f0, f1);
    a = p0 + (fabsf(a) < 128.0f ? f0 : 0.0f);
    b = p1 + (fabsf(b) < 128.0f ? f1 : 0.0f);
  } else if constexpr (A == ACT_GELU_TANH) {
    const F2 z(a, b), zz = mul2(z, z), p = sigma_tanh2(z, zz);
    float p0, p1, f0, f1;
    p.get(p0, p1);
    const F2 rest = mul2(mul2(z, p), fma2(p, F2(-1.0f), F2(1.0f)));
    mul2(rest, fma2(zz, F2(ACT_TANH_K * 0.134145f), F2(ACT_TANH_K))).get(f0, f1);
    a = p0 + (fabsf(a) < 128.0f ? f0 : 0.0f);
    b = p1 + (fabsf(b) < 128.0f ? f1 : 0.0f);
  } else if constexpr (A == ACT_SILU) {
    const float p0 = sigmoid_f32(a), p1 = sigmoid_f32(b);
    a = fabsf(a) < 128.0f ? fmaf(a * p0, 1.0f - p0, p0) : p0;
    b = fabsf(b) < 128.0f ? fmaf(b * p1, 1.0f - p1, p1) : p1;
  } else {
    a = b = 1.0f;
  }
}

// fp32 storage: CUDA's functions
struct ActPrecise {
  static __device__ __forceinline__ float sigmoid(float x) {
    const float t = expf(-fabsf(x));
    return x >= 0.0f ? 1.0f / (1.0f + t) : t / (1.0f + t);
  }
  template <int A>
  static __device__ __forceinline__ float value(float z) {
    if constexpr (A == ACT_RELU) return z < 0.0f ? 0.0f : z;
    if constexpr (A == ACT_GELU) return z * normcdff(z);
    if constexpr (A == ACT_GELU_TANH) return z * sigmoid(ACT_TANH_K * z * fmaf(0.044715f * z, z, 1.0f));
    if constexpr (A == ACT_SILU) return z * sigmoid(z);
    return z;
  }
  template <int A>
  static __device__ __forceinline__ float slope(float z) {
    if constexpr (A == ACT_RELU) return z <= 0.0f ? 0.0f : 1.0f;
    const bool in = fabsf(z) < 128.0f;
    if constexpr (A == ACT_GELU) {
      const float p = normcdff(z);
      return in ? fmaf(z * expf(-0.5f * z * z), 0.3989422804014327f, p) : p;
    }
    if constexpr (A == ACT_GELU_TANH) {
      const float p = sigmoid(ACT_TANH_K * z * fmaf(0.044715f * z, z, 1.0f));
      return in ? fmaf(z * p * (1.0f - p), ACT_TANH_K * fmaf(0.134145f * z, z, 1.0f), p) : p;
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

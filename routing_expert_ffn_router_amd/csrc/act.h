// Activations of the experts' linear layers and their slopes.
//   silu       z s(z), s(z) = 1 / (1 + e^-z)         slope s (1 + z (1 - s))
//   gelu       z P(z), P the normal distribution      slope P(z) + z e^(-z^2 / 2) / sqrt(2 pi)
//   gelu_tanh  z s(u), u = sqrt(8 / pi) (z + 0.044715 z^3): (1 + tanh(u / 2)) / 2 = s(u)
//                                                     slope s + z s (1 - s) u'
#pragma once

#include "common.h"

namespace moe {

// moe_activation
constexpr int kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4;

constexpr float kSqrt8OverPi = 1.59576912160573071f;

// s(u), and s (1 - s) without the difference, which would leave 2^-24 of 1 in it.  (The hardware's
// exponential and reciprocal: a t within (|u| + 2) 2^-24 of itself, t |u| < 0.4.)
struct Sigmoid {
  float s, slope;
};
__device__ inline Sigmoid sigmoid_f32(float u) {
  const float t = __expf(-fabsf(u)), r = __builtin_amdgcn_rcpf(1.0f + t);
  return Sigmoid{u < 0.f ? t * r : r, t * r * r};
}

// The normal distribution P(z), and e^(-z^2 / 2).  P(-|z|) = e^(-z^2 / 2) Q(t), t = 1 / (1 + a |z|), Q a
// polynomial without constant term (the form of Hastings' approximations) fitted to the least
// largest relative error, 1.2e-7 for |z| < 15; evaluated in fp32 P is within 5 2^-24, and relative to
// itself within 1.4e-6 for z > -6.  (The library's erfc and exp took 234 us where this takes 150: the
// slopes of 8191 x 14336 bf16 values.  fp32 values take the same form, and its error with it.)
struct Normal {
  float p, density;  // density without its 1 / sqrt(2 pi)
};
__device__ inline Normal normal_f32(float z) {
  const float t = __builtin_amdgcn_rcpf(fmaf(0.30582368f, fabsf(z), 1.0f));
  const float e = __expf(-0.5f * z * z);
  float q = 0.036402709f;
  q = fmaf(q, t, -0.15044943f);
  q = fmaf(q, t, 0.17941881f);
  q = fmaf(q, t, -0.032952356f);
  q = fmaf(q, t, 0.1185694f);
  q = fmaf(q, t, 0.10433945f);
  q = fmaf(q, t, 0.12269732f);
  q = fmaf(q, t, 0.1219741f);
  q *= t * e;
  return Normal{z < 0.f ? q : 1.0f - q, e};
}

template <int ACT>
__device__ inline float act_value(float z) {
  if constexpr (ACT == kActRelu) return z > 0.f || z != z ? z : 0.f;
  if constexpr (ACT == kActSilu) return z * sigmoid_f32(z).s;
  if constexpr (ACT == kActGelu) return z * normal_f32(z).p;
  if constexpr (ACT == kActGeluTanh)
    return z * sigmoid_f32(kSqrt8OverPi * fmaf(0.044715f * z * z, z, z)).s;
  return z;
}

// The slope at z, a NaN's is NaN.  Past +-most it is exactly 0 or 1 in fp32, and z is held there so
// that no product of a large z and a vanishing factor is formed.
__device__ inline float within(float z, float most) {
  return z > most ? most : z < -most ? -most : z;
}
template <int ACT>
__device__ inline float act_slope(float z) {
  if constexpr (ACT == kActSilu) z = within(z, 110.f);
  if constexpr (ACT == kActGelu || ACT == kActGeluTanh) z = within(z, 15.f);
  if constexpr (ACT == kActRelu) return z > 0.f ? 1.f : z != z ? z : 0.f;
  if constexpr (ACT == kActSilu) {
    const Sigmoid p = sigmoid_f32(z);
    return fmaf(z, p.slope, p.s);
  }
  if constexpr (ACT == kActGelu) {
    const Normal n = normal_f32(z);
    return fmaf(0.398942280401432678f * z, n.density, n.p);
  }
  if constexpr (ACT == kActGeluTanh) {
    const Sigmoid p = sigmoid_f32(kSqrt8OverPi * fmaf(0.044715f * z * z, z, z));
    return fmaf(z * p.slope, kSqrt8OverPi * fmaf(3.f * 0.044715f * z, z, 1.f), p.s);
  }
  return 1.f;
}

// f(IntC-like tag of the activation)
template <class F>
inline hipError_t with_act(int act, F&& f) {
  switch (act) {
    case kActNone: return f(std::integral_constant<int, kActNone>{});
    case kActRelu: return f(std::integral_constant<int, kActRelu>{});
    case kActSilu: return f(std::integral_constant<int, kActSilu>{});
    case kActGelu: return f(std::integral_constant<int, kActGelu>{});
    default: return f(std::integral_constant<int, kActGeluTanh>{});
  }
}

}  // namespace moe

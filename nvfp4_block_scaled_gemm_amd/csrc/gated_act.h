// Activations of the gated blocks (gfx950 only): act(g) = g * sigma(z(g)) with
//
//   silu  z = g
//   gelu  z = 2 sqrt(2 / pi) (g + 0.044715 g^3)    (the tanh form: 1 + tanh(t) = 2 sigma(2 t))
//
// and act'(g) = sigma + act(g) (1 - sigma) z'.  With t = exp(-|z|), which never
// overflows: the larger of sigma and 1 - sigma is 1 / (1 + t), the smaller t / (1 + t),
// so nothing cancels on either side.  Both keep their bits down to the least normal
// number and go on to the least subnormal one; |z| is cut at kEdge, where the smaller is
// less than half of that and rounds to 0.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {

constexpr int kSilu = 0, kGelu = 1;

struct Sigma {
  float sigma, turn;  // sigma(z) and (1 - sigma) z': act = g sigma, act' = sigma + act turn
};

// exp(x) for -110 < x <= 0 within about 1.5 ulp: the hardware's exp2 takes the rounded
// product, and what the rounding left out is applied to its result.  exp2 has no results
// below the normal numbers: there it takes t + 32 (exact, since it is nearer to zero), and
// the result is scaled back.
__device__ __forceinline__ float exp_near(float x) {
#pragma clang fp contract(off)  // t + 32 is that of the rounded t, whose error r holds
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.925963033500e-8f;
  constexpr float kLn2 = 0.69314718055994530942f;
  const float t = x * kLog2e;
  const float r = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
  const bool low = t < -100.0f;
  const float e = __builtin_amdgcn_exp2f(t + (low ? 32.0f : 0.0f)) * __builtin_fmaf(r, kLn2, 1.0f);
  return e * (low ? 0x1p-32f : 1.0f);
}

template <int ACT>
__device__ __forceinline__ Sigma sigma_of(float g) {
  constexpr float kA = 1.59576912160573071176f, kB = 0.044715f;  // 2 sqrt(2 / pi)
  constexpr float kEdge = 105.0f;
  float z = g, slope = 1.0f;
  if constexpr (ACT == kGelu) {
    // 8: past the edge, and z' stays finite
    const float s = __builtin_fminf(kB * g * g, 8.0f);
    z = kA * __builtin_fmaf(g, s, g);
    slope = __builtin_fmaf(3.0f * kA, s, kA);
  }
  // (a NaN is lost in the minima, not in the product with g)
  const float t = exp_near(-__builtin_fminf(__builtin_fabsf(z), kEdge));
  // 1 / (1 + t), with what the sum rounds off and what the hardware's reciprocal leaves put
  // back: one rounding instead of three
  const float sum = 1.0f + t, near = __builtin_amdgcn_rcpf(sum);
  const float left = __builtin_fmaf(-(t - (sum - 1.0f)), near, __builtin_fmaf(-sum, near, 1.0f));
  const float large = __builtin_fmaf(near, left, near), small = t * large;
  return {z >= 0.0f ? large : small, slope * (z >= 0.0f ? small : large)};
}

// act(g) * u of eight elements; `act` is the same for a whole launch.
__device__ __forceinline__ void gated8(int act, const float* g, const float* u, float* v) {
  if (act == kGelu) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = g[e] * sigma_of<kGelu>(g[e]).sigma * u[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = g[e] * sigma_of<kSilu>(g[e]).sigma * u[e];
  }
}

}  // namespace nvfp4

// Activations of the gated blocks (gfx950 only): act(g) = g * sigma(z(g)) with
//
//   silu  z = g
//   gelu  z = 2 sqrt(2 / pi) (g + 0.044715 g^3)    (the tanh form: 1 + tanh(t) = 2 sigma(2 t))
//
// and act'(g) = sigma + g sigma (1 - sigma) z'.  With e = exp(-z): sigma = 1 / (1 + e)
// and 1 - sigma = e sigma, which loses nothing where sigma is near 1.  Beyond
// |g| = kEdge (z around 87) sigma is 0 or 1 in fp32; g is cut there inside z, z' and
// their product, so that no finite g makes an infinity times a zero.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {

constexpr int kSilu = 0, kGelu = 1;

struct Sigma {
  float sigma, slope;  // sigma(z), and 1 + g z' (1 - sigma): act' = sigma * slope
};

// exp(x) for |x| < 100 within about 1.5 ulp: the hardware's exp2 takes the rounded
// product, and what the rounding left out is applied to its result.
__device__ __forceinline__ float exp_near(float x) {
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.925963033500e-8f;
  constexpr float kLn2 = 0.69314718055994530942f;
  const float t = x * kLog2e;
  const float r = __builtin_fmaf(x, kLog2eLow, __builtin_fmaf(x, kLog2e, -t));
  return __builtin_amdgcn_exp2f(t) * __builtin_fmaf(r, kLn2, 1.0f);
}

template <int ACT>
__device__ __forceinline__ Sigma sigma_of(float g) {
  constexpr float kA = 1.59576912160573071176f, kB = 0.044715f;  // 2 sqrt(2 / pi)
  constexpr float kEdge = ACT == kGelu ? 9.9f : 87.0f;
  const float c = fminf(fmaxf(g, -kEdge), kEdge);
  float z = c, zc = c;  // z and c z'
  if constexpr (ACT == kGelu) {
    const float s = kB * c * c;
    z = kA * __builtin_fmaf(c, s, c);
    zc = kA * __builtin_fmaf(c, 3.0f * s, c);
  }
  const float e = exp_near(-z);
  const float inv = __builtin_amdgcn_rcpf(1.0f + e);
  // 0 * g: a NaN stays one
  return {g > -kEdge ? inv : 0.0f * g, __builtin_fmaf(zc, e * inv, 1.0f)};
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

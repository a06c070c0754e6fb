// The gated unit act(g) * u in fp32, and its derivatives.
#pragma once

#include "ffn_internal.h"

namespace muon {

struct FfnSlope { float act, slope; };   // act(g) and its derivative

// kFast: for results that are rounded to bf16, whose exponentials and quotients may be off
// by 2^-20 of themselves, and by 2^-24 for each unit of the exponential's argument.  An
// overflowing e^-g makes the sigmoid 0.
template <bool kFast, int kAct> __device__ __forceinline__ FfnSlope ffn_act(float g) {
  if constexpr (kAct == kFfnSilu) {
    const float s = kFast ? __fdividef(1.f, 1.f + __expf(-g)) : 1.f / (1.f + expf(-g));
    const float a = g * s;
    return {a, fmaf(a, 1.f - s, s)};
  } else if constexpr (kFast) {
    // Phi(-|g|) = e^(-g^2 / 2) t P(t) with t = 1 / (1 + 0.2644 |g|) and P of degree 6, fitted
    // for the least largest relative error over |g| <= 14 (5.7e-7; by reweighted least squares):
    // the tail, where g Phi(g) is small, is as exact as the rest.  Its exponential is also the
    // density's.
    const float x = fabsf(g), e = __expf(-0.5f * g * g), t = __fdividef(1.f, fmaf(0.2644f, x, 1.f));
    float q = fmaf(-0.06866673f, t, 0.2000890f);
    q = fmaf(q, t, -0.07218982f);
    q = fmaf(q, t, 0.14611025f);
    q = fmaf(q, t, 0.08149237f);
    q = fmaf(q, t, 0.10781986f);
    q = fmaf(q, t, 0.10534476f);
    const float tail = q * t * e, cdf = g < 0.f ? tail : 1.f - tail;
    return {g * cdf, fmaf(g * 0.39894228f, e, cdf)};
  } else {
    const float cdf = 0.5f * erfcf(-0.70710678f * g);
    return {g * cdf, fmaf(g * 0.39894228f, expf(-0.5f * g * g), cdf)};
  }
}
template <bool kFast> __device__ __forceinline__ FfnSlope ffn_act(float g, int activation) {
  return activation == kFfnSilu ? ffn_act<kFast, kFfnSilu>(g) : ffn_act<kFast, kFfnGelu>(g);
}

}  // namespace muon

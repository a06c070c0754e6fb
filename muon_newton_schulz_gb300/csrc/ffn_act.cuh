// The gated unit act(g) * u in fp32, and its derivatives.
#pragma once

#include "ffn_internal.h"

namespace muon {

struct FfnSlope { float act, slope; };   // act(g) and its derivative

// kFast: for results that are rounded to bf16, where exponentials and quotients
// within 2^-20 of themselves are enough.  An overflowing e^-g makes the sigmoid 0.
template <bool kFast, int kAct> __device__ __forceinline__ FfnSlope ffn_act(float g) {
  if constexpr (kAct == kFfnSilu) {
    const float s = kFast ? __fdividef(1.f, 1.f + __expf(-g)) : 1.f / (1.f + expf(-g));
    const float a = g * s;
    return {a, fmaf(a, 1.f - s, s)};
  } else if constexpr (kFast) {
    // Phi(-|g|) = erfc(|g| / sqrt 2) / 2 by the rational approximation 7.1.26 of
    // Abramowitz and Stegun, off by at most 1.5e-7 in erfc; its e^(-g^2 / 2) is also
    // the density's
    const float x = fabsf(g), e = __expf(-0.5f * g * g), t = __fdividef(1.f, fmaf(0.3275911f * 0.70710678f, x, 1.f));
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    const float tail = 0.5f * q * t * e, cdf = g < 0.f ? tail : 1.f - tail;
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

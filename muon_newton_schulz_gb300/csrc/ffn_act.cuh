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
  } else {
    const float cdf = 0.5f * erfcf(-0.70710678f * g);
    const float pdf = 0.39894228f * (kFast ? __expf(-0.5f * g * g) : expf(-0.5f * g * g));
    return {g * cdf, fmaf(g, pdf, cdf)};
  }
}
template <bool kFast> __device__ __forceinline__ FfnSlope ffn_act(float g, int activation) {
  return activation == kFfnSilu ? ffn_act<kFast, kFfnSilu>(g) : ffn_act<kFast, kFfnGelu>(g);
}

}  // namespace muon

// softcap.cuh -- capped scores of the paged attentions.
#pragma once
#include "common.cuh"

namespace gqa {

// cap * tanh(s / cap), to 2^-19 of itself (cap_out = cap, cap_inv = 1 / cap).  With u = s / cap
// and |u| >= 1/4, tanh u = 1 - 2 / (exp(2 u) + 1), whose error of up to 1.6 * 2^-22 (the
// exponential's and the reciprocal's) is 2^-19 of it at 1/4 and would be any multiple of it nearer
// to 0.  There the series u - u^3 / 3 + 2 u^5 / 15 - 17 u^7 / 315 + 62 u^9 / 2835 is taken, 2^-26
// off at 1/4, as s (1 + u^2 (...)): under a cap far above the scores u may be denormal, and s stays
// as it is.  (Both are formed and one is chosen: the one-token attention's window case with its cap
// 50 109.7 us, 48 x 16001 over E4M3 pages with cap 30 128.7 us; 109.1 and 127.2 with the exponential
// alone, 115.5 and 134.5 with tanhf.)
__device__ __forceinline__ float capped(float s, float cap_out, float cap_inv) {
  const float u = s * cap_inv, w = u * u;
  const float series = fmaf(fmaf(fmaf(62.f / 2835.f, w, -17.f / 315.f), w, 2.f / 15.f), w, -1.f / 3.f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fast_exp2(u * 2.8853900817779268f) + 1.f));
  const float far = fmaf(-2.f * cap_out, r, cap_out);
  return fabsf(u) < 0.25f ? fmaf(s * w, series, s) : far;
}

}  // namespace gqa

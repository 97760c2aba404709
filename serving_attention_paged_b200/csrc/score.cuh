// Scores with options (pa_attention_options): tanh cap and distance bias,
// in base 2, shared by the decode and prefill kernels.
#pragma once

#include <cmath>

#include "common.cuh"
#include "pa_internal.h"

namespace pa {

// tanh(y).  |y| <= 1/2: y times a polynomial in y^2, a minimax fit of relative
// error (2.8e-8 with these fp32 coefficients) computed for this library; so
// a small score keeps its relative accuracy under any cap.  Beyond:
// 1 - 2 / (e^(2y) + 1), whose absolute error is a few fp32 steps of 1 and
// which saturates by itself (e^(2y) = inf or 0).
constexpr float kTanhSmall = 0.5f;
__device__ __forceinline__ float tanh_score(float y) {
  const float u = y * y;
  float p = fmaf(0.017135007306933403f, u, -0.05298607423901558f);
  p = fmaf(p, u, 0.13324779272079468f);
  p = fmaf(p, u, -0.3333306908607483f);
  p = fmaf(p, u, 1.0f);
  const float e = fast_exp2(y * (2.f * kLog2e));
  const float big = 1.f - __fdividef(2.f, e + 1.f);
  return fabsf(y) <= kTanhSmall ? y * p : big;
}

// tanh of a pair with |y| <= 1, on the FMA pipe with packed arithmetic: the
// same kind of fit, degree 6 in y^2, relative error 7e-8.
__device__ __forceinline__ float2 tanh_poly2(float2 y) {
  const float2 u = __fmul2_rn(y, y);
  float2 p = __ffma2_rn(make_float2(0.0010410224786028266f, 0.0010410224786028266f), u,
                        make_float2(-0.006203378550708294f, -0.006203378550708294f));
  p = __ffma2_rn(p, u, make_float2(0.020289979875087738f, 0.020289979875087738f));
  p = __ffma2_rn(p, u, make_float2(-0.05345702916383743f, -0.05345702916383743f));
  p = __ffma2_rn(p, u, make_float2(0.13325203955173492f, 0.13325203955173492f));
  p = __ffma2_rn(p, u, make_float2(-0.33332839608192444f, -0.33332839608192444f));
  p = __ffma2_rn(p, u, make_float2(0.9999999403953552f, 0.9999999403953552f));
  return __fmul2_rn(y, p);
}

// The options of a run as the kernels take them.  With a cap the kernels'
// score_scale is sm_scale / cap (times k_scale), so that cap_out *
// tanh(scaled score) is the capped score in base 2.
struct ScoreArgs {
  const float* slopes;  // [Hq] or null: per unit of distance
  float cap_out;        // cap * log2(e), 0 = no cap
};

// From the caller's options; score_scale is the run's sm_scale * log2(e)
// (times k_scale) and becomes what the kernels multiply with.
inline void set_score_args(const pa_attention_options& o, ScoreArgs* a, float* score_scale) {
  a->slopes = o.alibi_slopes;
  a->cap_out = 0.f;
  if (o.logit_cap > 0.f) {
    a->cap_out = o.logit_cap * kLog2e;
    *score_scale /= a->cap_out;
  }
}

// cap_out * tanh(score_scale * x) for raw scores |x| <= small, as x times a
// polynomial in x^2 with the powers of score_scale and the cap folded in: a
// minimax fit of tanh(y) / y, degree 4 in y^2 on |y| <= 1/2, relative error
// 1.3e-8, below fp32's rounding.  (Degree 3 is one operation less and 5.4e-7
// off, all one way for small scores: 9e-4 of a score of 1,600; on |y| <= 5/16
// it is right, but scores beyond take the longer polynomial: 376 us a prefill
// where degree 4 took 332.)  |x| <= mid: |score_scale * x| <= 1.
struct CapPoly {
  float k[5], small, mid;
};
inline CapPoly make_cap_poly(const ScoreArgs& a, float score_scale) {
  constexpr double c[5] = {0.9999999868759589, -0.3333306944690451, 0.13324780408767786,
                           -0.05298614099119273, 0.017135126142517644};
  CapPoly out{};
  const double s = score_scale;
  double f = double(a.cap_out) * s;
  for (int i = 0; i < 5; ++i, f *= s * s) out.k[i] = float(c[i] * f);
  const double r = s < 0 ? -s : s;
  double reach = kTanhSmall;
  if (std::fabs(out.k[4]) < 0x1p-120f) {  // a huge cap: the last terms leave fp32's range, but
    out.k[3] = out.k[4] = 0.f;            // up to 2^-5 of it they are below 1e-10 of the score
    reach = 0x1p-5;
  }
  const bool finite = std::isfinite(out.k[0]) && std::isfinite(out.k[4]);
  out.small = finite && r > 0 ? float(reach / r) : -1.f;
  out.mid = r > 0 ? float(1.0 / r) : INFINITY;
  return out;
}

// The base-2 score of a scaled dot product x: capped, then biased by
// -slope2 * distance (slope2 = slope * log2(e), 0 without slopes).
__device__ __forceinline__ float final_score(float x, const ScoreArgs& a, float slope2,
                                             float distance) {
  if (a.cap_out > 0.f) x = a.cap_out * tanh_score(x);
  return fmaf(-slope2, distance, x);
}

}  // namespace pa

// Score arithmetic shared by the tensor-core kernels of the attention with modified scores.
//
// Scores are kept in units of log2: s2 = s log2(e), so that P = 2^(s2 - m).  With
// x = scale q.k / cap the capped score is cap tanh(x).  Where all of a warp's |x| are small,
// tanh(x) = x times a polynomial in x^2, fitted for the least largest relative error on the
// interval (a linear program over points of it forms them again: 3.9e-7 and 5.3e-7 at best): degree 2
// up to 1/4 (4.0e-7) and degree 3 up to 1/2 (5.4e-7); the scale and the cap are folded into the
// coefficients, so a score costs two or three multiply-adds more than an uncapped one.
// Elsewhere tanh(x) = 1 - 2 / (1 + e^2x), exact at saturation, for two more operations of the
// exponential unit.  (tanh.approx is one instruction, but off by 2^-11: 0.02 of a score at a
// cap of 50.)
#pragma once
#include "score_common.cuh"
#include "tc_common.cuh"

namespace oomb {

constexpr float kTanhEdge2 = 0.25f, kTanhEdge3 = 0.5f;  // |x| up to which degree 2 and 3 hold

struct CapConst {
  float poly2[3], poly3[4];  // tanh(x) = S (poly[0] + poly[1] S^2 + ...), S the raw dot product
  float edge2, edge3;        // |S| up to which they hold
  float arg;                 // 2 scale log2(e) / cap:  e^2x = 2^(arg S)
  float cap2;                // cap log2(e)
};

inline CapConst make_cap(float cap, float scale) {
  static const double kFit2[3] = {0.9999996043444983, -0.33321908225036645, 0.1284161343106791};
  static const double kFit3[4] = {0.9999994557709395, -0.3332631793593743, 0.13190296603150334, -0.04440222612595766};
  CapConst c = {};
  if (!(cap > 0.f)) return c;
  const double k = (double)scale / (double)cap, ak = k < 0 ? -k : k;
  double p = k;
  for (int i = 0; i < 4; ++i, p *= k * k) {
    if (i < 3) c.poly2[i] = (float)(kFit2[i] * p);
    c.poly3[i] = (float)(kFit3[i] * p);
  }
  c.edge2 = ak > 0.0 ? (float)(kTanhEdge2 / ak) : INFINITY;
  c.edge3 = ak > 0.0 ? (float)(kTanhEdge3 / ak) : INFINITY;
  if (ak > 1e4) c.edge2 = c.edge3 = -1.f;  // coefficients (ak^7) out of fp32's range: the wide form only
  c.arg = (float)(2.0 * k * 1.4426950408889634);
  c.cap2 = (float)((double)cap * 1.4426950408889634);
  return c;
}

enum TanhForm { kDegree2, kDegree3, kWide };

template <TanhForm F>
__device__ __forceinline__ float tanh_of(float S, const CapConst& c) {
  if constexpr (F == kWide) return fmaf(-2.f, rcp_approx(1.f + ex2_approx(c.arg * S)), 1.f);
  const float z = S * S;
  if constexpr (F == kDegree2) return S * fmaf(fmaf(c.poly2[2], z, c.poly2[1]), z, c.poly2[0]);
  return S * fmaf(fmaf(fmaf(c.poly3[3], z, c.poly3[2]), z, c.poly3[1]), z, c.poly3[0]);
}

}  // namespace oomb

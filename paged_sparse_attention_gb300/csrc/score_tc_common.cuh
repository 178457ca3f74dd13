// Score arithmetic shared by the tensor-core kernels of the attention with modified scores.
//
// Scores are kept in units of log2: s2 = s log2(e), so that P = 2^(s2 - m).  For |x| <= 1,
// x = scale q.k / cap, the capped score is S times a polynomial in S^2 (S the raw dot
// product, the cap and the scale folded into the coefficients): tanh(x) / x as a polynomial
// of degree 5 in x^2 fitted on [0, 1] for the least relative error (5.9e-7).  That is seven
// packed multiply-adds for two scores and leaves the exponential unit, which bounds these
// kernels, to the softmax; tanh.approx would be one instruction but is off by 2^-11, half a
// unit of the score at a cap of 1000.  Outside, tanh(x) = 1 - 2 / (1 + e^2x), two operations
// of that unit each, exact at saturation.
#pragma once
#include "score_common.cuh"
#include "tc_common.cuh"

namespace oomb {

constexpr int kTanhTerms = 6;

struct CapConst {
  float poly[kTanhTerms];  // s2 = S (poly[0] + poly[1] S^2 + ...), |S| <= s_small
  float s_small;           // |S| up to which the polynomial holds
  float arg;               // 2 scale log2(e) / cap:  e^2x = 2^(arg S)
  float cap2;              // cap log2(e)
  float unit;              // scale / cap:  x = unit S
  float poly_t[kTanhTerms];  // tanh(x) = S (poly_t[0] + poly_t[1] S^2 + ...)
};

inline CapConst make_cap(float cap, float scale) {
  static const double kFit[kTanhTerms] = {0.9999994135992796,   -0.333290423785063,  0.1328143388055857,
                                          -0.05160567399853968, 0.016743115061095788, -0.003067060325955233};
  CapConst c = {};
  if (!(cap > 0.f)) return c;
  const double k = (double)scale / (double)cap;
  double p = k;
  for (int i = 0; i < kTanhTerms; ++i, p *= k * k) {
    c.poly[i] = (float)(kFit[i] * p * (double)cap * 1.4426950408889634);
    c.poly_t[i] = (float)(kFit[i] * p);
  }
  c.s_small = k != 0.0 ? (float)(1.0 / (k < 0 ? -k : k)) : INFINITY;
  c.arg = (float)(2.0 * k * 1.4426950408889634);
  c.cap2 = (float)((double)cap * 1.4426950408889634);
  c.unit = (float)k;
  return c;
}

// 1 / x to one unit in the last place or so (x >= 1 here; infinity gives 0).
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float tanh_wide(float S, const CapConst& c) {
  return fmaf(-2.f, rcp_approx(1.f + ex2_approx(c.arg * S)), 1.f);
}
__device__ __forceinline__ float tanh_small(float S, const CapConst& c) {
  const float z = S * S;
  float p = c.poly_t[kTanhTerms - 1];
#pragma unroll
  for (int i = kTanhTerms - 2; i >= 0; --i) p = fmaf(p, z, c.poly_t[i]);
  return S * p;
}
__device__ __forceinline__ float capped(float S, const CapConst& c) {
  if (fabsf(S) <= c.s_small) {
    const float z = S * S;
    float p = c.poly[kTanhTerms - 1];
#pragma unroll
    for (int i = kTanhTerms - 2; i >= 0; --i) p = fmaf(p, z, c.poly[i]);
    return S * p;
  }
  return c.cap2 * tanh_wide(S, c);
}

}  // namespace oomb

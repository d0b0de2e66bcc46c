// fpx_rule.cuh -- the score rule (cap, distance bias, key spans) as the kernels see it.
#pragma once

#include "fpx_common.cuh"

namespace fpx {

struct RuleDesc {
  float softcap = 0.f;            // 0: none
  int window = 0;                 // 0: none
  const float* slopes = nullptr;  // [hq] or null
  const int32_t* lo = nullptr;    // [query tokens] or null (both or neither)
  const int32_t* hi = nullptr;
};

struct KeySpan {
  int lo, hi;  // inclusive; lo > hi: no key
};

// Keys of a sequence of `n` tokens that the query at position i, row `tok` of Q, sees.
__device__ __forceinline__ KeySpan rule_span(const RuleDesc& r, int64_t tok, int i, int n) {
  KeySpan s;
  s.lo = r.lo ? r.lo[tok] : 0;
  s.hi = r.lo ? r.hi[tok] : i;
  if (r.window > 0) {
    const int64_t first = static_cast<int64_t>(i) - r.window + 1;
    if (first > s.lo) s.lo = static_cast<int>(first);
  }
  if (s.lo < 0) s.lo = 0;
  if (s.hi > n - 1) s.hi = n - 1;
  return s;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(x) = 1 - 2 / (1 + 2^(2 x log2 e)): absolute error at most 4e-7 for any x (with e = 2^(..), the
// quotient q = 2 / (1 + e) <= 2 has the relative errors 2^-22 e / (1 + e) of ex2, 2^-24 of the sum and
// 2^-23 of rcp; the exponent's own rounding, |2 x log2 e| 2^-24, is damped by e / (1 + e) or by q, and
// 2^-25 for the result).  Enough for a score where x is not small, as the error is then small
// against the score too.
__device__ __forceinline__ float tanh_ex2(float x) {
  return fmaf(-2.f, rcp_approx(1.f + ex2_approx(x * 2.8853900817779268f)), 1.f);
}
// The same with a small relative error for small x (scores far below the cap, whatever the cap): the
// series to x^7 below 1/5, its next term 6e-8 of the sum there.
__device__ __forceinline__ float tanh_any(float x) {
  const float u = x * x;
  const float p = fmaf(fmaf(fmaf(-17.f / 315.f, u, 2.f / 15.f), u, -1.f / 3.f), u, 1.f);
  return u < 0.04f ? x * p : tanh_ex2(x);
}

// Scores in log2 units from raw dot products: scale, cap, distance bias.
struct ScoreMap {
  float k;      // dot -> x / softcap with a cap, dot -> log2 units without
  float cap2;   // softcap * log2 e; 0: no cap
  float slope2; // slopes[h] * log2 e; 0: no bias
  __device__ __forceinline__ float operator()(float dot, float dist) const {
    float y = dot * k;
    if (cap2 != 0.f) y = cap2 * tanhf(y);  // the 32-bit kernels: to the last bits
    return fmaf(-slope2, dist, y);
  }
};

__device__ __forceinline__ ScoreMap score_map(const RuleDesc& r, float scale, int h) {
  constexpr float kLog2e = 1.4426950408889634f;
  ScoreMap m;
  m.k = r.softcap > 0.f ? scale / r.softcap : scale * kLog2e;
  m.cap2 = r.softcap * kLog2e;
  m.slope2 = r.slopes ? r.slopes[h] * kLog2e : 0.f;
  return m;
}

}  // namespace fpx

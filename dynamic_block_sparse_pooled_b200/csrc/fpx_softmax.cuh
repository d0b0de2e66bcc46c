// fpx_softmax.cuh -- the softmax arithmetic of the tensor-core attention kernels: row maxima, the
// exponentials, and the score rule on a row of S in registers.
#pragma once

#include <cuda_runtime.h>
#include <math_constants.h>

#include "fpx_rule.cuh"
#include "fpx_sm100.cuh"

namespace fpx {
namespace sm100 {

constexpr float kRescaleLog2 = 8.0f;    // lazy rescale threshold (log2 units)

// Maximum of 64 fp32 values (3-input max, four independent chains).
__device__ __forceinline__ float row_max64(const uint32_t* r) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = __uint_as_float(r[k]);
#pragma unroll
  for (int j = 4; j < 60; j += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = max3f(m[k], __uint_as_float(r[j + k]), __uint_as_float(r[j + 4 + k]));
  return max3f(max3f(m[0], m[1], __uint_as_float(r[60])), max3f(m[2], m[3], __uint_as_float(r[61])),
               fmaxf(__uint_as_float(r[62]), __uint_as_float(r[63])));
}

// Minimum of 64 fp32 values.
__device__ __forceinline__ float row_min64(const uint32_t* r) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) m[k] = __uint_as_float(r[k]);
#pragma unroll
  for (int j = 4; j < 60; j += 8)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      m[k] = min3f(m[k], __uint_as_float(r[j + k]), __uint_as_float(r[j + 4 + k]));
  return min3f(min3f(m[0], m[1], __uint_as_float(r[60])), min3f(m[2], m[3], __uint_as_float(r[61])),
               fminf(__uint_as_float(r[62]), __uint_as_float(r[63])));
}

// One in kPolyEvery element pairs takes exp2 on the FMA pipe instead of the MUFU (0: none).  The
// MUFU issues four ex2 per cycle per SM sub-partition, so a 128-column row costs ~1000 cycles
// there; moving a quarter of the pairs to the FMA pipe was measured fastest (one in two or three
// saturates the FMA pipe instead).
#ifndef FPX_POLY_EVERY
#define FPX_POLY_EVERY 4
#endif
constexpr int kPolyEvery = FPX_POLY_EVERY;

// Columns [J0, J0 + N) of the S row in r become P, packed in place (bf16 pairs at r[J0 / 2 ..],
// or e4m3 quads at r[J0 / 4 ..]); returns their sum.
// kPoly: share the exponentials with the FMA pipe.  Under a score rule all of them stay on the MUFU:
// the rule's own arithmetic takes the FMA pipe, and rows with few keys that count (a steep distance
// bias) would show the polynomial's 7.5e-5 in their LSE.
template <bool kFp8, bool kPoly, int J0, int N>
__device__ __forceinline__ float softmax_part_to_p(uint32_t* r, float sl2, float neg_m) {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = J0; j < J0 + N; j += 2) {
    float x0, x1, p0, p1;
    ffma2(x0, x1, __uint_as_float(r[j]), __uint_as_float(r[j + 1]), sl2, sl2, neg_m, neg_m);
    constexpr int kEvery = kPolyEvery > 0 ? kPolyEvery : 1;
    if (kPoly && kPolyEvery > 0 && (j / 2) % kEvery == kEvery - 1) {
      exp2_poly2(p0, p1, x0, x1);
    } else {
      p0 = ex2_approx(x0);
      p1 = ex2_approx(x1);
    }
    fadd2(s[(j / 2) % 4 * 2], s[(j / 2) % 4 * 2 + 1], p0, p1);
    if (kFp8) {
      const uint32_t v = __nv_cvt_float2_to_fp8x2(make_float2(p0, p1), __NV_SATFINITE, __NV_E4M3);
      if ((j & 2) == 0) r[j / 4] = v;
      else r[j / 4] |= v << 16;
    } else {
      r[j / 2] = pack_bf16x2(p0, p1);
    }
  }
  return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// Columns [J0, J0 + N) of raw capped scores, all at most kTanhNear of the cap, become P: tanh as
// x (c0 + c1 x^2 + c2 x^4 + c3 x^6) (largest relative error 6.2e-7 for |x| <= 1/2, fitted by
// tanh_poly_fit.py), the maximum subtracted by the last multiply-add.  Four pairs at a time, stage by stage: eight
// independent values hide the latency of the chain, which one warp per SM sub-partition and tile
// otherwise waits for (8192 tokens, 32 heads: two pairs at a time 719 us, four 660, eight 659).
constexpr float kTanhNear = 0.5f;
constexpr float kNear0 = 9.999994636e-01f, kNear1 = -3.332631886e-01f,
                kNear2 = 1.319029629e-01f, kNear3 = -4.440220818e-02f;
struct NearTanh {
  float c[4];  // with the factor cap log2 e
  // The score of x = dot / cap, by the operations that capped_part_to_p forms its weight's exponent
  // with: the reference that the weights are taken against has to be one of their own scores, as any
  // other form of tanh is off by its error times the cap.
  __device__ __forceinline__ float operator()(float x) const {
    const float u = x * x;
    return x * fmaf(fmaf(fmaf(c[3], u, c[2]), u, c[1]), u, c[0]);
  }
};
template <bool kFp8, int J0, int N>
__device__ __forceinline__ float capped_part_to_p(uint32_t* r, float k, const NearTanh& th,
                                                  float neg_m) {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = J0; j < J0 + N; j += 8) {
    float t[8], u[8], p[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      fmul2(t[i], t[i + 1], __uint_as_float(r[j + i]), __uint_as_float(r[j + i + 1]), k, k);
#pragma unroll
    for (int i = 0; i < 8; i += 2) fmul2(u[i], u[i + 1], t[i], t[i + 1], t[i], t[i + 1]);
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      ffma2(p[i], p[i + 1], u[i], u[i + 1], th.c[3], th.c[3], th.c[2], th.c[2]);
#pragma unroll
    for (int n = 1; n >= 0; --n)
#pragma unroll
      for (int i = 0; i < 8; i += 2)
        ffma2(p[i], p[i + 1], p[i], p[i + 1], u[i], u[i + 1], th.c[n], th.c[n]);
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      ffma2(t[i], t[i + 1], t[i], t[i + 1], p[i], p[i + 1], neg_m, neg_m);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = ex2_approx(t[i]);
#pragma unroll
    for (int i = 0; i < 8; i += 2) fadd2(s[i], s[i + 1], p[i], p[i + 1]);
    if (kFp8) {
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        r[(j + i) / 4] =
            __nv_cvt_float2_to_fp8x2(make_float2(p[i], p[i + 1]), __NV_SATFINITE, __NV_E4M3) |
            __nv_cvt_float2_to_fp8x2(make_float2(p[i + 2], p[i + 3]), __NV_SATFINITE, __NV_E4M3)
                << 16;
    } else {
#pragma unroll
      for (int i = 0; i < 8; i += 2) r[(j + i) / 2] = pack_bf16x2(p[i], p[i + 1]);
    }
  }
  return ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
}

// Largest cap (log2 units) whose scores may all take tanh_ex2: 4e-7 of it is 2e-4, less than a
// twentieth of a bf16 weight's rounding.
constexpr float kEx2Cap = 512.f;

// 64 columns of a row of S, the first of them column j0 of its key block, under a score rule: cap,
// distance bias (rel = the row's position - the block's first key) and mask (columns [c_lo, c_hi] are
// seen; partial: some row of the warp does not see all of the block before (bit 0) or behind (bit 1)
// what it sees).  The result is in log2 units,
// unless the rule has neither cap nor bias: then raw.
template <bool kCap, bool kBias>
__device__ __forceinline__ void rule_half(uint32_t* x, int j0, const ScoreMap& map,
                                          const TanhPoly& poly, float rel, int c_lo, int c_hi,
                                          int partial) {
  constexpr unsigned kFull = 0xffffffffu;
  if (kCap) {
    // Capped scores mostly lie well within the cap, where tanh is a polynomial on the
    // FMA pipe; a warp with a score beyond that takes 2^x and a reciprocal on the MUFU.  That form's
    // error is absolute, 4e-7 of the cap: for all of the warp's scores where the cap is at most
    // kEx2Cap, for those beyond alone where it is larger, as a score far below its cap would not
    // keep its precision (per-score choice: 8192 tokens, cap 50, every warp with such a score, 1525 us
    // instead of 1360).
    // Only seen scores count, so that no result depends on an unseen one.
    float top[4] = {0.f, 0.f, 0.f, 0.f};
    if (partial & 1) {
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (j0 + j < c_lo) x[j] = 0u;
    }
    if (partial & 2) {
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (j0 + j > c_hi) x[j] = 0u;
    }
#pragma unroll
    for (int j = 0; j < 64; j += 2)
      top[j / 2 % 4] = absmax3f(top[j / 2 % 4], __uint_as_float(x[j]),
                                __uint_as_float(x[j + 1]));
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (__all_sync(kFull, most * fabsf(map.k) <= TanhPoly::kMost)) {
#pragma unroll
      for (int j = 0; j < 64; j += 2) {
        float x0 = __uint_as_float(x[j]), x1 = __uint_as_float(x[j + 1]);
        poly(x0, x1, map.k);
        x[j] = __float_as_uint(x0);
        x[j + 1] = __float_as_uint(x1);
      }
    } else if (map.cap2 <= kEx2Cap) {
#pragma unroll
      for (int j = 0; j < 64; ++j)
        x[j] = __float_as_uint(map.cap2 * tanh_ex2(__uint_as_float(x[j]) * map.k));
    } else {
#pragma unroll
      for (int j = 0; j < 64; j += 2) {
        float x0 = __uint_as_float(x[j]), x1 = __uint_as_float(x[j + 1]);
        const float t0 = x0 * map.k, t1 = x1 * map.k;
        poly(x0, x1, map.k);
        x[j] = __float_as_uint(fabsf(t0) <= TanhPoly::kMost ? x0 : map.cap2 * tanh_ex2(t0));
        x[j + 1] = __float_as_uint(fabsf(t1) <= TanhPoly::kMost ? x1 : map.cap2 * tanh_ex2(t1));
      }
    }
  }
  if (kBias) {
    // -slope |i - j| is linear in the column unless the block holds the row's diagonal
    const float kk = kCap ? 1.f : map.k;
    const bool before = rel >= 127.f;
    if (__all_sync(kFull, before || rel <= 0.f)) {
      const float b1 = before ? map.slope2 : -map.slope2;
      const float base = -b1 * rel;
#pragma unroll
      for (int j = 0; j < 64; j += 2) {
        float y0, y1;
        ffma2(y0, y1, __uint_as_float(x[j]), __uint_as_float(x[j + 1]), kk, kk,
              fmaf(b1, static_cast<float>(j0 + j), base),
              fmaf(b1, static_cast<float>(j0 + j + 1), base));
        x[j] = __float_as_uint(y0);
        x[j + 1] = __float_as_uint(y1);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 64; ++j)
        x[j] = __float_as_uint(fmaf(-map.slope2, fabsf(rel - static_cast<float>(j0 + j)),
                                    __uint_as_float(x[j]) * kk));
    }
  }
  if (partial & 1) {
#pragma unroll
    for (int j = 0; j < 64; ++j)
      if (j0 + j < c_lo) x[j] = __float_as_uint(-CUDART_INF_F);
  }
  if (partial & 2) {
#pragma unroll
    for (int j = 0; j < 64; ++j)
      if (j0 + j > c_hi) x[j] = __float_as_uint(-CUDART_INF_F);
  }
}

}  // namespace sm100
}  // namespace fpx

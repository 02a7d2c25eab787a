// Scores that are changed between the product q.k and the softmax, and masks beside the causal one:
//   x = cap tanh(scale q.k / cap)            (cap > 0),
//   x + slope_h (key - position)             (a bias that falls with the distance),
//   keys below visible_lens[s] are seen by every query of sequence s (a prefix read both ways).
// The passes work in units of log2: x log2(e).
#pragma once

#include "cb_common.cuh"
#include "cb_launch.h"

namespace cb {

// cap tanh(u) log2(e) from the raw product s, u = s scale / cap: with t = 2^(cap_in s),
// cap_in = 2 log2(e) scale / cap, tanh(u) = 1 - 2 / (1 + t).  Off by 2^-22 of the cap at most (two
// approximations of 2^-22, and the cancellation near 0, which is absolute as well): 2e-5 of a score at a
// cap of 50.  t = inf gives 1.
__device__ __forceinline__ float cap_score(float s, const ScoreArgs& sc) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(s * sc.cap_in)));
  return fmaf(-2.f * sc.cap_out, r, sc.cap_out);
}
// The same for two scores with |u| <= 0.6 each, without the two special-function instructions per
// score: tanh(u) / u is a polynomial in u^2, here the interpolation of degree 4 at Chebyshev's points of
// [0, 0.36], off by 4e-8 in tanh.  The host multiplies scale log2(e) and the powers of scale / cap into
// the coefficients (ScoreArgs::near), so it takes six instructions on pairs of the raw products s.  The chunk
// pass computes it for all scores and cap_score for those beyond its range, in tiles that have any.
// (8 chunks of 512 tokens on up to 4096 keys, 32 query, 8 KV heads of 128, the whole call: with slopes instead
// 204 us, capped at 50 237, at 2, where a quarter of the scores is beyond, 343; with one form for a warp's tile
// as a whole, by its largest product, 239 and 282, but then a row's bits depend on what stands beside it.  A
// shorter polynomial for smaller scores beside this one, degree 2 to 0.3 caps, made the pass 4 % faster where
// it applied and 15 % slower where it did not.)
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t cap_near(uint64_t s, const uint64_t (&k)[5]) {
  const uint64_t z = f2_mul(s, s);
  return f2_mul(s, f2_fma(f2_fma(f2_fma(f2_fma(k[4], z, k[3]), z, k[2]), z, k[1]), z, k[0]));
}
// The raw product s of a query at `pos` and key `key`, in units of log2.
__device__ __forceinline__ float change_score(float s, float scale_log2, float slope_log2, int key,
                                              int pos, const ScoreArgs& sc) {
  const float x = sc.cap_in > 0.f ? cap_score(s, sc) : s * scale_log2;
  return fmaf(slope_log2, (float)(key - pos), x);
}
// Head h's slope in units of log2 (0 without slopes).
__device__ __forceinline__ float slope_of(const ScoreArgs& sc, int h) {
  return sc.slopes != nullptr ? __ldg(sc.slopes + h) * 1.4426950408889634f : 0.f;
}

}  // namespace cb

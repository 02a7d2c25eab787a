// Scores that are changed between the product q.k and the softmax, and masks beside the causal one:
//   x = cap tanh(scale q.k / cap)            (cap > 0),
//   x + slope_h (key - position)             (a bias that falls with the distance),
//   keys below visible_lens[s] are seen by every query of sequence s (a prefix read both ways).
// The passes work in units of log2: x log2(e).
#pragma once

#include "cb_common.cuh"
#include "cb_launch.h"

namespace cb {

// Capped scores, to within 2^-20 of themselves whatever the cap's size: two forms, each where it is exact.
//
// (Where scale and cap are so far apart that the constants would leave fp32, s stands for the product times a
// power of two, ScoreArgs::near_in.)
//
// cap tanh(u) log2(e) from the raw product s, u = s scale / cap, |u| > 0.6: with t = 2^(cap_in s),
// cap_in = 2 log2(e) scale / cap, tanh(u) = 1 - 2 / (1 + t).  Two approximations of 2^-22 of 2 / (1 + t), which is
// 0.86 tanh(u) at most there (nearer to 0 the difference would cancel, down to an error of 2^-22 of the cap).
// t = inf gives 1.
__device__ __forceinline__ float cap_far(float s, const ScoreArgs& sc) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(s * sc.cap_in)));
  return fmaf(-2.f * sc.cap_out, r, sc.cap_out);
}
// The same where |u| <= 0.6, for two scores, without special functions: tanh(u) / u is a polynomial in u^2, here
// the interpolation of degree 4 at Chebyshev's points of [0, 0.36], off by 6e-8 of itself.  The host multiplies
// scale log2(e) and the powers of scale / cap into the coefficients (ScoreArgs::near), so it takes six
// instructions on pairs of the raw products s.  Tiles of a warp that have scores beyond its range take both forms
// for all scores.
// (8 chunks of 512 tokens on up to 4096 keys, 32 query, 8 KV heads of 128, bf16 cache, the whole call: with slopes
// instead 200 us, capped at 50 233, at 2, where a quarter of the scores is beyond, 303, with the scores beyond
// replaced in the unrolled registers instead of the small loop over TMEM 238 and 344.  With one form for a warp's
// tile as a whole, by its largest product, 240 and 283, but then a row's bits depend on what stands beside it.  A
// shorter polynomial for smaller scores beside this one, degree 2 to 0.3 caps, made the pass 4 % faster where it
// applied and 15 % slower where it did not.  Over the 8-bit cache, where the decode pass is bound by its
// instructions, 100 decodes of head_dim 64 take 73 us, capped at 50 82, at 2 91.)
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t cap_near(uint64_t s, const uint64_t (&k)[5]) {
  const uint64_t z = f2_mul(s, s);
  return f2_mul(s, f2_fma(f2_fma(f2_fma(f2_fma(k[4], z, k[3]), z, k[2]), z, k[1]), z, k[0]));
}
// A decode lane's N raw products become scores in units of log2: s[x] is of its first or second query head
// (x & 1), at one position, and of key 8 (x / 2) behind the first, which is `dist` from the position.  By all
// lanes of a warp.
template <int N>
__device__ __forceinline__ void change_scores(float* s, float scale_log2, const float (&slope)[2], int dist,
                                              const ScoreArgs& sc) {
  if (sc.cap_in > 0.f) {
    float raw[N], big = 0.f;
    uint64_t near[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) near[i] = f2_pack(sc.near[i], sc.near[i]);
#pragma unroll
    for (int x = 0; x < N; ++x) {
      raw[x] = s[x] * sc.near_in;
      big = fmaxf(big, fabsf(raw[x]));
    }
#pragma unroll
    for (int x = 0; x < N; x += 2) f2_unpack(cap_near(f2_pack(raw[x], raw[x + 1]), near), s[x], s[x + 1]);
    if (!__all_sync(0xffffffffu, big <= sc.near_max)) {
#pragma unroll
      for (int x = 0; x < N; ++x) {
        const float far = cap_far(raw[x], sc);
        if (!(fabsf(raw[x]) <= sc.near_max)) s[x] = far;
      }
    }
  } else {
#pragma unroll
    for (int x = 0; x < N; ++x) s[x] *= scale_log2;
  }
#pragma unroll
  for (int x = 0; x < N; ++x) s[x] = fmaf(slope[x & 1], (float)(dist + 8 * (x >> 1)), s[x]);
}
// Head h's slope in units of log2 (0 without slopes).
__device__ __forceinline__ float slope_of(const ScoreArgs& sc, int h) {
  return sc.slopes != nullptr ? __ldg(sc.slopes + h) * 1.4426950408889634f : 0.f;
}

}  // namespace cb

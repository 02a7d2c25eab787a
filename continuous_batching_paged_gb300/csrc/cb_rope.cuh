// Device code of the rotary KV-append: one token's query and key heads rotated by its position's
// angles, the queries to q_out, the keys (and the values as they are) to their cache slots.
//
// A head's first rot_dim elements are rot_dim / 2 pairs (a, b): elements (i, i + rot_dim / 2), or
// (2i, 2i + 1) when interleaved.  With (c, s) = (cos, sin) of pair i at the token's position,
//   a' = a c - b s,   b' = b c + a s,
// in fp32 on the bf16 values, rounded once to bf16 (the cache's and the attention's type).  Each
// product and sum is rounded by itself: the result does not depend on contraction.
//
// Bound by bytes (3 operations per 2-byte element).  The work of a token is cut into "units" of
// two 16-byte chunks that hold eight whole pairs, D / 16 to a head, so 32 lanes cover 4 (D = 128)
// or 8 (D = 64) heads at once and a lane keeps the same unit, and so the same eight (c, s), in
// registers for every head it works on.
#pragma once

#include "cb_append.cuh"

namespace cb {

__device__ __forceinline__ void unpack8(const uint4& v, float* x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// The pair (a, b) turned by (c, s).
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float a1 = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = a1;
}

// A unit's two chunks turned by its eight (c, s): chunk against chunk, or neighbours inside each.
__device__ __forceinline__ void turn_unit(uint4& va, uint4& vb, const float* c, const float* s,
                                          bool interleaved) {
  float a[8], b[8];
  unpack8(va, a);
  unpack8(vb, b);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn(a[2 * i], a[2 * i + 1], c[i], s[i]);
      turn(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn(a[i], b[i], c[i], s[i]);
  }
  va = pack8(a);
  vb = pack8(b);
}

// Items first_warp, first_warp + nwarps, ... of the r.parts x T items (token, part): part p of a
// token does its head groups p, p + parts, ... (a head group: the 32 / (D / 16) heads that a warp
// covers at once; the heads are the queries', then the keys', then the values').  The loads of the
// first kUnroll groups are issued before the token's slot is looked up, so that the chain of
// metadata loads (sequence, length, block) runs under them.
template <int kUnroll>
__device__ __forceinline__ void rope_tokens(const RopeArgs& r, long long first_warp,
                                            long long nwarps) {
  const AppendArgs& a = r.ap;
  const int lane = threadIdx.x & 31;
  const int units = a.D >> 4, per_warp = 32 / units;
  const int unit = lane & (units - 1), sub = lane / units;
  const int n_q = r.q != nullptr ? r.Hq : 0;
  const int heads = n_q + 2 * a.Hkv;
  const int groups = (heads + per_warp - 1) / per_warp;
  const int rot_units = r.rot_dim >> 4;
  const bool rotates = unit < rot_units;
  // the unit's chunks within a head
  const bool across = rotates && !r.interleaved;
  const int ca = across ? unit : 2 * unit, cb_ = across ? unit + rot_units : 2 * unit + 1;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(r.q);
  const __nv_bfloat16* kn = static_cast<const __nv_bfloat16*>(a.k_new);
  const __nv_bfloat16* vn = static_cast<const __nv_bfloat16*>(a.v_new);
  __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(r.q_out);
  __nv_bfloat16* kp = static_cast<__nv_bfloat16*>(a.k_pages);
  __nv_bfloat16* vp = static_cast<__nv_bfloat16*>(a.v_pages);
  const long long n_items = (long long)a.T * r.parts;
  for (long long item = first_warp; item < n_items; item += nwarps) {
    const int t = (int)(item / r.parts), part = (int)(item - (long long)t * r.parts);
    long long slot = 0;
    int pos = 0;
    float c[8], s[8];
    for (int g0 = part; g0 < groups; g0 += kUnroll * r.parts) {
      uint4 x[kUnroll][2];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int h = (g0 + i * r.parts) * per_warp + sub;
        if (h < heads) {
          const __nv_bfloat16* src = h < n_q ? q + t * r.q_stride + h * a.D
                                     : h < n_q + a.Hkv
                                         ? kn + t * r.k_stride + (h - n_q) * a.D
                                         : vn + t * r.v_stride + (h - n_q - a.Hkv) * a.D;
          x[i][0] = reinterpret_cast<const uint4*>(src)[ca];
          x[i][1] = reinterpret_cast<const uint4*>(src)[cb_];
        }
      }
      if (g0 == part) {
        slot = token_slot<true>(a, t, lane, pos);
        if (slot >= 0 && pos >= r.max_positions) {
          if (lane == 0) report(a.err, kErrOutOfRange);
          slot = -1;
        }
        if (slot < 0) break;
        if (rotates) {
          const float4* row = reinterpret_cast<const float4*>(r.cos_sin + (long long)pos * r.rot_dim) +
                              2 * unit;
          const float4 c0 = __ldg(row), c1 = __ldg(row + 1);
          const float4 s0 = __ldg(row + 2 * rot_units), s1 = __ldg(row + 2 * rot_units + 1);
          c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
          c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
          s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
          s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
        }
      }
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int h = (g0 + i * r.parts) * per_warp + sub;
        if (h < heads) {
          if (rotates && h < n_q + a.Hkv) turn_unit(x[i][0], x[i][1], c, s, r.interleaved != 0);
          __nv_bfloat16* dst =
              h < n_q ? qo + ((long long)t * r.Hq + h) * a.D
              : h < n_q + a.Hkv ? kp + (slot * a.Hkv + (h - n_q)) * a.D
                                : vp + (slot * a.Hkv + (h - n_q - a.Hkv)) * a.D;
          reinterpret_cast<uint4*>(dst)[ca] = x[i][0];
          reinterpret_cast<uint4*>(dst)[cb_] = x[i][1];
        }
      }
    }
  }
}

}  // namespace cb

// Device code of the quantised cache: rows of keys and values as e4m3 codes with one power-of-two
// scale per (token, KV head), written (quant_tokens) and read back (gather_rows).
//
// A row x of D values is stored as codes c and an exponent e:
//   e = the smallest integer in [-32, 31] with max |x| <= 448 * 2^e,   c = e4m3(x * 2^-e),
// 448 being the largest e4m3 value.  Scaling by a power of two is exact, so each value is rounded once
// (to 4 significant bits: off by 2^-4 of its own size at most, or by 2^-10 * 2^e where that is more),
// and c * 2^e is exact in bf16.  The type's own exponent covers what the scale leaves out, so a finer
// scale than a power of two would gain nothing but the last bit of the range.  Values above 448 * 2^31
// are clamped.  A row with a value that is not finite is stored as NaN: its exponent byte is 255, and all
// its values read back as NaN.  (Single NaN codes would cost the chunk pass a test of every code.)
#pragma once

#include "cb_rope.cuh"

namespace cb {

constexpr int kQuantLow = -32, kQuantHigh = 31;  // exponents of the scales
constexpr int kQuantBias = 127;                  // a stored exponent byte is e + 127
constexpr int kQuantNan = 255;                   // that of a row that is NaN

// Four values to four e4m3 codes, the first in the lowest byte (round to nearest even, clamped; NaN
// stays NaN).
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Two codes (the low 16 bits of x, and the high ones) to two fp16 values each: exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// The biased exponent of a row's scale, from the largest finite |x| of the row.
__device__ __forceinline__ int quant_exponent(float top) {
  const uint32_t b = __float_as_uint(top);  // 448 = 1.75 * 2^8
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kQuantLow), kQuantHigh) + kQuantBias;
}

// Items first_warp, first_warp + nwarps, ... of the r.parts x T items (token, part), laid out like
// rope_tokens': part p of a token does its head groups p, p + parts, ..., a lane one unit of two
// 16-byte chunks of a head, whose D / 16 lanes find the row's largest value together.  Rotated keys are
// quantised from their fp32 values, without a rounding to bf16 between.
template <int kUnroll>
__device__ __forceinline__ void quant_tokens(const QuantAppendArgs& x, long long first_warp,
                                             long long nwarps) {
  const RopeArgs& r = x.r;
  const AppendArgs& a = r.ap;
  const int lane = threadIdx.x & 31;
  const int units = a.D >> 4, per_warp = 32 / units;
  const int unit = lane & (units - 1), sub = lane / units;
  const int n_q = r.q != nullptr ? r.Hq : 0;
  const int heads = n_q + 2 * a.Hkv;
  const int groups = (heads + per_warp - 1) / per_warp;
  const int rot_units = r.rot_dim >> 4;
  const bool rotates = unit < rot_units;
  const bool across = rotates && !r.interleaved;
  const int ca = across ? unit : 2 * unit, cb_ = across ? unit + rot_units : 2 * unit + 1;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(r.q);
  const __nv_bfloat16* kn = static_cast<const __nv_bfloat16*>(a.k_new);
  const __nv_bfloat16* vn = static_cast<const __nv_bfloat16*>(a.v_new);
  __nv_bfloat16* qo = static_cast<__nv_bfloat16*>(r.q_out);
  uint8_t* kp = static_cast<uint8_t*>(a.k_pages);
  uint8_t* vp = static_cast<uint8_t*>(a.v_pages);
  const long long n_items = (long long)a.T * r.parts;
  for (long long item = first_warp; item < n_items; item += nwarps) {
    const int t = (int)(item / r.parts), part = (int)(item - (long long)t * r.parts);
    long long slot = 0;
    int pos = 0;
    float c[8], s[8];
    for (int g0 = part; g0 < groups; g0 += kUnroll * r.parts) {
      uint4 v[kUnroll][2];
#pragma unroll
      for (int i = 0; i < kUnroll; ++i) {
        const int h = (g0 + i * r.parts) * per_warp + sub;
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        if (h < heads) {
          const __nv_bfloat16* src = h < n_q ? q + t * r.q_stride + h * a.D
                                     : h < n_q + a.Hkv
                                         ? kn + t * r.k_stride + (h - n_q) * a.D
                                         : vn + t * r.v_stride + (h - n_q - a.Hkv) * a.D;
          v[i][0] = reinterpret_cast<const uint4*>(src)[ca];
          v[i][1] = reinterpret_cast<const uint4*>(src)[cb_];
        }
      }
      if (g0 == part) {
        slot = token_slot<true>(a, t, lane, pos);
        if (slot >= 0 && rot_units > 0 && pos >= r.max_positions) {
          if (lane == 0) report(a.err, kErrOutOfRange);
          slot = -1;
        }
        if (slot < 0) break;
        if (rotates) {
          const float4* row =
              reinterpret_cast<const float4*>(r.cos_sin + (long long)pos * r.rot_dim) + 2 * unit;
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
        const int g = g0 + i * r.parts;  // (the same in the whole warp)
        if (g >= groups) break;
        const int h = g * per_warp + sub;
        if (h < n_q) {
          if (rotates) turn_unit(v[i][0], v[i][1], c, s, r.interleaved != 0);
          uint4* dst = reinterpret_cast<uint4*>(qo + ((long long)t * r.Hq + h) * a.D);
          dst[ca] = v[i][0];
          dst[cb_] = v[i][1];
        }
        if ((g + 1) * per_warp <= n_q) continue;  // (queries only)
        const bool key = h < n_q + a.Hkv;
        float y[16], top = 0.f;
        bool nan = false;
        unpack8(v[i][0], y);
        unpack8(v[i][1], y + 8);
        if (rotates && key) turn_unit(y, y + 8, c, s, r.interleaved != 0);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          nan = nan || !(fabsf(y[j]) < INFINITY);
          top = fmaxf(top, fabsf(y[j]));
        }
        // the head's lanes together (what is not finite as the largest value)
        if (nan) top = INFINITY;
        for (int o = 1; o < units; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        nan = top == INFINITY;
        if (h >= n_q && h < heads) {
          const long long row = slot * a.Hkv + (h - n_q - (key ? 0 : a.Hkv));
          const int e = nan ? kQuantNan : quant_exponent(top);
          const float inv = nan ? __int_as_float(0x7fffffff) : __int_as_float((2 * kQuantBias - e) << 23);
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] *= inv;
          const uint2 lo = make_uint2(pack_e4m3x4(y[0], y[1], y[2], y[3]),
                                      pack_e4m3x4(y[4], y[5], y[6], y[7]));
          const uint2 hi = make_uint2(pack_e4m3x4(y[8], y[9], y[10], y[11]),
                                      pack_e4m3x4(y[12], y[13], y[14], y[15]));
          uint8_t* dst = (key ? kp : vp) + row * a.D;
          if (across) {
            reinterpret_cast<uint2*>(dst)[ca] = lo;
            reinterpret_cast<uint2*>(dst)[cb_] = hi;
          } else {
            reinterpret_cast<uint4*>(dst)[unit] = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
          if (unit == 0) x.scales[2 * row + (key ? 0 : 1)] = (uint8_t)e;
        }
      }
    }
  }
}

// Eight codes times 2^(e - 127) as bf16 (exact; NaN for kQuantNan).
__device__ __forceinline__ uint4 codes_to_bf16(uint2 codes, int e) {
  const float f = e == kQuantNan ? __int_as_float(0x7fffffff) : __int_as_float(e << 23);
  uint32_t h[4];
  e4m3x4_to_f16(codes.x, h[0], h[1]);
  e4m3x4_to_f16(codes.y, h[2], h[3]);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    o[i] = pack_bf16x2(p.x * f, p.y * f);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Output rows g.rows * w .. of warp w.  Each lane finds the cache row of one of them (a binary search
// of its own, so a warp's rows cost one chain of metadata loads together); then the warp takes the rows
// one after the other, 8 codes of a lane becoming 16 bytes, so that loads and stores are both whole
// lines.  Bound by bytes: (2 D + 2) Hkv read and 4 D Hkv written per row; 95859 rows of 8 heads of 128
// take 89 us, 6.0 TB/s.  (8 pieces in flight per lane instead of 4 gain nothing there and cost small
// ranges: 10690 rows of 5 heads of 64 12.9 and 17 us.)
template <int kUnroll>
__device__ __forceinline__ void gather_rows(const GatherArgs& g, long long warp) {
  const int lane = threadIdx.x & 31;
  const int t_end = min(g.T, __ldg(g.cu_seqlens_k + g.S));
  const long long t0 = warp * g.rows;
  long long slot = -1;
  if (lane < g.rows && t0 + lane < t_end) {
    const int t = (int)(t0 + lane);
    int lo = 0, hi = g.S;  // the last s with cu[s] <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(g.cu_seqlens_k + mid) <= t) lo = mid; else hi = mid - 1;
    }
    bool ok = lo < g.S;
    if (ok) {
      const int c0 = __ldg(g.cu_seqlens_k + lo), c1 = __ldg(g.cu_seqlens_k + lo + 1);
      const long long start = g.key_starts != nullptr ? __ldg(g.key_starts + lo) : 0;
      const long long pos = start + (t - c0);
      const long long lb = pos / g.bs;
      ok = c0 >= 0 && t >= c0 && t < c1 && start >= 0 && lb < g.max_blocks;
      if (ok) {
        const int blk = __ldg(g.block_table + (size_t)lo * g.max_blocks + lb);
        ok = blk >= 0 && blk < g.P;
        if (ok) slot = (long long)blk * g.bs + (pos - lb * g.bs);
      }
    }
    if (!ok) report(g.err, kErrOutOfRange);
  }
  const int per_row = g.Hkv * g.D / 8, shift = g.D == 128 ? 4 : 3;  // 8-value pieces of a row, of a head
  const int n = (int)max(0ll, min((long long)g.rows, t_end - t0));
  const int pieces = n * per_row;
  for (int base = 0; base < pieces; base += 32 * kUnroll) {
    uint2 k[kUnroll], v[kUnroll];
    unsigned short sc[kUnroll];
    int at[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int p = base + 32 * i + lane;
      const int row = p / per_row, piece = p - row * per_row;
      const long long from = __shfl_sync(0xffffffffu, slot, row & 31);
      at[i] = p < pieces && from >= 0 ? p : -1;
      if (at[i] >= 0) {
        const long long src = from * per_row + piece;
        k[i] = __ldg(reinterpret_cast<const uint2*>(g.k_pages) + src);
        v[i] = __ldg(reinterpret_cast<const uint2*>(g.v_pages) + src);
        sc[i] = __ldg(reinterpret_cast<const unsigned short*>(g.scales) + from * g.Hkv + (piece >> shift));
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (at[i] >= 0) {
        const long long dst = t0 * per_row + at[i];
        static_cast<uint4*>(g.k_out)[dst] = codes_to_bf16(k[i], sc[i] & 255);
        static_cast<uint4*>(g.v_out)[dst] = codes_to_bf16(v[i], sc[i] >> 8);
      }
    }
  }
}

}  // namespace cb

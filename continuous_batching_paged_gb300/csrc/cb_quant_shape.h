// How the decode pass over the quantised cache cuts its tiles, from the shape alone.
#pragma once

#include "cb_launch.h"

namespace cb {

constexpr int kQTileKeys = 32;  // keys per warp and tile

// Warps that share a KV head when a CTA has HB of them and QS warps per head's group of 8 query heads: a
// power of two, QS * HB * this <= 8.
inline int quant_slices(int HB, int QS) {
  const int most = 8 / QS / HB;
  return most >= 8 ? 8 : most >= 4 ? 4 : most >= 2 ? 2 : 1;
}

inline QuantArgs quant_shape(int bs, int Hkv, int G, int D) {
  const int QS = G > 8 ? 2 : 1, HB = Hkv < 8 / QS ? Hkv : 8 / QS;
  QuantArgs q = {};
  q.KB = 1;
  while (q.KB < kQTileKeys && bs % (2 * q.KB) == 0) q.KB *= 2;  // rows of a page that one box holds
  // A box lands on a multiple of 128 bytes.  Where it is not one itself (single rows of 64 bytes of an
  // odd number of heads), the gaps leave room for the shortest tile only.
  int slices = quant_slices(HB, QS);
  if (q.KB * HB * D % 128 != 0) slices = 1;
  q.tile_log2 = 5;
  while (1 << (q.tile_log2 - 5) < slices) ++q.tile_log2;
  // Scales are copied in pieces that stay inside a box's rows: where the CTA has all heads, consecutive
  // keys', in one bulk copy if they are a multiple of 16 bytes; else one key's.
  const int run = 2 * HB * (Hkv == HB ? q.KB : 1);
  q.copy = run % 16 == 0 ? (Hkv == HB ? 0 : 16) : run % 8 == 0 ? 8 : run % 4 == 0 ? 4 : 2;
  return q;
}

}  // namespace cb

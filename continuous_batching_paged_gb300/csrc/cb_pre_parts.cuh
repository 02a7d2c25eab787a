// Index arithmetic of the shared prefixes' work (PreGroup): which steps of which chains a CTA does,
// and, for the planner and the merge, the same read the other way.
#pragma once

#include "cb_common.cuh"

namespace cb {

// Groups of KV heads that the decode CTAs are divided into (8 KV heads, or 4 with more than 8 query
// heads each).
__device__ __forceinline__ int pre_head_groups(int Hkv, int G) {
  const int heads = G > 8 ? kMaxDecodeHeadsPerCta / 2 : kMaxDecodeHeadsPerCta;
  return (Hkv + heads - 1) / heads;
}
// Decode CTAs without work when n of `grid` per head group work, and the index among them of CTA bx
// of head group hg (-1 if it has work): see decode_cta_index.
__device__ __forceinline__ int pre_idle_count(int head_groups, int n, int grid) {
  return head_groups * (grid - n);
}
__device__ __forceinline__ int pre_idle_index(int bx, int hg, int n, int grid) {
  if (decode_cta_index(bx, n, grid) >= 0) return -1;
  const bool pairs = ((n | grid) & 1) == 0;
  const int units = pairs ? grid / 2 : grid, wanted = pairs ? n / 2 : n;
  const int u = pairs ? bx >> 1 : bx;  // (unit 0 always works)
  const int rank = u - ((u - 1) * wanted / units + 1);
  return hg * (grid - n) + (pairs ? 2 * rank + (bx & 1) : rank);
}

// Shape of a group's chains.
struct PreShape {
  int nt;         // K/V tiles
  int full;       // units with two tiles of rows (the units before the last, at least)
  int units;      // units in all
  long long per;  // cost of all units under one KV head (kPreMaxCost at most, once planned)
};
__device__ __forceinline__ PreShape pre_shape(int n_tok, int nt, int G) {
  PreShape s;
  const int per_tile = pre_tile_tokens(G);
  const int tiles = (n_tok + per_tile - 1) / per_tile;
  s.nt = nt;
  s.full = tiles >> 1;
  s.units = (tiles + 1) >> 1;
  s.per = (long long)nt * (kPreCost2 * s.full + kPreCost1 * (tiles & 1));
  return s;
}
// K/V tiles that keys first .. keys - 1 lie in.
__device__ __forceinline__ int pre_tiles(int first, int keys) {
  return (keys + kChunkKeys - 1) / kChunkKeys - first / kChunkKeys;
}

// CTA c of N does the cost range [pre_bound(W, c, N), pre_bound(W, c + 1, N)) of the W units.
__device__ __forceinline__ long long pre_bound(long long W, int c, int N) { return W * c / N; }

// First step of a chain (start cs, cost w per step, nt steps) at or behind cost position b: a step
// belongs to the range that its start lies in.
__device__ __forceinline__ int pre_step(long long cs, int w, int nt, long long b) {
  if (b <= cs) return 0;
  if (b - cs >= (long long)w * nt) return nt;
  return ((int)(b - cs) + w - 1) / w;
}

// Part of a chain that one CTA does: K/V tiles [j0, j1) of `seq` under KV head kvh, as far as keys
// first .. keys - 1 lie in them, for `two` tiles of rows (or one): ntok[] query tokens from token list
// entry tok0 on, the first of them token `at` of the group (see PreGroup for ctx and second).
struct PreSeg {
  int kvh, seq, first, keys, ctx, second, j0, j1, tok0, at;
  int ntok[2];
  bool two;
  bool once;  // the group has this unit alone: its keys are read once per KV head
  bool cut;   // not the chain's first part
};

// Walks the parts of one CTA's range, in order.
struct PreWalk {
  const PreGroup* groups;
  int n_groups, gi, G, head_cost;
  long long b0, b1, pos;

  // W: cost per KV head, of Hkv heads.
  __device__ __forceinline__ PreWalk(const PreGroup* list, int n, int G_, int Hkv, int W, int c, int N)
      : groups(list), n_groups(n), gi(-1), G(G_), head_cost(W),
        b0(pre_bound((long long)W * Hkv, c, N)), b1(pre_bound((long long)W * Hkv, c + 1, N)), pos(b0) {}

  __device__ __forceinline__ bool next(PreSeg& s) {
    while (pos < b1) {
      const int kvh = (int)(pos / head_cost);
      const long long head0 = (long long)kvh * head_cost;
      const int rel = (int)(pos - head0);
      if (gi < 0) {  // the range's first group: the last one with cost0 <= rel
        int hi = n_groups - 1;
        gi = 0;
        while (gi < hi) {
          const int mid = (gi + hi + 1) >> 1;
          if (groups[mid].cost0 <= rel) gi = mid; else hi = mid - 1;
        }
      } else if (rel == 0) {
        gi = 0;
      } else if (gi + 1 < n_groups && groups[gi + 1].cost0 <= rel) {
        ++gi;
      }
      const PreGroup g = groups[gi];
      const int tile0 = g.first / kChunkKeys;
      const PreShape sh = pre_shape(g.n_tok, pre_tiles(g.first, g.keys), G);
      const int u = (rel - g.cost0) / (kPreCost2 * sh.nt);  // (a cheaper last unit: same index)
      const int w = u < sh.full ? kPreCost2 : kPreCost1;
      const long long cs = head0 + g.cost0 + u * kPreCost2 * sh.nt;
      pos = cs + w * sh.nt;
      const int r0 = pre_step(cs, w, sh.nt, b0), r1 = pre_step(cs, w, sh.nt, b1);
      if (r0 >= r1) continue;
      const int per_tile = pre_tile_tokens(G);
      s.j0 = tile0 + r0;
      s.j1 = tile0 + r1;
      s.cut = r0 > 0;
      s.at = u * 2 * per_tile;
      s.kvh = kvh;
      s.seq = g.seq;
      s.first = g.first;
      s.keys = g.keys;
      s.ctx = g.ctx;
      s.second = g.second;
      s.tok0 = g.tok0 + s.at;
      s.ntok[0] = min(per_tile, g.n_tok - s.at);
      s.ntok[1] = max(0, min(per_tile, g.n_tok - s.at - per_tile));
      s.two = s.ntok[1] > 0;
      s.once = sh.units == 1;
      return true;
    }
    return false;
  }
};

}  // namespace cb

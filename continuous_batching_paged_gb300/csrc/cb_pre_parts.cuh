// Index arithmetic of the shared prefixes' work (PreGroup): which steps of which chains a CTA does,
// and, for the planner and the merge, the same read the other way.
#pragma once

#include "cb_common.cuh"

namespace cb {

// Shape of a group's chains.
struct PreShape {
  int nt;         // K/V tiles of the prefix
  int full;       // units with two tiles of rows (the units before the last, at least)
  int units;      // units in all
  long long per;  // cost of all units under one KV head
};
__device__ __forceinline__ PreShape pre_shape(int n_tok, int keys, int G) {
  PreShape s;
  const int per_tile = pre_tile_tokens(G);
  const int tiles = (n_tok + per_tile - 1) / per_tile;
  s.nt = (keys + kChunkKeys - 1) / kChunkKeys;
  s.full = tiles >> 1;
  s.units = (tiles + 1) >> 1;
  s.per = (long long)s.nt * (kPreCost2 * s.full + kPreCost1 * (tiles & 1));
  return s;
}
__device__ __forceinline__ long long pre_cost_per_head(int n_tok, int keys, int G) {
  return pre_shape(n_tok, keys, G).per;
}

// CTA c of N does the cost range [pre_bound(W, c, N), pre_bound(W, c + 1, N)) of the W units.
__device__ __forceinline__ long long pre_bound(long long W, int c, int N) { return W * c / N; }

// First step of a chain (start cs, cost w per step, nt steps) at or behind cost position b: a step
// belongs to the range that its start lies in.
__device__ __forceinline__ int pre_step(long long cs, int w, int nt, long long b) {
  if (b <= cs) return 0;
  const long long j = (b - cs + w - 1) / w;
  return j < nt ? (int)j : nt;
}

// Part of a chain that one CTA does: K/V tiles [j0, j1) of the prefix of `seq` (keys long) under KV
// head kvh, for `two` tiles of rows (or one): ntok[] query tokens from token list entry tok0 on.
struct PreSeg {
  int kvh, seq, keys, j0, j1, tok0;
  int ntok[2];
  bool two;
};

// Walks the parts of one CTA's range, in order.
struct PreWalk {
  const PreGroup* groups;
  int n_groups, gi, G;
  long long b0, b1, pos;

  __device__ __forceinline__ PreWalk(const PreGroup* list, int n, int G_, long long W, int c, int N)
      : groups(list), n_groups(n), gi(0), G(G_), b0(pre_bound(W, c, N)), b1(pre_bound(W, c + 1, N)),
        pos(b0) {
    int hi = n - 1;  // largest index with cost0 <= b0
    while (gi < hi) {
      const int mid = (gi + hi + 1) >> 1;
      if (groups[mid].cost0 <= b0) gi = mid; else hi = mid - 1;
    }
  }

  __device__ __forceinline__ bool next(PreSeg& s) {
    while (pos < b1) {
      while (gi + 1 < n_groups && groups[gi + 1].cost0 <= pos) ++gi;
      const PreGroup g = groups[gi];
      const PreShape sh = pre_shape(g.n_tok, g.keys, G);
      const long long rel = pos - g.cost0;
      const int kvh = (int)(rel / sh.per);
      const long long unit_cost = (long long)kPreCost2 * sh.nt;
      const long long in_head = rel - kvh * sh.per;
      const int u = (int)(in_head / unit_cost);  // (the last unit may be a cheaper one: same index)
      const int w = u < sh.full ? kPreCost2 : kPreCost1;
      const long long cs = g.cost0 + kvh * sh.per + u * unit_cost;
      pos = cs + (long long)w * sh.nt;
      s.j0 = pre_step(cs, w, sh.nt, b0);
      s.j1 = pre_step(cs, w, sh.nt, b1);
      if (s.j0 >= s.j1) continue;
      const int per_tile = pre_tile_tokens(G), first = u * 2 * per_tile;
      s.kvh = kvh;
      s.seq = g.seq;
      s.keys = g.keys;
      s.tok0 = g.tok0 + first;
      s.ntok[0] = min(per_tile, g.n_tok - first);
      s.ntok[1] = max(0, min(per_tile, g.n_tok - first - per_tile));
      s.two = s.ntok[1] > 0;
      return true;
    }
    return false;
  }
};

}  // namespace cb

// Batch planner of the attention pass (device code; run by one CTA).
#pragma once

#include "cb_common.cuh"
#include "cb_launch.h"
#include "cb_pre_parts.cuh"

namespace cb {

// ------------------------------------------------------------------------------------------
// Planner: one CTA classifies every sequence (q_len == 1 -> decode, q_len > 1 -> chunk),
// validates its lengths, and writes the compacted lists and prefix sums the attention passes
// read.  Nothing returns to the host.

constexpr int kPlanThreads = 1024;
// With shared prefixes the planner has more to compute per sequence and its time is instructions: a
// batch of one round (a sequence per thread) takes 5 us with kPrePlanThreads = 256 threads and 8 us
// with 1024, whose idle warps run through every step too.
template <bool kPre>
constexpr int plan_threads() { return kPre ? kPrePlanThreads : kPlanThreads; }

// Exclusive block-wide scan of four counters at once (NT threads); returns the block totals in tot[].
template <int NT>
__device__ __forceinline__ void block_scan4(int v[4], int ex[4], int tot[4], int (*sw)[4]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    int x = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    inc[k] = x;
  }
  if (lane == 31) {
#pragma unroll
    for (int k = 0; k < 4; ++k) sw[warp][k] = inc[k];
  }
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      int x = NT == 1024 || lane < NT / 32 ? sw[lane][k] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      sw[lane][k] = x;  // inclusive over warps
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    ex[k] = inc[k] - v[k] + (warp > 0 ? sw[warp - 1][k] : 0);
    tot[k] = sw[31][k];
  }
  __syncthreads();
}

// Decode CTA count for a batch whose chunk pass runs beside the decode pass.  Model, fitted to
// GB300 measurements of these kernels: decode on N SMs streams its bytes at
// BW(N) = ((0.11 N)^-3 + 6.8^-3)^(-1/3) TB/s (linear in N until HBM saturates), taking td; the
// chunk pass runs at ~6.4 TFLOP/s per SM on the other M SMs meanwhile and on every SM
// afterwards.  Chunk CTAs claim whole items (one query tile of one or two heads against its
// whole key range), so the chunk pass ends on item boundaries: if its work W fits in M SMs
// before td it ends near W/M (plus a short longest-first tail); if not, the items still
// unclaimed when decode ends each take a full item time on the newly free SMs, so the step is
// td + (W - M td)/SMs + about half an item.  The choice is the largest N within 1% of the
// modelled minimum, so that the decode pass keeps its bandwidth where the curve is flat --
// unless the minimum lies where the chunk pass is the longer one: there the model is flat in N
// (decode SM time is about constant while it is not bandwidth-bound) and the measured step
// is shortest with few decode CTAs that still finish early (chunk-heavy batch: N = 24..40
// 0.307 ms, N = 56 0.314 ms), so the choice is the smallest N within 1% whose decode pass
// takes at most a quarter of the step.  Without chunk work all CTAs decode.  Called by one
// full warp; candidates
// N = 4, 8, ... are spread over the lanes, in fp32 (the fp64 rate of this part is far too low
// for even this much arithmetic on one thread).
__device__ __forceinline__ int choose_decode_ctas(float dec_bytes, float chunk_flops, int chunk_items,
                                  int max_ctas, long long tiles) {
  const int lane = threadIdx.x & 31;
  if (tiles <= 0) return 1;
  const int cap = (int)(tiles < max_ctas ? tiles : max_ctas);
  if (chunk_flops <= 0.f || chunk_items <= 0) return cap;
  const float w_us = chunk_flops * (1.f / 6.4e6f);  // chunk work in SM-microseconds
  const float item_us = w_us / (float)chunk_items;
  const float b_mb = dec_bytes * 1e-6f;             // decode bytes / 1e6: MB / (TB/s) = us
  const int n_cand = (cap + 3) / 4;
  float t[4], td[4];
  bool chunk_bound[4];
  int n[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = lane + 32 * k;
    n[k] = 4 * (i + 1) < cap ? 4 * (i + 1) : cap;
    t[k] = 3.4e38f;
    td[k] = 0.f;
    chunk_bound[k] = false;
    if (i < n_cand) {
      const float lin = 0.11f * n[k], sat = 6.8f;
      const float bw = rcbrtf(1.f / (lin * lin * lin) + 1.f / (sat * sat * sat));
      td[k] = b_mb / bw;
      const int m = max_ctas - n[k];
      const float rest = w_us - (float)m * td[k];  // chunk work not done when decode ends
      chunk_bound[k] = rest > 0.f;
      t[k] = rest <= 0.f ? fmaxf(td[k], w_us / (float)m + 0.15f * item_us)
                         : td[k] + rest / (float)max_ctas + 0.5f * item_us;
    }
  }
  float t_min = fminf(fminf(t[0], t[1]), fminf(t[2], t[3]));
  for (int o = 16; o > 0; o >>= 1) t_min = fminf(t_min, __shfl_xor_sync(0xffffffffu, t_min, o));
  bool min_chunk_bound = false;
#pragma unroll
  for (int k = 0; k < 4; ++k) min_chunk_bound |= (t[k] == t_min && chunk_bound[k]);
  min_chunk_bound = __any_sync(0xffffffffu, min_chunk_bound);
  if (min_chunk_bound) {
    int small = cap + 1;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (t[k] <= 1.01f * t_min && td[k] <= 0.25f * t[k]) small = small < n[k] ? small : n[k];
    for (int o = 16; o > 0; o >>= 1) small = min(small, __shfl_xor_sync(0xffffffffu, small, o));
    if (small <= cap) return small;
  }
  int best = 1;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (t[k] <= 1.01f * t_min) best = best > n[k] ? best : n[k];
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  return best;
}

// Histogram bin of chunk unit g (global index in chunk-sequence order): units that stream
// more K/V tiles get lower bins, so an ascending walk over the bins is longest first.
// With `lens` (shared memory: q_len and prior context of the i-th chunk sequence, interleaved)
// the lengths need no global loads.
__device__ inline int pf_unit_bin(const AttnArgs& a, const int32_t* pf_seq, const int32_t* pf_prefix,
                           const int2* lens, int n_pf, int g) {
  int lo = 0, hi = n_pf - 1;  // largest i with pf_prefix[i] <= g
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pf_prefix[mid] <= g) lo = mid; else hi = mid - 1;
  }
  const int u = g - pf_prefix[lo];
  int q_len, ctx;
  if (lens != nullptr) {
    q_len = lens[lo].x;
    ctx = lens[lo].y;
  } else {
    const int s = pf_seq[lo];
    q_len = a.cu_seqlens_q[s + 1] - a.cu_seqlens_q[s];
    ctx = a.kv_lens[s] - q_len;
  }
  const int rows = min((u + 1) * pf_unit_tiles(a.G) * kPrefillTileM, q_len);
  const int first = window_first_key(ctx + u * pf_unit_tiles(a.G) * kPrefillTileM, a.window);
  const int tiles = (ctx + rows + kChunkKeys - 1) / kChunkKeys - first / kChunkKeys;
  return kCostBins - 1 - min(tiles, kCostBins - 1);
}

// Times that the planner weighs, in us of an SM, fitted to GB300 measurements: a step of a chain with
// one tile of rows, a chain's start and end, and a decode record's 16-key tile (0.8 at 64 KB: 8 KV
// heads of 128; 0.54 at 8 KB).
constexpr float kPreStepUs = 0.9f, kPreChainUs = 7.f;
__device__ __forceinline__ float pre_decode_tile_us(const AttnArgs& a) {
  return 0.5f + 0.3f * (float)((a.Hkv < 8 ? a.Hkv : 8) * a.D) * (1.f / 1024.f);
}

// Up to this many groups the planner keeps in shared memory (five arrays).
constexpr int kPlanSmemGroups = 768;

// What the first look at a sequence finds (kept for the second where one round covers the batch).
struct PreSeq {
  int c0, c1, kv, group, keys;
  // in batches of one round, for a sequence with a place in the token list:
  int list, at;     // its first entry (else -1), and that entry's place in the group's chain
  int chain;        // its own keys' group: PreGroup's cost0 (else -1)
  int own_first;    // and that group's first key (0: it is the sequence's only chain)
};

// Places of a round's members among their groups' tokens, in the order of the sequences, so that a
// token's tile, and with it the rounding of its parts, is the same on every call.  Returns the group's
// tokens listed before this thread's q (<= kPreMaxQ), and adds the round's to cnt; group -1: no member.
// Warps take turns, lanes of a group count the tokens of the lanes before them.  All threads call it.
__device__ __forceinline__ int group_place(int32_t* cnt, int group, int q, int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned peers = __match_any_sync(0xffffffffu, group), below = peers & ((1u << lane) - 1);
  int before = 0, total = 0;
#pragma unroll
  for (int b = 0; (1 << b) <= kPreMaxQ; ++b) {
    const unsigned bit = __ballot_sync(0xffffffffu, (q >> b) & 1);
    before += __popc(bit & below) << b;
    total += __popc(bit & peers) << b;
  }
  int at = 0;
  for (int w = 0; w < warps; ++w) {
    if (warp == w) {
      if (group >= 0) at = cnt[group];
      __syncwarp();
      if (group >= 0 && below == 0) cnt[group] = at + total;
    }
    __syncthreads();
  }
  return at + before;
}

// With shared prefixes: which groups' prefixes are computed once.  Fills the group list, and per
// group number map (index in the list, -1: every member's own pass does it all), first (its first
// entry of the token list), cost (cost0) and cnt (the tokens listed so far): in shared memory, since a
// look at the list itself is a trip to L2 (two of them: 0.3 us).  Returns the work of the prefixes per
// KV head in cost units (0: no group takes part; the same in every thread).
//
// A group takes part when it has at least two query tokens (from members with at most kPreMaxQ
// each) and kPreMinKeys keys; after bad metadata none does, and each sequence is computed alone.
// Sequences that are groups of their own (PreGroup; in batches of one round) follow the others in the
// list.
// lens: the groups' prefix lengths (in shared memory where all of them fit, else a.prefix_lens).
// period: CTAs per KV head that give each unit of a lone group a whole number of them (else 1).
__device__ __forceinline__ int plan_prefixes(const AttnArgs& a, int (*sw)[4], int32_t* cnt,
                                             int32_t* first, int32_t* map, int32_t* cost,
                                             const int32_t* lens,
                                             PreSeq& mine, int& period) {
  const PreLayout PL = pre_layout(a.S, a.R, a.LT, a.T, a.Hq, a.D, a.NG, a.pack);
  PreGroup* groups = reinterpret_cast<PreGroup*>(a.ws + PL.group);
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(a.ws + ws_layout(a.R, a.T, a.Hq, a.D, a.pack).header);
  const int tid = threadIdx.x;
  const long long max_kv = (long long)a.max_blocks * a.bs;
  __shared__ unsigned long long s_total, s_units;
  __shared__ int s_period;
  if (tid == 0) s_total = s_units = 0;
  for (int g = tid; g < a.NG; g += kPrePlanThreads) {
    cnt[g] = 0;
    first[g] = 0x7fffffff;
  }
  bool bad = false;
  for (int base = 0; base < a.S; base += kPrePlanThreads) {
    const int s = base + tid;
    PreSeq q = {0, 0, 0, -1, 0, -1, 0, -1, 0};
    if (s < a.S) {
      q.c0 = a.cu_seqlens_q[s];
      q.c1 = a.cu_seqlens_q[s + 1];
      q.kv = a.kv_lens[s];
      q.group = a.prefix_group[s];
    }
    const int q_len = q.c1 - q.c0;
    const bool lens_ok = !(q.c0 < 0 || q.c1 > a.T || (s == 0 && q.c0 != 0) || q_len < 0 ||
                           q.kv < q_len || q.kv > max_kv);
    if (base == 0) __syncthreads();  // cnt, first and lens are set
    bool group_ok = true, member = lens_ok && s < a.S && q_len > 0 && q.group != -1;
    if (member) {
      q.keys = q.group >= 0 && q.group < a.NG ? lens[q.group] : -1;
      group_ok = q.keys >= 0 && q.keys <= q.kv - q_len;
      if (!group_ok) report(a.err, kErrOutOfRange);
      member = group_ok && q_len <= kPreMaxQ;
    }
    bad |= !lens_ok || !group_ok;  // (bad lengths are reported by the caller)
    if (base == 0) mine = q;
    if (member) {
      atomicAdd(&cnt[q.group], q_len);
      atomicMin(&first[q.group], s);
    }
    // units of the chunk pass (a warp's sum first: 64-bit atomics on shared memory are slow)
    const int rows = pf_unit_tiles(a.G) * kPrefillTileM;
    const bool chunk = lens_ok && s < a.S && q_len > kPreMaxQ;
    if (__any_sync(0xffffffffu, chunk)) {
      unsigned long long n = chunk ? (unsigned long long)((q_len + rows - 1) / rows) : 0ull;
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      if ((tid & 31) == 0) atomicAdd(&s_units, n);
    }
  }
  bad = __syncthreads_or(bad) != 0;
  auto shared_tokens = [&](int g, int keys) {  // tokens of group g if its prefix is computed once
    return bad || g >= a.NG || cnt[g] < 2 || keys < kPreMinKeys ? 0 : cnt[g];
  };
  // This thread's sequence: a member, and its keys as a group of their own (0: not).
  const int my_q = mine.c1 - mine.c0, my_ctx = mine.kv - my_q;
  const bool one_round = !bad && a.S <= kPrePlanThreads;
  const bool my_member = one_round && my_q > 0 && my_q <= kPreMaxQ && mine.group >= 0 &&
                         shared_tokens(mine.group, mine.keys) > 0;
  const bool few_chunks =
      s_units * (unsigned long long)(pf_pair_heads(a.G) ? a.Hq / 2 : a.Hq) < kPreChunkItems;
  int own_nt = 0;
  if (my_member) {
    // its own keys as a group of their own, or as decode records: whatever takes fewer SM-us
    const int nt = pre_tiles(mine.keys, mine.kv), records = (my_q + a.pack - 1) / a.pack;
    const float as_chain = (float)a.Hkv * ((float)nt * kPreStepUs + kPreChainUs);
    const float as_records = (float)(records * pre_head_groups(a.Hkv, a.G)) *
                             (pre_decode_tile_us(a) * (float)((mine.kv - mine.keys) / kDecodeTileKeys + 1) + 1.f);
    if (records > 1 && as_chain < as_records) own_nt = nt;
  } else if (one_round && my_q > 1 && mine.kv >= kPreMinKeys &&
             (my_q <= kPreMaxQ || (few_chunks && my_ctx >= my_q))) {
    own_nt = pre_tiles(0, mine.kv);
  }
  auto work = [&](int n, int nt) { return pre_shape(n, nt, a.G).per; };
  auto set_period = [&](const PreShape& sh) {  // by the thread with the first group of the list
    s_period = sh.full == 0 ? 1 : sh.units > sh.full ? kPreCost2 * sh.full + kPreCost1 : sh.full;
  };
  const int own_cost =
      own_nt > 0 ? (int)min((long long)kPreMaxCost + 1, work(my_q, own_nt)) : 0;
  unsigned long long total = own_cost;
  for (int g = tid; g < a.NG; g += kPrePlanThreads) {
    const int n = shared_tokens(g, lens[g]);
    if (n > 0) total += (unsigned long long)work(n, pre_tiles(0, lens[g]));
  }
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if ((tid & 31) == 0 && total > 0) atomicAdd(&s_total, total);
  const bool any_own = __syncthreads_or(own_nt) != 0;
  const bool too_much = s_total > kPreMaxCost;  // (32 bits hold every cost below)
  bad |= too_much;
  int carry[4] = {0, 0, 0, 0};  // groups, tokens, cost, chains
  for (int base = 0; base < a.NG; base += kPrePlanThreads) {
    const int g = base + tid;
    const int keys = g < a.NG ? lens[g] : 0;
    const int n = shared_tokens(g, keys);
    int v[4] = {n > 0, n, 0, 0};
    PreShape sh = {};
    if (n > 0) {
      sh = pre_shape(n, pre_tiles(0, keys), a.G);
      v[2] = (int)sh.per;
      v[3] = sh.units;
    }
    int ex[4], tot[4];
    block_scan4<kPrePlanThreads>(v, ex, tot, sw);  // (its barriers also part the reads of cnt from the writes)
    if (n > 0) {
      groups[carry[0] + ex[0]] =
          {carry[2] + ex[2], n, carry[1] + ex[1], 0, keys, first[g], -1, 0};
      if (carry[0] + ex[0] == 0) set_period(sh);
    }
    if (g < a.NG) {
      map[g] = n > 0 ? carry[0] + ex[0] : -1;
      first[g] = carry[1] + ex[1];
      cost[g] = carry[2] + ex[2];
      cnt[g] = 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) carry[k] += tot[k];
  }
  if (!too_much && one_round) {
    __syncthreads();  // the groups and map are written, cnt is 0
    mine.at = group_place(cnt, my_member ? mine.group : -1, my_q, (a.S + 31) / 32);
    if (my_member) {
      mine.list = first[mine.group] + mine.at;
      mine.own_first = mine.keys;
    }
    if (any_own) {
      const PreShape sh = pre_shape(my_q, own_nt, a.G);
      int v[4] = {own_nt > 0, own_nt > 0 && !my_member ? my_q : 0, own_nt > 0 ? own_cost : 0,
                  own_nt > 0 ? sh.units : 0};
      int ex[4], tot[4];
      block_scan4<kPrePlanThreads>(v, ex, tot, sw);
      if (own_nt > 0) {
        mine.chain = carry[2] + ex[2];
        if (!my_member) {
          mine.list = carry[1] + ex[1];
          mine.at = 0;
        }
        groups[carry[0] + ex[0]] = {mine.chain, my_q,   mine.list, mine.own_first,
                                    mine.kv,    tid,    my_ctx,    my_member};
        if (carry[0] + ex[0] == 0) set_period(sh);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) carry[k] += tot[k];
    }
  }
  if (tid == 0) {
    hdr->pre_groups = carry[0];
    hdr->pre_tokens = carry[1];
    hdr->pre_cost = carry[2];
    hdr->pre_chains = carry[3];
  }
  __syncthreads();
  period = carry[0] == 1 ? s_period : 1;
  return carry[2];
}

// Prefix CTAs where `free` SMs are left to them and to `items` chunk items (up to a third of them for
// those, an SM per item: an item is mostly latency): as many for each KV head (PreGroup), where there
// are enough a multiple of `per` (Hkv x plan_prefixes' period), no more than the work is worth (`most`).
// (Quotients by reciprocals, exact for numbers below 1024: integer divisions cost the
// planner 0.2 us.)
struct PreRound {
  int Hkv, per;
  float inv_hkv, inv_per;
};
__device__ __forceinline__ PreRound pre_round(int Hkv, int per) {
  return {Hkv, per, __fdividef(1.f, (float)Hkv), __fdividef(1.f, (float)per)};
}
__device__ __forceinline__ int pre_cta_count(int free, int items, int most, const PreRound& m) {
  const int third = (free * 43691) >> 17;  // free / 3
  free -= items < third ? items : third;
  int np = free < most ? free : most;
  const bool whole = np > m.per;
  const int of = whole ? m.per : m.Hkv;
  if (np > of) np = of * (int)(((float)np + 0.5f) * (whole ? m.inv_per : m.inv_hkv));
  return np < 1 ? 1 : np;
}
__device__ __forceinline__ int pre_cta_most(int cost, int Hkv, int min_steps) {
  const long long most = (long long)cost * Hkv / (min_steps * kPreCost1);
  return most < kMaxPreCtas ? (int)most : kMaxPreCtas;
}

// Decode CTAs per head group where prefixes are computed apart; the other SMs are the prefixes'.
// Called by one full warp.  Model, in us:
//   decode = 7.2 + hypot(x, y): x the CTA's tiles (1.19 each at 64 KB, 0.87 at 8 KB; a record counts
//            as one more), y a share of the HBM time of their bytes;
//   prefix = 12 + 1.1 per cost unit of a CTA and 4.9 per chain; chunk work follows on the same SMs.
// The choice is the n with the least max(decode, prefix + chunk), plus a little of the other one and
// 0.019 a CTA for the parts it adds.  The constants are those with the least loss over every even n of
// 24 batches timed on a GB300 (4 to 256 sequences, 1 to 40 groups, prefixes of 300 to 64k keys, 1 to 8 KV
// heads, head_dim 64 and 128): the choice is within 3.5 % of the best n on all of them.
__device__ __forceinline__ int choose_prefix_split(const AttnArgs& a, float dec_bytes,
                                                   int cost, int chains, const PreRound& m, float chunk_flops,
                                                   int items, long long tiles, int records, int most) {
  const int lane = threadIdx.x & 31;
  const int hg = pre_head_groups(a.Hkv, a.G), sms = a.chunk_ctas;
  const int cap = (int)(tiles < a.decode_ctas ? tiles : a.decode_ctas);
  const float tile_us = 0.82f + 0.37f * (float)((a.Hkv < 8 ? a.Hkv : 8) * a.D) * (1.f / 1024.f);
  const float x1 = tile_us * ((float)tiles + (float)records);
  const float y = dec_bytes * 0.013e-6f;
  const float pre_us = (1.1f * (float)cost + 4.9f * (float)chains) * (float)a.Hkv;
  const float chunk_us = chunk_flops * (1.f / 6.4e6f);
  float best = 3.4e38f;
  int best_n = 1;
  for (int n = 2 * (lane + 1); n <= (cap > 2 ? cap : 2) && n * hg < sms; n += 64) {
    const int free = sms - n * hg;
    const float x = __fdividef(x1, (float)n), d = 7.2f + sqrt_approx(x * x + y * y);
    const float p = 12.f + __fdividef(pre_us,
                                      (float)pre_cta_count(free, items, most, m)) +
                    __fdividef(chunk_us, (float)free);
    const float t = fmaxf(d, p) + 0.018f * fminf(d, p) + 0.019f * (float)n;
    if (t < best) {
      best = t;
      best_n = n;
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    const float t = __shfl_xor_sync(0xffffffffu, best, o);
    const int n = __shfl_xor_sync(0xffffffffu, best_n, o);
    if (t < best || (t == best && n < best_n)) {
      best = t;
      best_n = n;
    }
  }
  return cap < 1 ? 1 : best_n < cap ? best_n : cap;
}

// Batches of up to this many decode (or chunk) sequences keep the planner's prefix arrays in
// shared memory as well, so its binary searches cost no global round trips.
constexpr int kPlanSmemSeqs = 2048;
// (with shared prefixes half as many, beside kPlanSmemGroups groups)
template <bool kPre>
constexpr int plan_smem_seqs() { return kPre ? kPlanSmemSeqs / 2 : kPlanSmemSeqs; }

// kPre: with shared prefixes (a.NG > 0).
template <bool kPre>
__device__ __forceinline__ void plan_cta(const AttnArgs& a) {
  constexpr int NT = plan_threads<kPre>();  // threads
  constexpr int kBins = kCostBins / NT;      // histogram bins per thread
  constexpr int kSeqs = plan_smem_seqs<kPre>();
  __shared__ int sw[32][4];
  __shared__ int32_t s_dec_prefix[kSeqs + 1], s_pf_prefix[kSeqs + 1];
  __shared__ int32_t s_pf_seq[kSeqs];
  __shared__ int2 s_pf_lens[kSeqs];  // (q_len, prior context) of each chunk sequence
  __shared__ int32_t s_groups[kPre ? 5 * kPlanSmemGroups : 1];
  const WsLayout L = ws_layout(a.R, a.T, a.Hq, a.D, a.pack);
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(a.ws + L.header);
  int32_t* dec_seq = reinterpret_cast<int32_t*>(a.ws + L.dec_seq);
  int32_t* dec_prefix = reinterpret_cast<int32_t*>(a.ws + L.dec_prefix);
  int4* dec_rec = reinterpret_cast<int4*>(a.ws + L.dec_rec);
  int32_t* cta_first = reinterpret_cast<int32_t*>(a.ws + L.cta_first);
  int32_t* pf_seq = reinterpret_cast<int32_t*>(a.ws + L.pf_seq);
  int32_t* pf_prefix = reinterpret_cast<int32_t*>(a.ws + L.pf_prefix);
  const int tid = threadIdx.x;
  const long long max_kv = (long long)a.max_blocks * a.bs;

  float my_keys = 0.f, my_pairs = 0.f;  // work estimates for the decode / chunk balance
  // shared prefixes: their work per KV head, and per group number what plan_prefixes finds
  int pre_cost = 0, period = 1;
  const PreLayout PL = kPre ? pre_layout(a.S, a.R, a.LT, a.T, a.Hq, a.D, a.NG, a.pack) : PreLayout{};
  const bool few = a.NG <= kPlanSmemGroups;
  int32_t* grp_cnt = few ? s_groups : reinterpret_cast<int32_t*>(a.ws + PL.cnt);
  int32_t* grp_first = few ? s_groups + kPlanSmemGroups : reinterpret_cast<int32_t*>(a.ws + PL.first);
  int32_t* grp_map = few ? s_groups + 2 * kPlanSmemGroups : reinterpret_cast<int32_t*>(a.ws + PL.map);
  int32_t* grp_cost = few ? s_groups + 4 * kPlanSmemGroups : reinterpret_cast<int32_t*>(a.ws + PL.cost);
  const int32_t* grp_lens = few ? s_groups + 3 * kPlanSmemGroups : a.prefix_lens;
  PreSeq mine = {0, 0, 0, -1, 0, -1, 0, -1, 0};
  if constexpr (kPre) {
    if (few)  // (the function's first barrier follows)
      for (int g = tid; g < a.NG; g += NT) s_groups[3 * kPlanSmemGroups + g] = a.prefix_lens[g];
    pre_cost = plan_prefixes(a, sw, grp_cnt, grp_first, grp_map, grp_cost, grp_lens, mine, period);
  }
  // kPre: chunks that are groups of their own: (first token, tokens, first list entry, K/V tiles), cost0
  __shared__ int s_chunks;
  __shared__ int4 s_chunk[kPre ? kPreChunkItems : 1][2];
  if (kPre && tid == 0) s_chunks = 0;  // (the loop's barriers follow)
  bool bad = false;
  const int unit_rows = pf_unit_tiles(a.G) * kPrefillTileM;
  int carry[4] = {0, 0, 0, 0};
  for (int base = 0; base < a.S; base += NT) {
    const int s = base + tid;
    int v[4] = {0, 0, 0, 0};
    int tok = 0, kv = 0, q_len = 0;
    int grp = -1, keys = 0;  // kPre: the group that computes this sequence's prefix, its length
    if (s < a.S) {
      int c0, c1;
      if (kPre && base == 0) {
        c0 = mine.c0;
        c1 = mine.c1;
        kv = mine.kv;
      } else {
        c0 = a.cu_seqlens_q[s];
        c1 = a.cu_seqlens_q[s + 1];
        kv = a.kv_lens[s];
      }
      q_len = c1 - c0;
      tok = c0;
      if (s == 0 && c0 != 0) report(a.err, kErrOutOfRange);  // cu_seqlens_q[0] must be 0
      const bool ok = c0 >= 0 && c1 <= a.T && q_len >= 0 && kv >= q_len && kv <= max_kv;
      if (!ok) {
        report(a.err, kErrOutOfRange);
        bad = true;
      } else if (kPre && base == 0 && mine.chain >= 0) {
        // all its own keys are a group of their own
      } else if (kPre && pre_cost > 0 && q_len > 0 && q_len <= kPreMaxQ &&
                 (grp = base == 0 ? mine.group : a.prefix_group[s]) >= 0 && grp_map[grp] >= 0) {
        // records of a.pack tokens: the tiles from the one holding the prefix's end to the one
        // holding the last key that the record's last token sees
        keys = grp_lens[grp];
        const int first = keys / kDecodeTileKeys * kDecodeTileKeys;
        for (int i = 0; i < q_len; i += a.pack) {
          v[0] += 1;
          v[1] += (kv - max(q_len - i - a.pack, 0) - first + kDecodeTileKeys - 1) / kDecodeTileKeys;
        }
        my_keys += (float)(kv - keys);
      } else if (q_len == 1) {
        grp = -1;
        // tiles from the one holding the window's first key (every key without a window)
        const int first = window_first_key(kv - 1, a.window) / kDecodeTileKeys * kDecodeTileKeys;
        v[0] = 1;
        v[1] = (kv - first + kDecodeTileKeys - 1) / kDecodeTileKeys;
        my_keys += (float)(kv - window_first_key(kv - 1, a.window));
      } else if (q_len > 1) {
        grp = -1;
        v[2] = 1;
        if (a.window > 0) {  // sum over the chunk's rows of min(position + 1, window)
          const float W = (float)a.window;
          for (int i = 0; i < q_len; i += 64) {
            const int i1 = min(i + 64, q_len);
            const float p0 = (float)(kv - q_len + i + 1), p1 = (float)(kv - q_len + i1);
            my_pairs += (i1 - i) * fminf(0.5f * (p0 + p1), W);
          }
        } else {
          my_pairs += (float)q_len * (float)(kv - q_len) + 0.5f * (float)q_len * (float)(q_len + 1);
        }
        v[3] = (q_len + unit_rows - 1) / unit_rows;  // work units (pf_unit_tiles)
      }
    }
    int ex[4], tot[4];
    block_scan4<NT>(v, ex, tot, sw);
    int at = mine.at;
    if constexpr (kPre) {
      if (a.S > NT && pre_cost > 0)  // (else plan_prefixes has found them)
        at = group_place(grp_cnt, v[0] ? grp : -1, q_len, (min(a.S - base, NT) + 31) / 32);
    }
    if (kPre && base == 0 && mine.chain >= 0) {
      const int own_nt = pre_tiles(mine.own_first, mine.kv);
      if (q_len > kPreMaxQ) {  // a chunk's list entries are written below, by all threads
        const int x = atomicAdd(&s_chunks, 1);  // (fewer than kPreChunkItems)
        s_chunk[x][0] = make_int4(tok, q_len, mine.list, own_nt);
        s_chunk[x][1] = make_int4(mine.chain, 0, 0, 0);
      } else {
        int4 shared = make_int4(0, 0, 0, 0);  // the prefix's chain
        if (mine.own_first > 0)
          shared = make_int4(mine.at, grp_cnt[mine.group], pre_tiles(0, mine.keys), grp_cost[mine.group]);
        for (int t = 0; t < q_len; ++t) {
          int4* entry = reinterpret_cast<int4*>(a.ws + PL.tok) + 3 * (size_t)(mine.list + t);
          const int4 own = make_int4(t, q_len, own_nt, mine.chain);
          entry[0] = make_int4(tok + t, -1, 0, 0);
          entry[1] = mine.own_first > 0 ? shared : own;
          entry[2] = mine.own_first > 0 ? own : make_int4(0, 0, 0, 0);
          ++shared.x;
        }
      }
    } else if (kPre && grp >= 0 && v[0]) {
      const int first = keys / kDecodeTileKeys * kDecodeTileKeys;
      // (all of the group's tokens are listed by now, unless the batch takes several rounds)
      const int n_tok = a.S <= NT ? grp_cnt[grp]
                                  : reinterpret_cast<const PreGroup*>(a.ws + PL.group)[grp_map[grp]].n_tok;
      const int tok0 = grp_first[grp], cost0 = grp_cost[grp];
      int tile = carry[1] + ex[1], i = carry[0] + ex[0];
      for (int j = 0; j < q_len; j += a.pack, ++i) {
        const int n = min(a.pack, q_len - j), n_keys = kv - (q_len - j - n);
        const int n_tiles = (n_keys - first + kDecodeTileKeys - 1) / kDecodeTileKeys;
        dec_seq[i] = s;
        dec_prefix[i] = tile;
        dec_rec[i] = make_int4(s, tok + j, n_keys, tile);
        if (i < kSeqs) s_dec_prefix[i] = tile;
        reinterpret_cast<int2*>(a.ws + PL.rec)[i] = make_int2(keys, n);
        for (int t = 0; t < n; ++t) {
          int4* entry = reinterpret_cast<int4*>(a.ws + PL.tok) + 3 * (size_t)(tok0 + at + j + t);
          entry[0] = make_int4(tok + j + t, 8 * i + t, tile, tile + n_tiles);
          entry[1] = make_int4(at + j + t, n_tok, pre_tiles(0, keys), cost0);
          entry[2] = make_int4(0, 0, 0, 0);
        }
        tile += n_tiles;
      }
    } else if (v[0]) {
      const int i = carry[0] + ex[0];
      if constexpr (kPre) reinterpret_cast<int2*>(a.ws + PL.rec)[i] = make_int2(0, 0);
      dec_seq[i] = s;
      dec_prefix[i] = carry[1] + ex[1];
      dec_rec[i] = make_int4(s, tok, kv, carry[1] + ex[1]);
      if (i < kSeqs) s_dec_prefix[i] = carry[1] + ex[1];
    }
    if (v[2]) {
      const int i = carry[2] + ex[2];
      pf_seq[i] = s;
      pf_prefix[i] = carry[3] + ex[3];
      if (i < kSeqs) {
        s_pf_seq[i] = s;
        s_pf_prefix[i] = carry[3] + ex[3];
        const int q_len = a.cu_seqlens_q[s + 1] - a.cu_seqlens_q[s];
        s_pf_lens[i] = make_int2(q_len, a.kv_lens[s] - q_len);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) carry[k] += tot[k];
  }
  if constexpr (kPre) {
    __syncthreads();
    for (int x = 0; x < s_chunks; ++x) {
      const int4 ch = s_chunk[x][0];
      const int cost0 = s_chunk[x][1].x;
      for (int t = tid; t < ch.y; t += NT) {
        int4* entry = reinterpret_cast<int4*>(a.ws + PL.tok) + 3 * (size_t)(ch.z + t);
        entry[0] = make_int4(ch.x + t, -1, 0, 0);
        entry[1] = make_int4(t, ch.y, ch.w, cost0);
        entry[2] = make_int4(0, 0, 0, 0);
      }
    }
  }
  // With every length valid the query ranges are disjoint, so the units fit pf_order (at most
  // S + T / 128); after an invalid length the chunk pass is given no work.
  bad = __syncthreads_or(bad) != 0;
  const int n_pf = carry[2];
  const int n_units = bad ? 0 : carry[3];
  if (tid == 0) {
    dec_prefix[carry[0]] = carry[1];
    dec_rec[carry[0]] = make_int4(-1, 0, 0, carry[1]);
    pf_prefix[carry[2]] = carry[3];
    if (carry[0] <= kSeqs) s_dec_prefix[carry[0]] = carry[1];
    if (carry[2] <= kSeqs) s_pf_prefix[carry[2]] = carry[3];
    hdr->n_dec = carry[0];
    hdr->dec_tiles = carry[1];
    hdr->n_pf = n_pf;
    hdr->pf_qtiles = n_units;
    hdr->pf_counter = 0;
    hdr->t_dec_start = hdr->t_pf_start = ~0ull;
    hdr->t_dec_end = hdr->t_pf_end = 0ull;
  }
  __syncthreads();
  // Chunk units longest first (a counting sort on the K/V tiles each streams, descending), so
  // that the chunk CTAs, taking items in this order from a shared counter, schedule them
  // longest-processing-time first.  Units of equal cost land in any order: each item writes
  // its own output rows, so the order never changes a result.  (n_units is the same in every
  // thread, so a batch without chunk work skips the section, barriers included.)
  if (n_units > 0) {
    __shared__ int hist[kCostBins];
    int32_t* pf_order = reinterpret_cast<int32_t*>(a.ws + L.pf_order);
    for (int i = 0; i < kBins; ++i) hist[kBins * tid + i] = 0;
    __syncthreads();
    const bool pf_local = n_pf <= kSeqs;
    const int32_t* ps = pf_local ? s_pf_seq : pf_seq;
    const int32_t* pp = pf_local ? s_pf_prefix : pf_prefix;
    const int2* lens = pf_local ? s_pf_lens : nullptr;
    for (int g = tid; g < n_units; g += NT)
      atomicAdd(&hist[pf_unit_bin(a, ps, pp, lens, n_pf, g)], 1);
    __syncthreads();
    int v[4] = {0, 0, 0, 0}, ex[4], tot[4];
    for (int i = 0; i < kBins; ++i) v[0] += hist[kBins * tid + i];
    block_scan4<NT>(v, ex, tot, sw);
    for (int i = 0; i < kBins; ++i) {
      const int n = hist[kBins * tid + i];
      hist[kBins * tid + i] = ex[0];
      ex[0] += n;
    }
    __syncthreads();
    for (int g = tid; g < n_units; g += NT)
      pf_order[atomicAdd(&hist[pf_unit_bin(a, ps, pp, lens, n_pf, g)], 1)] = g;
  }
  // First decode sequence of each decode CTA: CTA c owns tiles [c*n/N, (c+1)*n/N), with N
  // capped at the tile count so that no CTA range is empty.
  const int n_dec = carry[0];
  const long long ntiles = carry[1];
  __shared__ int s_N;
  __shared__ float s_red[2][NT / 32];
  // fixed-order reduction, so that the CTA count (and with it the rounding of the split-KV
  // merge) is the same on every call with the same lengths
  for (int o = 16; o > 0; o >>= 1) {
    my_keys += __shfl_xor_sync(0xffffffffu, my_keys, o);
    my_pairs += __shfl_xor_sync(0xffffffffu, my_pairs, o);
  }
  if ((tid & 31) == 0) {
    s_red[0][tid >> 5] = my_keys;
    s_red[1][tid >> 5] = my_pairs;
  }
  __syncthreads();
  if (tid < 32) {
    float keys = 0.f, pairs = 0.f;
    if constexpr (kPre) {
      keys = tid < NT / 32 ? s_red[0][tid] : 0.f;
      pairs = tid < NT / 32 ? s_red[1][tid] : 0.f;
      for (int o = 16; o > 0; o >>= 1) {
        keys += __shfl_xor_sync(0xffffffffu, keys, o);
        pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
      }
    } else {
      for (int w = 0; w < NT / 32; ++w) {
        keys += s_red[0][w];
        pairs += s_red[1][w];
      }
    }
    int n = (int)(ntiles < a.decode_ctas ? (ntiles > 0 ? ntiles : 1) : a.decode_ctas);
    if (kPre && pre_cost > 0) {
      const PreRound m = pre_round(a.Hkv, a.Hkv * period <= kPrePeriod ? a.Hkv * period : a.Hkv);
      const float row = (float)(a.Hkv * a.D * 4);  // bytes of a key and its value
      const int items = n_units * (pf_pair_heads(a.G) ? a.Hq / 2 : a.Hq);
      const int most = pre_cta_most(pre_cost, a.Hkv, pre_min_steps((long long)hdr->pre_tokens * a.Hq));
      if (a.decode_auto)
        n = choose_prefix_split(a, keys * row, pre_cost,
                                hdr->pre_chains, m,
                                pairs * (float)(4 * a.D * a.Hq), items, ntiles, n_dec, most);
      // the decode CTAs without work; where a given number leaves none, an eighth of the chunk CTAs
      const int idle = pre_idle_count(pre_head_groups(a.Hkv, a.G), n, a.decode_ctas);
      if (tid == 0)
        hdr->pre_ctas = pre_cta_count(idle > 0 ? idle : a.chunk_ctas / 8, items, most, m);
    } else if (a.decode_auto) {
      n = choose_decode_ctas(keys * (float)(a.Hkv * a.D * 4), pairs * (float)(4 * a.D * a.Hq),
                             n_units * (pf_pair_heads(a.G) ? a.Hq / 2 : a.Hq), a.decode_ctas,
                             ntiles);
    }
    if (kPre && pre_cost == 0 && tid == 0) hdr->pre_ctas = 0;
    if (tid == 0) {
      s_N = n;
      hdr->decode_ctas = n;
    }
  }
  __syncthreads();
  const int N = s_N;
  // Merge counters of the decode pass: one per (decode sequence, KV head), zero at start.
  int32_t* merge_cnt = reinterpret_cast<int32_t*>(a.ws + L.merge_cnt);
  // (one per decode sequence, KV head and group of 8 query heads: two groups when G > 8)
  const int head_groups = a.G > 8 ? 2 : 1;
  for (int i = tid; i < n_dec * a.Hkv * head_groups; i += NT) merge_cnt[i] = 0;
  // Indexed by the grid's decode CTA, so that a CTA reads its first sequence in the same round
  // trip as the plan header.
  const int32_t* dp = n_dec <= kSeqs ? s_dec_prefix : dec_prefix;
  for (int bx = tid; bx < a.decode_ctas; bx += NT) {
    const int c = decode_cta_index(bx, N, a.decode_ctas);
    int lo = -1;
    if (c >= 0 && c < N) {
      const long long t0 = ntiles * c / N;
      lo = 0;
      int hi = n_dec;  // largest d in [0, n_dec] with dec_prefix[d] <= t0
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (dp[mid] <= t0) lo = mid; else hi = mid - 1;
      }
    }
    cta_first[bx] = lo;
  }
}

// Both planner launches let the attention kernel that follows them on the stream start early
// (it is launched as their programmatic dependent and waits for their completion itself).
__device__ __forceinline__ void allow_dependent_launch() {
  asm volatile("griddepcontrol.launch_dependents;");
}

}  // namespace cb

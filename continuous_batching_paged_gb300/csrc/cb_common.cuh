// Shared device helpers for libcb: error word, bounded mbarrier waits, TMA, warp MMA and
// tcgen05 (5th-generation tensor core) wrappers.  sm_103a only.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/cb.h"

namespace cb {

// Bits of the per-device error word.
constexpr uint32_t kErrOutOfRange = 1u;
constexpr uint32_t kErrTimeout = 2u;

// A device-side wait gives up after this many nanoseconds of %globaltimer.
constexpr uint64_t kWaitLimitNs = 1000ull * 1000ull * 1000ull;  // 1 s

constexpr int kDecodeTileKeys = 16;     // keys per decode pipeline stage
constexpr int kPrefillTileM = 128;      // queries per prefill tile (TMEM lanes)
constexpr int kChunkKeys = 128;         // keys per K/V tile of the chunk pass
constexpr int kMaxDecodeHeadsPerCta = 8;

// A chunk-pass CTA runs two 128-query tiles A and B against the same K/V tiles.  With an even
// GQA group size they are one query tile under two query heads of one KV group (equal key
// ranges); otherwise two consecutive query tiles under one head.  A "unit" is what one item
// covers under one head (pair): 1 tile or 2 tiles.
__host__ __device__ inline bool pf_pair_heads(int G) { return (G & 1) == 0; }
__host__ __device__ inline int pf_unit_tiles(int G) { return pf_pair_heads(G) ? 1 : 2; }

constexpr int kCostBins = 1024;  // histogram bins of the planner's longest-first unit order

// Sliding window: the first key a query at absolute position p sees (0 without a window).
__host__ __device__ inline int window_first_key(int p, int window) {
  return (window > 0 && p >= window) ? p - window + 1 : 0;
}

// %globaltimer (ns since an arbitrary origin, the same on every SM).
__device__ __forceinline__ unsigned long long global_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Workspace header (int32 words).
struct PlanHeader {
  int32_t n_dec;          // number of decode sequences (q_len == 1)
  int32_t dec_tiles;      // total 16-key tiles over all decode sequences
  int32_t n_pf;           // number of chunk sequences (q_len > 1)
  int32_t pf_qtiles;      // total work units over all chunk sequences (pf_unit_tiles)
  int32_t pf_counter;     // dynamic work counter of the prefill pass (reset by the planner)
  int32_t decode_ctas;    // CTAs the decode pass was planned for
  int32_t pre_groups;     // shared prefixes (only with them): groups whose prefix is computed once,
  int32_t pre_ctas;       // CTAs that do it (0: no such group),
  // %globaltimer stamps (ns) of the attention kernel's roles, reset by the planner: first
  // start and last end of the decode CTAs that had work, and of the chunk CTAs.
  unsigned long long t_dec_start, t_dec_end, t_pf_start, t_pf_end;
  int32_t pre_cost;         // their work per KV head, in cost units (PreGroup),
  int32_t pre_tokens;       // entries of the groups' token list,
  int32_t pre_chains;       // and their chains per KV head
  // of claim_range (cb_place.cuh), reset by the planner: decode CTAs that have arrived (high half), and
  // ranges that they took
  unsigned long long dec_claims;
};

// Byte offsets of the workspace sections (all 256-byte aligned).
struct WsLayout {
  size_t header, dec_seq, dec_prefix, dec_rec, cta_first, pf_seq, pf_prefix, pf_order, merge_cnt,
      part_ml, part_o, total;
};

__host__ __device__ inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// S: the most decode records and the most chunk sequences (the sequences; with shared prefixes,
// pre_records).  pack: query tokens of a decode record at most (1; with shared prefixes, pre_pack).
__host__ __device__ inline WsLayout ws_layout(int S, int T, int Hq, int D, int pack = 1) {
  WsLayout L;
  size_t off = 0;
  L.header = off;     off = align_up(off + sizeof(PlanHeader), 256);
  L.dec_seq = off;    off = align_up(off + sizeof(int32_t) * (size_t)(S + 1), 256);
  L.dec_prefix = off; off = align_up(off + sizeof(int32_t) * (size_t)(S + 1), 256);
  // per decode sequence (sequence, query token, kv_len, first tile) in one 16-byte record, so
  // that the decode pass gets a sequence's metadata in one load
  L.dec_rec = off;    off = align_up(off + sizeof(int32_t) * 4 * (size_t)(S + 1), 256);
  // per decode CTA of the grid: the decode sequence holding its first tile, -1 if it is idle
  L.cta_first = off;  off = align_up(off + sizeof(int32_t) * (size_t)(CB_MAX_DECODE_CTAS + 1), 256);
  L.pf_seq = off;     off = align_up(off + sizeof(int32_t) * (size_t)(S + 1), 256);
  L.pf_prefix = off;  off = align_up(off + sizeof(int32_t) * (size_t)(S + 1), 256);
  // chunk units, longest first: at most one per 128 query tokens plus one per sequence
  L.pf_order = off;   off = align_up(off + sizeof(int32_t) * ((size_t)S + (size_t)T / kPrefillTileM + 1), 256);
  L.merge_cnt = off;  off = align_up(off + sizeof(int32_t) * (size_t)S * (size_t)Hq, 256);
  const size_t slots = (size_t)CB_MAX_DECODE_CTAS + (size_t)S;
  const size_t part_rows = slots * (size_t)pack * (size_t)Hq;
  L.part_ml = off;    off = align_up(off + sizeof(float2) * part_rows, 256);
  L.part_o = off;     off = align_up(off + sizeof(float) * part_rows * (size_t)D, 256);
  L.total = off;
  return L;
}

// ------------------------------------------------------------------------------------------
// Shared prefixes (cb_prefix.cuh).  The query tokens of a group's members with at most kPreMaxQ each
// go into the group's tiles of kPrefillTileM rows for the prefix.  For its own keys a member gets
// decode records of up to pre_pack tokens; with more than one, where that is estimated to be cheaper
// (long own keys, few KV heads), it is a group of its own for them, with a causal edge at their end: a
// K/V tile of 128 keys costs the tensor cores 0.9 us for one KV head and all its rows, the decode pass
// 0.8 us per 16 keys, 8 KV heads and record.  A sequence outside the groups with 2 to kPreMaxQ tokens
// is such a group, too.  Longer ones (chunks) run the chunk pass, which sharing saves nothing: but
// where its work items are fewer than kPreChunkItems, so that it would leave SMs idle, a chunk after
// at least its own length of keys is such a group too, cut to equal shares like the others.  Groups of one
// sequence are planned in batches of up to kPrePlanThreads sequences, which the planner sees at once; in
// larger ones members of several tokens have records, and other sequences of several tokens the chunk pass.
constexpr int kPreMaxQ = 8;
constexpr int kPrePlanThreads = 256;  // of the planner (cb_plan.cuh); sequences it sees at once
constexpr int kPreChunkItems = 152;
// Tokens of one sequence that a decode warp's 8 columns hold with G query heads each.
__host__ __device__ inline int pre_pack(int G) { return G <= 8 ? 8 / G : 1; }
// Prefixes shorter than one K/V tile are left to each sequence's own pass.
constexpr int kPreMinKeys = kChunkKeys;
constexpr int kMaxPreCtas = 160;   // CTAs of the prefix pass (at most one per SM)
// A chain's start and end cost 8 us besides its steps (rows and first tiles loaded, the part written),
// and a CTA whose range holds the end of one chain and the start of another pays them twice: 128
// sequences on 4096 keys (2 units under each of 8 KV heads) took 59.4 us on 48 CTAs, none of which
// does, and 70.4 on 40; 40 sequences on 30k keys under one KV head 41.7 us on 96 and 50.4 on 98.  So a
// lone group gets a multiple of the CTAs that make up whole ones for every unit, in proportion to its
// steps' cost, where that is kPrePeriod or less.  (Counting a start as 11 cost units instead, so that such a CTA gets
// fewer steps, helped several groups by 2 % and cost the rest 1 us of planning.)
constexpr int kPrePeriod = 32;
// K/V tiles per CTA at least: more CTAs end sooner but leave the merge more parts per row (16 rows of
// 500 keys: 20.8 us with at least 3, 17.9 with 1; 1024 rows of 2000 keys: 29.1 and 32.4).
__host__ __device__ inline int pre_min_steps(long long rows) { return rows <= 512 ? 1 : 3; }

// Query tokens per tile: all G query heads of a KV head, token by token.
__host__ __device__ inline int pre_tile_tokens(int G) { return kPrefillTileM / G; }
// What a batch may need at most, whatever its lengths (the host does not know them).
// Decode records of up to `pack` tokens: those of kPreMaxQ tokens per sequence, and
// sum ceil(q / pack) <= (T + S (pack - 1)) / pack; at least S, as the lists of sequences are as long.
__host__ __device__ inline int pre_records(int S, int T, int pack) {
  const long long by_seq = (long long)S * ((kPreMaxQ + pack - 1) / pack);
  const long long by_tok = ((long long)T + (long long)S * (pack - 1)) / pack;
  const long long most = by_seq < by_tok ? by_seq : by_tok;
  return most > S ? (int)most : S;
}
// Query tokens with two chains: those of a prefix's members with a group of their own keys.
__host__ __device__ inline int pre_second(int S, int T) {
  const int most = S <= kPrePlanThreads ? S * kPreMaxQ : 0;
  return most < T ? most : T;
}
// Entries of the token list: kPreMaxQ per sequence and, where the planner sees all sequences at once,
// what fewer than kPreChunkItems chunk items hold (an item is 2 x 128 rows).
__host__ __device__ inline int pre_tokens(int S, int T, int Hq) {
  const long long most = (long long)S * kPreMaxQ +
                         (S <= kPrePlanThreads ? kPreChunkItems * 2 * kPrefillTileM / Hq : 0);
  return most < T ? (int)most : T;
}

// One group whose prefix is computed once.  Its query tokens make tiles, two tiles (the last time
// maybe one) make a unit, and a chain is one unit under one KV head against all K/V tiles of the
// prefix.  A step (one K/V tile) of a chain costs kPreCost2 units with two tiles of rows, kPreCost1
// with one.  All chains are laid end to end, all groups' units under KV head 0 first, then the same
// under KV head 1, ..., and cut into equal ranges of cost, one per CTA.  With as many CTAs for each
// KV head, those of all heads walk the same keys at the same time and HBM sees their pieces of a
// token's row (D * 2 bytes each) together: 64k shared keys, 24 sequences, 8 KV heads: 144 CTAs read
// at 5.3 TB/s where 146 read at 4.8 (head_dim 64: 4.0 and 3.0).
constexpr int kPreCost2 = 3, kPreCost1 = 2;
constexpr int kPreMaxCost = 1 << 28;  // per KV head; a batch beyond it is computed without sharing
struct PreGroup {
  int32_t cost0;    // where its first chain under a KV head starts, from the head's start
  int32_t n_tok;    // query tokens
  int32_t tok0;     // its first entry of the token list
  int32_t first;    // its keys: first .. keys - 1
  int32_t keys;
  int32_t seq;      // the sequence whose block table is read (the first member)
  int32_t ctx;      // -1: every token sees all the keys; else token i sees those up to ctx + i
  int32_t second;   // 1: its tokens have another chain, so its parts' rows are the second ones
};

// Entry of the token list: a query token whose keys are (in part) computed apart, with all that the
// merge needs to find its parts, in three 16-byte loads.
struct PreToken {
  int32_t token;         // packed token
  int32_t rec;           // 8 x its decode record + its place among the record's tokens; -1: none
  int32_t tile0, tile1;  // that record's tiles among all decode tiles
  struct {               // its chains (the second: nt 0 if there is none)
    int32_t at;          // its place among the group's tokens
    int32_t n_tok, nt, cost0;  // of the group (nt: K/V tiles)
  } chain[2];
};

// Sections of the workspace behind ws_layout's (all 256-byte aligned).  R: pre_records, LT: pre_tokens.
// `second` (pre_second) counts for the total alone, so that the kernels need not know it.
struct PreLayout {
  size_t rec, cnt, first, map, cost, group, tok, cut_ml, cut_o, base_ml, base_o, total;
};
__host__ __device__ inline PreLayout pre_layout(int S, int R, int LT, int T, int Hq, int D, int NG,
                                               int pack, int second = 0) {
  PreLayout L;
  size_t off = ws_layout(R, T, Hq, D, pack).total;
  // per decode record: keys of the prefix computed apart and query tokens, or zeros
  L.rec = off;     off = align_up(off + sizeof(int32_t) * 2 * (size_t)(R + 1), 256);
  // per group number: query tokens (then: tokens listed so far), first member (then: its first entry
  // of the token list), index in the list of groups, cost0
  L.cnt = off;     off = align_up(off + sizeof(int32_t) * (size_t)(NG + 1), 256);
  L.first = off;   off = align_up(off + sizeof(int32_t) * (size_t)(NG + 1), 256);
  L.map = off;     off = align_up(off + sizeof(int32_t) * (size_t)(NG + 1), 256);
  L.cost = off;    off = align_up(off + sizeof(int32_t) * (size_t)(NG + 1), 256);
  L.group = off;   off = align_up(off + sizeof(PreGroup) * (size_t)(NG + kPrePlanThreads + 1), 256);
  L.tok = off;     off = align_up(off + sizeof(PreToken) * (size_t)(LT + 1), 256);
  // Partial results of a chain: a part that a CTA's range begins with in the CTA's own 2 x 128 rows, the
  // part with the chain's first K/V tile in a row per (token list entry, query head), for an entry's
  // second chain LT entries further (the groups' members, who have those, are listed first).
  const size_t cut_rows = (size_t)kMaxPreCtas * 2 * kPrefillTileM;
  L.cut_ml = off;  off = align_up(off + sizeof(float2) * cut_rows, 256);
  L.cut_o = off;   off = align_up(off + sizeof(float) * cut_rows * (size_t)D, 256);
  const size_t ml_rows = (size_t)LT * (size_t)(S <= kPrePlanThreads ? 2 : 1) * (size_t)Hq;
  L.base_ml = off; off = align_up(off + sizeof(float2) * ml_rows, 256);
  L.base_o = off;
  off = align_up(off + sizeof(float) * (size_t)(LT + second) * (size_t)Hq * (size_t)D, 256);
  L.total = off;
  return L;
}

#if defined(__CUDACC__)

// Working index of decode CTA bx of a grid of `grid` decode CTAs when N of them work, -1 if bx
// is idle.  With N below the grid size the working CTAs are spread evenly over the grid, in
// pairs of consecutive CTAs where N and the grid are even: CTA b (or pair b/2) works when it is
// the first with its value of floor(b N / grid), and takes that value's range.  The block
// scheduler puts consecutive CTAs on the two SMs of a TPC and deals TPCs out across the GPCs.
// Measured beside a chunk pass: with the first N CTAs working the decode pass ran ~6% slower;
// with single CTAs spread, decode and chunk CTAs shared TPCs and the chunk pass ran ~5% slower;
// spread pairs ran both at the speed of a launch of exactly N CTAs.
__device__ __forceinline__ int decode_cta_index(int bx, int N, int grid) {
  if (N >= grid) return bx;
  const bool pairs = ((N | grid) & 1) == 0;
  const int units = pairs ? grid / 2 : grid, wanted = pairs ? N / 2 : N;
  const int u = pairs ? bx >> 1 : bx;
  const int cu = u * wanted / units;  // (both at most CB_MAX_DECODE_CTAS)
  if (u > 0 && (u - 1) * wanted / units == cu) return -1;
  return pairs ? 2 * cu + (bx & 1) : cu;
}

// A decode CTA of the grid with working index c.
__device__ __forceinline__ int decode_cta_of(int c, int N, int grid) {
  if (N >= grid) return c;
  const bool pairs = ((N | grid) & 1) == 0;
  const int units = pairs ? grid / 2 : grid, wanted = pairs ? N / 2 : N, cu = pairs ? c >> 1 : c;
  const int u = (cu * units + wanted - 1) / wanted;
  return pairs ? 2 * u + (c & 1) : u;
}

__device__ __forceinline__ void report(uint32_t* err, uint32_t bit) { atomicOr(err, bit); }

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------------------------------------
// mbarrier
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void fence_barrier_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Non-blocking test: has the phase of parity `parity` completed?
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Wait for the phase of parity `parity` to complete; false after `limit_ns` of %globaltimer.
__device__ __forceinline__ bool mbar_wait_for(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait(bar, parity)) return true;
    if (globaltimer_ns() - t0 > limit_ns) return false;
  }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  return mbar_wait_for(bar, parity, kWaitLimitNs);
}

// ------------------------------------------------------------------------------------------
// TMA (bulk tensor copies global -> shared, completion through an mbarrier transaction count)
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// The same load with an L2 eviction-priority policy (from l2_policy_evict_first).
__device__ __forceinline__ void tma_load_3d_hint(uint32_t dst, const CUtensorMap* map,
                                                 uint32_t bar, int c0, int c1, int c2,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

// Bulk prefetch of `bytes` (a multiple of 16) at `p` (16-byte aligned) into L2: a hint, no
// completion to wait for.
__device__ __forceinline__ void l2_prefetch_bulk(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(p)),
               "r"(bytes)
               : "memory");
}

// L2 policy for data read once (streamed K/V of decode tokens): its lines are the first to go,
// so data that other work re-reads stays in L2.
__device__ __forceinline__ uint64_t l2_policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// The policy of a load without one.
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// ------------------------------------------------------------------------------------------
// Warp-level tensor-core helpers (ldmatrix + mma.sync m16n8k16, bf16 in, fp32 accumulate)
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                        uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                          uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16_16816(float* c, const uint32_t* a, uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mbar_inval(uint32_t bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// Transpose an 8x8 matrix of 16-bit elements held in the mma fragment layout (thread i: row
// i / 4, columns 2 (i % 4) and 2 (i % 4) + 1) across the warp.
__device__ __forceinline__ uint32_t movm_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Hardware base-2 exponential (the MUFU approximation; exp2(-inf) = 0).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Packed pairs of fp32 values in one 64-bit register, for the paired fp32 instructions
// (fma / add on f32x2), which issue one instruction for two lanes of work.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// max of three fp32 values in one instruction
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Address of 16-byte chunk `chunk` (0..7) of 128-byte row `row` in a region laid out by TMA
// with the 128-byte swizzle: the chunk index is XORed with the row index modulo 8.
__device__ __forceinline__ uint32_t sw128(uint32_t region, uint32_t row, uint32_t chunk) {
  return region + row * 128u + (((chunk ^ row) & 7u) << 4);
}

// One lane of a fully active warp is elected (the same lane every time); the rest skip.  Used
// so that a warp runs the tcgen05 issue loop with warp-uniform control flow while a single
// thread issues the MMAs and the commits that track them.
__device__ __forceinline__ bool elect_one() {
  uint32_t pred;
  asm volatile(
      "{\n\t.reg .b32 r;\n\t.reg .pred p;\n\t"
      "elect.sync r|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// Register reallocation between warpgroups (all four warps of a warpgroup execute it).  The
// counts handed out must add up to no more than what the block was launched with.
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// ------------------------------------------------------------------------------------------
// tcgen05: tensor memory allocation, MMA issue, commit, and TMEM <-> register moves.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// D[tmem] (+)= A[smem desc] * B[smem desc]
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem desc]
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on an mbarrier once every tcgen05.mma issued so far by this thread has completed.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

#define CB_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                 "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define CB_W8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                 "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 consecutive 32-bit TMEM columns of this thread's lane -> r[0..31].
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : CB_R8(0), CB_R8(8), CB_R8(16), CB_R8(24)
      : "r"(taddr));
}
// r[0..31] -> 32 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(
          taddr),
      CB_W8(0), CB_W8(8), CB_W8(16), CB_W8(24)
      : "memory");
}

// Shared-memory matrix descriptor of the 5th-generation tensor core: start address, leading
// and stride byte offsets (all >> 4), descriptor version 1, and the 128-byte swizzle mode.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo & 0x3FFFFu) >> 4) << 16;
  d |= (uint64_t)((sbo & 0x3FFFFu) >> 4) << 32;
  d |= (uint64_t)1 << 46;  // version
  d |= (uint64_t)2 << 61;  // 128-byte swizzle
  return d;
}
// Instruction descriptor, kind::f16: fp32 accumulator, bf16 A and B, A K-major, B K-major
// (b_mn_major = 0) or MN-major (1), tile M x N.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int b_mn_major) {
  return (1u << 4)                      // D format: f32
         | (1u << 7)                    // A format: bf16
         | (1u << 10)                   // B format: bf16
         | ((uint32_t)b_mn_major << 16)  // B major-ness
         | ((uint32_t)(N >> 3) << 17)   // N / 8
         | ((uint32_t)(M >> 4) << 24);  // M / 16
}

#endif  // __CUDACC__

}  // namespace cb

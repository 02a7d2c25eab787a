// Prefix role of the attention kernel: a group's query rows against the keys that all its members
// share (tcgen05 tensor cores, K/V streamed by TMA).
//
// Rows are query tokens x the G query heads of one KV head, 128 to a tile, gathered by TMA (a box
// of G rows per token, from the group's token list); every row sees every key of a shared prefix, so
// there is no mask but at the keys' ends and, for groups that are one sequence's own keys, its causal
// edge.  A CTA does an equal share of all prefixes' work: a contiguous range of the
// chains (PreGroup) laid end to end, whose parts of chains it takes one after the other.  With two
// tiles of rows both read the same K/V tiles (as in the chunk pass) and the softmax bounds the step
// (16 K exponentials a tile and SM); with one tile a step is bound by the K/V bytes (64 KB a step,
// 1.4 us of an SM's share of HBM), so the ring holds five 32 KB K or V tiles in flight (160 KB; the
// latency of HBM covers about 70), and the K/V tiles alternate between the two softmax groups with
// an accumulator each, so that the two products and the softmax of a step overlap with the next
// step's.  The two accumulators are joined in TMEM at the part's end.
//
//   warp 0      TMA producer.  Order with one tile: K0, then K(i), V(i-1); with two: K(i), V(i).
//   warp 1      tcgen05 issuer (as in the chunk pass): S_t(i) = Q K_i^T, O_t += P_t(i) V_i.
//   warps 4-7   softmax group 0 (tile A, or the even K/V tiles), warps 8-11 group 1 (tile B, or the
//               odd ones): thread r owns row r; running max and sum in registers, P over S in
//               TMEM.  Warps whose rows hold no query only take part in the barriers.
// P is rounded to bf16 for its product with V, as in the other roles (the tensor cores take both operands
// in one type, and the cache holds bf16): half a step, 2^-8, of each p, while the row sums add p before the
// rounding.  Against 64 bits the outputs are off by 0.0023 of their norm; an fp32 P would leave 0.0017, the
// rounding of the output itself.
// TMEM columns: [0,128) S/P of 0, [128,256) S/P of 1, [256,256+D) O of 0, then O of 1.
#pragma once

#include "cb_launch.h"
#include "cb_pre_parts.cuh"

namespace cb {

template <int D>
struct PreSmem {
  static constexpr int kHalves = D / 64;
  static constexpr int kHalf = 128 * 128;              // 128 rows (queries or keys) of 128 B
  static constexpr int kTile = kHalves * kHalf;        // a Q, K or V tile
  static constexpr int kSlots = D == 128 ? 5 : 12;     // ring of K or V tiles
  static constexpr int kRing = 2 * kTile;              // Q_A and Q_B first
  static constexpr int kBar = kRing + kSlots * kTile;
  static constexpr int bQFull = 0, bQEmpty = 1, bFull = 2, bEmpty = bFull + kSlots,
                       bSFull = bEmpty + kSlots, bPFull = bSFull + 2, bOFinal = bPFull + 2,
                       bOFree = bOFinal + 1, bStat = bOFree + 1, bWeight = bStat + 1,
                       kNumBars = bWeight + 1;
  static constexpr int kMisc = (kBar + kNumBars * 8 + 127) / 128 * 128;  // TMEM base
  static constexpr int kXch = kMisc + 64;              // (m, l), then weights, per row
  static constexpr int kTotal = kXch + 128 * 8 + 1024;
};
static_assert(PreSmem<128>::kTotal <= 232448 && PreSmem<64>::kTotal <= 232448, "shared memory");

// CTA `c` < hdr->pre_ctas of the prefix role (all kPrefillThreads threads).
template <int D>
__device__ __forceinline__ void prefix_cta(const AttnArgs& a, const CUtensorMap* qmap,
                                           const CUtensorMap* qmap_run, const CUtensorMap* kmap,
                                           const CUtensorMap* vmap, uint8_t* smem_raw, int c) {
  using SM = PreSmem<D>;
  constexpr int NS = SM::kSlots;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(a.ws + ws_layout(a.R, a.T, a.Hq, a.D, a.pack).header);
  const int N = hdr->pre_ctas;
  const PreLayout PL = pre_layout(a.S, a.R, a.LT, a.T, a.Hq, a.D, a.NG, a.pack);
  const PreToken* list = reinterpret_cast<const PreToken*>(a.ws + PL.tok);
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) -> uint32_t { return sbase + SM::kBar + 8 * i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + SM::kMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(bar(SM::bQFull), 1);
    mbar_init(bar(SM::bQEmpty), 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(SM::bFull + i), 1);
      mbar_init(bar(SM::bEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(SM::bSFull + i), 1);
      mbar_init(bar(SM::bPFull + i), 4);  // one arrival per softmax warp
    }
    mbar_init(bar(SM::bOFinal), 1);
    mbar_init(bar(SM::bOFree), 8);        // the warps of both groups
    mbar_init(bar(SM::bStat), 4);
    mbar_init(bar(SM::bWeight), 4);
    fence_barrier_init();
    atomicMin(&hdr->t_pf_start, global_ns());
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), kTmemCols);
    tmem_relinquish();
  }
  PreWalk walk(reinterpret_cast<const PreGroup*>(a.ws + PL.group), hdr->pre_groups, a.G,
               a.Hkv, hdr->pre_cost, c, N);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PreSeg s;

  if (warp < 4) {
    regs_dec<kRegsIssue>();
    if (warp == 0) {
      // =================================================================== TMA producer
      if (lane == 0) {
        tma_prefetch_desc(qmap_run);
        tma_prefetch_desc(qmap);
        tma_prefetch_desc(kmap);
        tma_prefetch_desc(vmap);
      }
      // A tile is nsb page runs of KB keys (a power of two; a box each per half of D).  Each lane
      // keeps the pool row of one run, 32 / nsb tiles at a time, so block-table loads and divisions
      // are one per 32 runs, and the next 32 are loaded a batch ahead.
      const int KB = a.KBp, nsb = kChunkKeys / KB;  // 1 .. 128
      const int per_batch = nsb < 32 ? 32 / nsb : 1, batches = nsb < 32 ? 1 : nsb / 32;
      uint32_t g = 0;
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t parity) {  // by lane 0, for the warp
        if (lane == 0 && ok && !mbar_wait(b, parity)) {
          report(a.err, kErrTimeout);
          ok = false;
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      };
      for (uint32_t k = 0; ok && walk.next(s); ++k) {
        const int n = s.j1 - s.j0;
        const int n_keys = min(s.keys, s.j1 * kChunkKeys);
        const int32_t* row = a.block_table + (size_t)s.seq * a.max_blocks;
        // Keys read once are the first to leave L2: they push out neither the decode pass's lines nor
        // those that other units of a group come back to (64k shared keys: 80 -> 70 us; without the
        // distinction, 256 sequences sharing 8192 keys, four units: 106 -> 114 us).
        const uint64_t policy = s.once ? l2_policy_evict_first() : l2_policy_evict_normal();
        // Block id of run `run` of the part (-1 behind its keys).
        auto entry = [&](int run) {
          const int pos = s.j0 * kChunkKeys + run * KB;
          return pos < n_keys ? __ldg(row + pos / a.bs) : -1;
        };
        // Its pool row (-1: none, or a bad block id, which is reported).
        auto pool_row = [&](int run, int blk) {
          const int pos = s.j0 * kChunkKeys + run * KB;
          if (pos >= n_keys) return -1;
          if (blk < 0 || blk >= a.P) {
            report(a.err, kErrOutOfRange);
            return -1;
          }
          return blk * a.bs + pos % a.bs;
        };
        int blk_next = entry(lane);
        // The part's query rows, behind its first K tile: their addresses are a load away, K's are here.
        // A tile's tokens are in ascending order.  Where they follow one another, as a batch of decodes
        // does, one box per half of D takes the tile (and rows behind its last token, which nobody
        // uses): token by token 2 x 32 tokens took 3.8 us, and K and V wait behind them, now 0.8.  For
        // fewer than 8 tokens a box of a whole tile is not worth it.
        int q_tok[2], q_last[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const PreToken* tok = list + s.tok0 + t * pre_tile_tokens(a.G);
          q_tok[t] = lane < s.ntok[t] ? tok[lane].token : 0;
          q_last[t] = s.ntok[t] >= 8 ? tok[s.ntok[t] - 1].token : 0;
        }
        auto load_q = [&]() {
          wait(bar(SM::bQEmpty), (k & 1) ^ 1);
          if (!ok) return;
          bool run[2];
          int rows = 0;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int first = __shfl_sync(0xffffffffu, q_tok[t], 0);
            run[t] = s.ntok[t] >= 8 && q_last[t] - first == s.ntok[t] - 1;
            rows += (run[t] ? pre_tile_tokens(a.G) : s.ntok[t]) * a.G;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(SM::bQFull), (uint32_t)(rows * SM::kHalves * 128));
          __syncwarp();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (run[t]) {
              if (lane < SM::kHalves)
                tma_load_3d(sbase + t * SM::kTile + lane * SM::kHalf, qmap_run, bar(SM::bQFull), lane * 64,
                            s.kvh * a.G, q_last[t] - (s.ntok[t] - 1));
              continue;
            }
            for (int i = lane; i < s.ntok[t]; i += 32) {
              const int tok =
                  i < 32 ? q_tok[t] : list[s.tok0 + t * pre_tile_tokens(a.G) + i].token;
#pragma unroll
              for (int half = 0; half < SM::kHalves; ++half)
                tma_load_3d(sbase + t * SM::kTile + half * SM::kHalf + i * a.G * 128, qmap,
                            bar(SM::bQFull), half * 64, s.kvh * a.G, tok);
            }
          }
        };
        // K or V tile into the next slot: the runs whose pool rows the lanes of `lanes` hold
        auto load = [&](int token, uint32_t lanes, const CUtensorMap* map) {
          const uint32_t slot = g % NS, full = bar(SM::bFull + slot);
          wait(bar(SM::bEmpty + slot), ((g / NS) & 1) ^ 1);
          if (!ok) return;
          lanes &= __ballot_sync(0xffffffffu, token >= 0);
          if (lane == 0)
            mbar_arrive_expect_tx(full, __popc(lanes) * (uint32_t)(SM::kHalves * KB * 128));
          __syncwarp();
          if ((lanes >> lane) & 1) {
            const uint32_t dst = sbase + SM::kRing + slot * SM::kTile + (lane & (nsb - 1)) * KB * 128;
#pragma unroll
            for (int half = 0; half < SM::kHalves; ++half)
              tma_load_3d_hint(dst + half * SM::kHalf, map, full, half * 64, s.kvh, token, policy);
          }
          ++g;
        };
        if (batches == 1) {
          const uint32_t tile_lanes = nsb == 32 ? 0xffffffffu : (1u << nsb) - 1u;
          int t_cur = -1, t_prev = -1;  // this batch's pool rows, and the batch's before it
          for (int i = 0; i <= n && ok; ++i) {
            const int in_batch = i & (per_batch - 1);
            if (in_batch == 0) {
              t_prev = t_cur;
              t_cur = pool_row(i * nsb + lane, blk_next);
              blk_next = entry((i + per_batch) * nsb + lane);
            }
            if (i < n) {
              load(t_cur, tile_lanes << (in_batch * nsb), kmap);
              if (i == 0 && ok) load_q();
              if (s.two && ok) load(t_cur, tile_lanes << (in_batch * nsb), vmap);
            }
            if (!s.two && i > 0 && ok) {
              if (in_batch == 0)
                load(t_prev, tile_lanes << ((per_batch - 1) * nsb), vmap);
              else
                load(t_cur, tile_lanes << ((in_batch - 1) * nsb), vmap);
            }
          }
        } else {
          // Runs of one or two keys (block sizes that share no larger power of two with a tile):
          // several batches per tile, looked up as they are needed.
          auto load_runs = [&](int j, const CUtensorMap* map) {
            const uint32_t slot = g % NS, full = bar(SM::bFull + slot);
            wait(bar(SM::bEmpty + slot), ((g / NS) & 1) ^ 1);
            if (!ok) return;
            int token[4];
            uint32_t runs = 0;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              token[p] = -1;
              if (p >= batches) continue;
              const int run = j * nsb + p * 32 + lane;
              token[p] = pool_row(run, entry(run));
              runs += __popc(__ballot_sync(0xffffffffu, token[p] >= 0));
            }
            if (lane == 0) mbar_arrive_expect_tx(full, runs * (uint32_t)(SM::kHalves * KB * 128));
            __syncwarp();
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              if (token[p] < 0) continue;
#pragma unroll
              for (int half = 0; half < SM::kHalves; ++half)
                tma_load_3d_hint(sbase + SM::kRing + slot * SM::kTile + half * SM::kHalf +
                                     (p * 32 + lane) * KB * 128,
                                 map, full, half * 64, s.kvh, token[p], policy);
            }
            ++g;
          };
          for (int i = 0; i <= n && ok; ++i) {
            if (i < n) load_runs(i, kmap);
            if (i == 0 && ok) load_q();
            if (s.two && i < n && ok) load_runs(i, vmap);
            if (!s.two && i > 0 && ok) load_runs(i - 1, vmap);
          }
        }
      }
    } else if (warp == 1) {
      // =================================================================== tcgen05 issuer
      constexpr uint32_t idesc_s = idesc_bf16(kPrefillTileM, kChunkKeys, 0);
      constexpr uint32_t idesc_o = idesc_bf16(kPrefillTileM, D, 1);
      const uint64_t q_desc0 = smem_desc_sw128(sbase, 16, 1024);
      const uint64_t k_desc0 = smem_desc_sw128(sbase + SM::kRing, 16, 1024);
      const uint64_t v_desc0 = smem_desc_sw128(sbase + SM::kRing, SM::kHalf, 1024);
      bool ok = true;
      auto wait = [&](uint32_t b, uint32_t parity) {
        if (ok && !mbar_wait(b, parity)) {
          report(a.err, kErrTimeout);
          ok = false;
        }
      };
      auto wait_slot = [&](uint32_t at) { wait(bar(SM::bFull + at % NS), (at / NS) & 1); };
      auto commit = [&](uint32_t b) {
        if (elect_one()) tc_commit(b);
        __syncwarp();
      };
      // S_t = Q K^T of ring position `at` with Q tile `qt`, and its commit
      auto mma_s = [&](const int t, const int qt, uint32_t at) {
        const uint64_t qd = q_desc0 + ((uint32_t)(qt * SM::kTile) >> 4);
        const uint64_t kd = k_desc0 + ((uint32_t)((at % NS) * SM::kTile) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = ((kk >> 2) * SM::kHalf + (kk & 3) * 32) >> 4;
            tc_mma_ss(tmem + t * 128, qd + o, kd + o, idesc_s, kk > 0 ? 1u : 0u);
          }
          tc_commit(bar(SM::bSFull + t));
        }
        __syncwarp();
      };
      // O_t += P_t V of ring position `at` (first: O_t = P_t V)
      auto mma_pv = [&](const int t, uint32_t at, bool first) {
        const uint64_t vd = v_desc0 + ((uint32_t)((at % NS) * SM::kTile) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kChunkKeys / 16; ++kk)
            tc_mma_ts(tmem + 256 + t * D, tmem + t * 128 + kk * 8, vd + ((uint32_t)(kk * 2048) >> 4),
                      idesc_o, (!first || kk > 0) ? 1u : 0u);
        }
        __syncwarp();
      };
      uint32_t g = 0, r0 = 0, r1 = 0;  // ring position, S/P rounds of group 0 and group 1 so far
      for (uint32_t k = 0; ok && walk.next(s); ++k) {
        const int n = s.j1 - s.j0;
        wait(bar(SM::bQFull), k & 1);
        wait_slot(g);
        if (!ok) break;
        mma_s(0, 0, g);
        if (s.two) {
          mma_s(1, 1, g);
          commit(bar(SM::bEmpty + g % NS));
          if (n == 1) commit(bar(SM::bQEmpty));
          for (int i = 0; i < n && ok; ++i) {
            const uint32_t v = g + 2 * i + 1, kn = v + 1;  // V tile i, K tile i + 1
            wait_slot(v);
            wait(bar(SM::bPFull + 0), r0++ & 1);
            if (i == 0 && k > 0) wait(bar(SM::bOFree), (k - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            mma_pv(0, v, i == 0);
            if (i + 1 < n) {
              wait_slot(kn);
              if (!ok) break;
              mma_s(0, 0, kn);
            }
            wait(bar(SM::bPFull + 1), r1++ & 1);
            if (!ok) break;
            tc_fence_after();
            mma_pv(1, v, i == 0);
            commit(bar(SM::bEmpty + v % NS));
            if (i + 1 < n) {
              mma_s(1, 1, kn);
              commit(bar(SM::bEmpty + kn % NS));
              if (i + 2 == n) commit(bar(SM::bQEmpty));
            }
          }
        } else {
          commit(bar(SM::bEmpty + g % NS));
          if (n > 1) {
            wait_slot(g + 1);
            if (!ok) break;
            mma_s(1, 0, g + 1);
            commit(bar(SM::bEmpty + (g + 1) % NS));
          }
          if (n <= 2) commit(bar(SM::bQEmpty));
          // step i on group i & 1, two steps per turn so that the groups are constants
          auto step = [&](const int t, int i, uint32_t& r) {
            const uint32_t v = g + (i + 1 < n ? 2 * i + 2 : 2 * n - 1);
            wait_slot(v);
            wait(bar(SM::bPFull + t), r++ & 1);
            if (i == 0 && k > 0) wait(bar(SM::bOFree), (k - 1) & 1);
            if (!ok) return;
            tc_fence_after();
            mma_pv(t, v, i < 2);
            commit(bar(SM::bEmpty + v % NS));
            if (i + 2 < n) {
              const uint32_t kn = g + 2 * i + 3;
              wait_slot(kn);
              if (!ok) return;
              mma_s(t, 0, kn);
              commit(bar(SM::bEmpty + kn % NS));
              if (i + 3 == n) commit(bar(SM::bQEmpty));
            }
          };
          for (int i = 0; i < n && ok; i += 2) {
            step(0, i, r0);
            if (i + 1 < n && ok) step(1, i + 1, r1);
          }
        }
        if (!ok) break;
        commit(bar(SM::bOFinal));
        g += 2 * n;
      }
    }
  } else {
    regs_inc<kRegsSoftmax>();
    // ===================================================================== softmax groups
    const int t = (warp - 4) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;  // row within the tile, and TMEM lane
    const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t s_col = t * 128, o_col = 256 + t * D;
    const uint32_t xch = sbase + SM::kXch + r * 8;
    const float sl2 = a.scale_log2;
    uint32_t g = 0, rx = 0, kx = 0;  // ring position, S/P rounds, parts with one tile so far
    bool ok = true;
    auto wait = [&](uint32_t b, uint32_t parity) {
      if (ok && !mbar_wait(b, parity)) {
        report(a.err, kErrTimeout);
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
    };
    for (uint32_t k = 0; ok && walk.next(s); ++k) {
      const int n = s.j1 - s.j0;
      const int n_keys = min(s.keys, s.j1 * kChunkKeys);
      const int rows = (s.two && t ? s.ntok[1] : s.ntok[0]) * a.G;
      const bool active = quad * 32 < rows;
      const int first = s.two ? 0 : t, stride = s.two ? 1 : 2;
      // keys that this row sees (its token's, where the group has a causal edge)
      const int i_tok = r / a.G;
      const int sees = s.ctx < 0 ? s.keys
                                 : min(s.keys, s.ctx + s.at + (s.two && t ? pre_tile_tokens(a.G) : 0) +
                                                   i_tok + 1);
      float m_run = -INFINITY, l_run = 0.f;
      for (int i = first; i < n; i += stride) {
        wait(bar(SM::bSFull + t), rx++ & 1);
        if (!ok) break;
        const int left = n_keys - (s.j0 + i) * kChunkKeys;  // keys of the prefix in this tile
        if (left < kChunkKeys) {
          // Keys behind the prefix: their V rows may be anything and P is 0 there, but 0 * NaN is
          // NaN, so zero them before the product reads them (with two tiles both groups do).
          const uint32_t at = g + 2 * n - 1;  // the part's last V tile
          wait(bar(SM::bFull + at % NS), (at / NS) & 1);
          if (!ok) break;
          const uint32_t v = sbase + SM::kRing + (at % NS) * SM::kTile;
          const int chunks = (kChunkKeys - left) * SM::kHalves * 8;
          for (int x = r; x < chunks; x += 128) {
            const int rr = left + x / (SM::kHalves * 8), rem = x % (SM::kHalves * 8);
            asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(
                             sw128(v + (rem >> 3) * SM::kHalf, rr, rem & 7)), "r"(0u) : "memory");
          }
          fence_proxy_async_smem();
        }
        if (active) {
          tc_fence_after();
          uint32_t sr[128];
#pragma unroll
          for (int x = 0; x < 4; ++x) tmem_ld32(t_lane + s_col + x * 32, sr + x * 32);
          tc_wait_ld();
          // the keys' end (or causal edge) and their start inside this tile
          const int key0 = (s.j0 + i) * kChunkKeys;
          const int hi = sees - key0, lo = s.first - key0;
          if (__any_sync(0xffffffffu, hi < kChunkKeys || lo > 0)) {
#pragma unroll
            for (int x = 0; x < 128; ++x)
              if (x >= hi || x < lo) sr[x] = __float_as_uint(-INFINITY);
          }
          float mx8[8];
#pragma unroll
          for (int x = 0; x < 8; ++x)
            mx8[x] = fmax3(__uint_as_float(sr[x]), __uint_as_float(sr[8 + x]), __uint_as_float(sr[16 + x]));
#pragma unroll
          for (int col = 24; col < 120; col += 16)
#pragma unroll
            for (int x = 0; x < 8; ++x)
              mx8[x] = fmax3(mx8[x], __uint_as_float(sr[col + x]), __uint_as_float(sr[col + 8 + x]));
#pragma unroll
          for (int x = 0; x < 8; ++x) mx8[x] = fmaxf(mx8[x], __uint_as_float(sr[120 + x]));
          const float mt = sl2 * fmaxf(fmax3(mx8[0], mx8[1], mx8[2]),
                                       fmax3(fmax3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
          // the running maximum follows only in steps of more than 2^8 (see the chunk pass)
          float alpha = 1.f;
          bool resc = false;
          if (i == first) {
            m_run = mt;
          } else if (mt > m_run + 8.f) {
            alpha = fast_exp2(m_run - mt);
            m_run = mt;
            resc = true;
          }
          // (a row that sees no key so far: its m is -inf, 0 is subtracted, every p is 0)
          const float m_sub = m_run == -INFINITY ? 0.f : m_run;
          const uint64_t scale2 = f2_pack(sl2, sl2), neg_m2 = f2_pack(-m_sub, -m_sub);
          uint64_t sum2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int col = 0; col < 128; col += 2) {
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[col]), __uint_as_float(sr[col + 1])), scale2,
                             neg_m2), x0, x1);
            const float p0 = fast_exp2(x0), p1 = fast_exp2(x1);
            sum2[(col >> 1) & 3] = f2_add(sum2[(col >> 1) & 3], f2_pack(p0, p1));
            sr[col >> 1] = pack_bf16x2(p0, p1);
          }
          float sm8[8];
#pragma unroll
          for (int x = 0; x < 4; ++x) f2_unpack(sum2[x], sm8[2 * x], sm8[2 * x + 1]);
          l_run = l_run * alpha + (((sm8[0] + sm8[1]) + (sm8[2] + sm8[3])) +
                                   ((sm8[4] + sm8[5]) + (sm8[6] + sm8[7])));
          tmem_st32(t_lane + s_col, sr);
          tmem_st32(t_lane + s_col + 32, sr + 32);
          if (__any_sync(0xffffffffu, resc)) {
            // O_t's products so far have completed: S of this tile was issued after them and its
            // commit signalled every earlier product done.
#pragma unroll
            for (int ch = 0; ch < D / 32; ++ch) {
              uint32_t ov[32];
              tmem_ld32(t_lane + o_col + ch * 32, ov);
              tc_wait_ld();
#pragma unroll
              for (int x = 0; x < 32; ++x) ov[x] = __float_as_uint(__uint_as_float(ov[x]) * alpha);
              tmem_st32(t_lane + o_col + ch * 32, ov);
            }
          }
          tc_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(SM::bPFull + t));
      }
      if (!ok) break;
      g += 2 * n;
      // ---- the part's end: partial (m, l) and O, unnormalised, to its rows.
      // Destination row of a token's head: the chain's own rows (part with its first tile), or
      // this CTA's.
      const int per_tile = pre_tile_tokens(a.G);
      const uint32_t row =  // (the workspace holds far less than 2^32 of them)
          s.cut ? (uint32_t)((c * 2 + (s.two ? t : 0)) * kPrefillTileM + r)
                : (uint32_t)(s.tok0 + (s.two ? t * per_tile : 0) + i_tok + s.second * a.LT) * (uint32_t)a.Hq +
                      s.kvh * a.G + (r - i_tok * a.G);
      float2* ml = reinterpret_cast<float2*>(a.ws + (s.cut ? PL.cut_ml : PL.base_ml)) + row;
      float* o = reinterpret_cast<float*>(a.ws + (s.cut ? PL.cut_o : PL.base_o));
      float w0 = 1.f, w1 = 0.f;  // weights of O_0 and O_1 (one tile of rows)
      if (!s.two) {
        // both groups' (m, l): group 1 hands its own over, group 0 hands the weights back
        if (t == 1) {
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(xch), "f"(m_run), "f"(l_run) : "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(SM::bStat));
        }
        wait(bar(t == 1 ? SM::bWeight : SM::bStat), kx & 1);
        if (!ok) break;
        float x0, x1;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x0), "=f"(x1) : "r"(xch) : "memory");
        if (t == 0) {
          const float M = fmaxf(m_run, x0), m_sub = M == -INFINITY ? 0.f : M;
          w0 = fast_exp2(m_run - m_sub);
          w1 = fast_exp2(x0 - m_sub);
          l_run = l_run * w0 + x1 * w1;
          m_run = M;
          __syncwarp();
          asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(xch), "f"(w0), "f"(w1) : "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(SM::bWeight));
        } else {
          w0 = x0;
          w1 = x1;
        }
        ++kx;
      }
      wait(bar(SM::bOFinal), k & 1);
      if (!ok) break;
      tc_fence_after();
      if (active) {
        // one tile: group t writes its half of the columns of both accumulators' sum
        const int ch0 = s.two ? 0 : t * (D / 64), ch1 = s.two ? D / 32 : ch0 + D / 64;
        const uint32_t o0 = s.two ? o_col : 256u;
        const bool both = !s.two && n > 1;
        // A lane holds 32 columns of its row.  With many rows 8 lanes turn their 8 x 8 pieces of 4
        // columns, so that they write a row's 128 bytes at once: each lane 16 bytes of a row of its
        // own, 2 x 128 rows took 4.8 us, so 3; with few the turning costs more than it saves.
        const bool turn = s.two || rows > 64;
        for (int ch = ch0; ch < ch1; ++ch) {
          uint32_t ov[32];
          tmem_ld32(t_lane + o0 + ch * 32, ov);
          if (both) {
            uint32_t ow[32];
            tmem_ld32(t_lane + 256 + D + ch * 32, ow);
            tc_wait_ld();
#pragma unroll
            for (int x = 0; x < 32; ++x)
              ov[x] = __float_as_uint(__uint_as_float(ov[x]) * w0 + __uint_as_float(ow[x]) * w1);
          } else {
            tc_wait_ld();
          }
          if (turn) {
#pragma unroll
            for (int sh = 1; sh < 8; sh *= 2)
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                if (x & (4 * sh)) continue;
                const bool up = lane & sh;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? ov[x] : ov[x + 4 * sh], sh);
                if (up) ov[x] = got;
                else ov[x + 4 * sh] = got;
              }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const uint32_t to = __shfl_sync(0xffffffffu, row, (lane & 24) + x);
              if (quad * 32 + (lane & 24) + x < rows)
                *reinterpret_cast<uint4*>(o + (size_t)to * D + ch * 32 + (lane & 7) * 4) =
                    make_uint4(ov[4 * x], ov[4 * x + 1], ov[4 * x + 2], ov[4 * x + 3]);
            }
          } else if (r < rows) {
            uint4* dst = reinterpret_cast<uint4*>(o + (size_t)row * D + ch * 32);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              dst[x] = make_uint4(ov[4 * x], ov[4 * x + 1], ov[4 * x + 2], ov[4 * x + 3]);
          }
        }
        if (r < rows && (s.two || t == 0)) *ml = make_float2(m_run, l_run);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(SM::bOFree));
    }
    if (lane == 0) atomicMax(&hdr->t_pf_end, global_ns());
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace cb

// Decode pass over the quantised cache: every sequence with one query token attends to its keys.
//
// The split of the work is the decode pass's (cb_decode.cuh): the key tiles of all decode sequences laid
// end to end, equal contiguous ranges for the CTAs, partial results (m, l, o) merged by the warp that
// finishes a sequence last.  Bound by HBM like that pass, at half its bytes, so the same bytes in flight
// hold twice the keys and a warp has half the time per key; the differences follow from that:
//
//   * A tile is 32 keys for each of the CTA's up to 8 KV heads (64 KB of codes at head_dim 128).  With
//     fewer KV heads several warps share a head, each with 32 keys of a longer tile, and merge at the
//     end of a sequence through shared memory, so a CTA has the same bytes in flight and the same number
//     of warps.
//   * The codes go from shared memory to the tensor cores through one conversion to fp16, which holds
//     every e4m3 value.  No ldmatrix: which element of the head dim (or which key) is which index of a
//     product's sum is free as long as both operands agree, so a lane reads 16 consecutive codes of
//     a key's row, K and V alike, and V's pairs of keys are made by byte permutes.
//   * The scales stay out of the products.  With k = 2^ek * kc, v = 2^ev * vc and the query row scaled
//     to fp16 range by 2^eq,
//       x_j = scale log2(e) 2^(eq + ek_j) (qc . kc_j),   y_j = x_j + ev_j,   p_j = 2^(y_j - m),
//       o = sum_j p_j vc_j,   l = sum_j p_j 2^-ev_j,   out = o / l,
//     with m the running maximum of y less 7, kept at the end of a sequence too: so p is at most 2^15 (the
//     maximum is followed lazily, 2^8) and its rounding to fp16 -- 2^-11 relative, and 2^-32 of the largest
//     where p is less than 2^-21 of that -- is small against the largest contribution to o, whatever the
//     sizes of the values.  (With the largest p at 1, keys with less than 2^-25 of it were lost from o but
//     not from l: 2^19 of them beside one that takes all are 1 / 65 of the result.)  l is summed in fp32,
//     where 2^-ev (ev in [-32, 31]) is safe.
#pragma once

#include "cb_decode.cuh"
#include "cb_place.cuh"
#include "cb_quant.cuh"
#include "cb_quant_shape.h"
#include "cb_score.cuh"

namespace cb {

__device__ __forceinline__ void mma_f16_16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}

template <int D, int QS>
struct QDecodeSmem {
  static constexpr int kKVBytes = 8 / QS * kQTileKeys * D;  // K (or V) of a tile, at most
  static constexpr int kScaleBytes = 8 / QS * kQTileKeys * 2;
  static constexpr int kStageBytes = 2 * kKVBytes;
  static constexpr int kStages = 3 * QS * (128 / D);        // 192 KB of codes
  static constexpr int kScales = kStages * kStageBytes;
  // merge of a head's warps: 4 writers at most, per lane D / 4 values of o, two m and two l
  static constexpr int kMergeWarp = 32 * (D / 4 + 4) * 4;
  static constexpr int kMerge = kScales + kStages * kScaleBytes;
  static constexpr int kBar = kMerge + 4 * kMergeWarp;      // full, empty per stage; 4 merge barriers
  static constexpr int kInfo = (kBar + (2 * kStages + 4) * 8 + 15) / 16 * 16;  // QuantStage per stage
  static constexpr int kTokens = kInfo + kStages * 32;  // of a tile's page runs, where they are many
  static constexpr int kRange = kTokens + 256 * 4;
  static constexpr int kTotal = kRange + 16 + 1024;
  static_assert(kMerge % 16 == 0 && kBar % 8 == 0, "alignment of shared-memory regions");
};

// `bytes` (a multiple of 16) from global to shared memory (both 16-byte aligned), counted on `bar`.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Bytes between the page runs of a tile (a run: [HB heads][KB keys] rows of D bytes); TMA writes to
// multiples of 128 bytes.
template <int D>
__device__ __forceinline__ int quant_run_stride(int HB, int KB) { return (HB * KB * D + 127) & ~127; }
// TMA's swizzle of a byte offset in a 1024-byte aligned region: 16-byte pieces of 128-byte lines, or of
// 64-byte rows (D = 64).
template <int D>
__device__ __forceinline__ uint32_t quant_swizzle(uint32_t off) {
  return off ^ ((off >> 3) & (D == 128 ? 0x70u : 0x30u));
}

// A stage's record, two 16-byte pieces in shared memory: its query's token, keys, index among the decode
// sequences and first key; flags, first key of the window, the sequence's tiles [p0, p1).
struct QuantStage {
  int tok, kv, dec, key0, flags, lo, p0, p1;
};
__device__ __forceinline__ QuantStage quant_stage(uint32_t addr) {
  const uint4 a = lds128(addr), b = lds128(addr + 16);
  return {(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}
__device__ __forceinline__ void sts128(uint32_t addr, int x, int y, int z, int w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// The producer warp: walks the CTA's tiles [t0, t1) and copies each tile's page runs by TMA and its scales
// beside them: a run's in one bulk copy where the CTA has all KV heads (qa.copy 0), else in small copies
// of every lane, which count on the same barrier.  Block-table entries are loaded for up to 32 runs at a
// time (several tiles), one such batch ahead, and a sequence's record one sequence ahead.  What this warp
// does per tile is on the path from a freed stage to its next bytes: 27949 tiles of 64 KB on 152 CTAs
// took 399 us with the entries and their divisions made per tile and all scales copied by lanes.
template <int D, int QS>
__device__ __forceinline__ void quant_produce(const AttnArgs& a, const QuantArgs& qa,
                                              const CUtensorMap* kmap, const CUtensorMap* vmap,
                                              uint32_t sbase, int* tokens, int n_dec,
                                              const int4* dec_rec, int d, int hg, int HB, long long t0,
                                              long long t1, int lane) {
  using SM = QDecodeSmem<D, QS>;
  if (lane == 0) {
    tma_prefetch_desc(kmap);
    tma_prefetch_desc(vmap);
  }
  const uint32_t bar_full = sbase + SM::kBar, bar_empty = bar_full + 8 * SM::kStages;
  const int KB = qa.KB, tile_keys = 1 << qa.tile_log2, runs = tile_keys / KB;  // (at most 256)
  const int run_stride = quant_run_stride<D>(HB, KB), scale_run = 2 * HB * KB;
  const uint32_t run_bytes = (uint32_t)(2 * KB * HB * D + (qa.copy == 0 ? scale_run : 0));
  const uint64_t policy = l2_policy_evict_first();  // each K/V row is read once
  const int head0 = hg * (8 / QS);
  // this lane's first small copy of scales: its run, and where it is in the run's source
  const int row_bytes = 2 * HB, copies = qa.copy == 0 ? 0 : tile_keys * row_bytes / qa.copy;
  auto copy_at = [&](int u, int& run) -> long long {
    const int key = u * qa.copy / row_bytes;
    run = key / KB;
    return (long long)(key - run * KB) * a.Hkv * 2 + (u * qa.copy - key * row_bytes) + 2 * head0;
  };
  int copy_run;
  const long long copy_src = copies > 0 ? copy_at(lane, copy_run) : 0;
  if (copies == 0) copy_run = 0;

  int4 rec = dec_rec[d], next = dec_rec[min(d + 1, n_dec)], after = dec_rec[min(d + 2, n_dec)];
  auto first_key = [&](const int4& r) {  // of the sequence's first tile
    return window_first_key(r.z - 1, a.window) / tile_keys * tile_keys;
  };
  // Tiles per batch of entries (a tile of more than 32 runs -- small blocks, few KV heads -- takes them
  // one by one below), and this lane's place in one.
  const int per_batch = runs <= 32 ? 32 / runs : 1;
  const int my_tile = runs <= 32 ? lane / runs : 0, my_key = runs <= 32 ? lane % runs * KB : 0;
  // Has a run that begins at key pos of r keys that are seen?  (Of those before a sliding window the table's
  // entries may name no block any more.)
  auto seen = [&](const int4& r, int pos) {
    return pos < r.z && pos + KB > window_first_key(r.z - 1, a.window);
  };
  // The key with which this lane's run in the batch of tiles [t, hi) of r begins, and whether there is one
  auto run_key = [&](const int4& r, long long t) {
    return first_key(r) + (int)(t + my_tile - r.w) * tile_keys + my_key;
  };
  auto has_run = [&](const int4& r, int pos) { return runs <= 32 && my_tile < per_batch && seen(r, pos); };
  // Its entry of the block table (-1 beyond the table; looked at only when the batch's turn has come), and
  // the offset in the block
  auto fetch = [&](const int4& r, long long t, int& off) -> int {
    const int pos = run_key(r, t);
    off = 0;
    if (!has_run(r, pos)) return -1;
    const int lb = pos / a.bs;
    off = pos - lb * a.bs;
    return lb < a.max_blocks ? __ldg(a.block_table + (size_t)r.x * a.max_blocks + lb) : -1;
  };
  int off, e = fetch(rec, t0, off);
  uint32_t stage = 0, phase = 1;
  bool begins = true;  // the next tile is this CTA's first of its sequence
  for (long long t = t0; t < t1;) {
    const long long p0 = rec.w, p1 = next.w;
    const long long hi = t1 < p1 ? t1 : p1;
    const int nb = (int)(hi - t < per_batch ? hi - t : per_batch);
    int off_n = 0, e_n = -1;
    if (t + nb < t1) e_n = fetch(t + nb < p1 ? rec : next, t + nb, off_n);
    if (begins && lane == 0)  // the consumers read the query rows a few stages from now
      l2_prefetch_bulk(static_cast<const __nv_bfloat16*>(a.q) + ((size_t)rec.y * a.Hq + (size_t)head0 * a.G) * D,
                       (uint32_t)(HB * a.G * D * 2));
    // (runs of this lane's tile count only where the tile is the sequence's and the CTA's)
    const bool want = t + my_tile < hi && has_run(rec, run_key(rec, t)), good = want && e >= 0 && e < a.P;
    if (want && !good) report(a.err, kErrOutOfRange);
    const int token = good ? e * a.bs + off : -1;
    const int key_t = first_key(rec) + (int)(t - p0) * tile_keys;
    bool ok = true;
    for (int i = 0; i < nb; ++i) {
      if (lane == 0) ok = mbar_wait(bar_empty + 8 * stage, phase);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      const int key0 = key_t + i * tile_keys;
      uint32_t n_runs;
      int tok = -1;
      if (runs <= 32) {
        tok = __shfl_sync(0xffffffffu, token, i * runs + (lane < runs ? lane : 0));
        if (lane >= runs) tok = -1;
        n_runs = __popc(__ballot_sync(0xffffffffu, tok >= 0));
      } else {
        n_runs = 0;
        __syncwarp();  // (the last tile's tokens are read)
        for (int run = lane; run < runs; run += 32) {  // (runs is a multiple of 32)
          const int pos = key0 + run * KB;
          int id = -1;
          if (seen(rec, pos)) {
            const int lb = pos / a.bs;
            const int block = lb < a.max_blocks ? __ldg(a.block_table + (size_t)rec.x * a.max_blocks + lb) : -1;
            if (block >= 0 && block < a.P)
              id = block * a.bs + (pos - lb * a.bs);
            else
              report(a.err, kErrOutOfRange);
          }
          tokens[run] = id;
          n_runs += __popc(__ballot_sync(0xffffffffu, id >= 0));
        }
      }
      const uint32_t full = bar_full + 8 * stage;
      if (lane == 0) {
        const uint32_t info = sbase + SM::kInfo + stage * (uint32_t)sizeof(QuantStage);
        const bool first = begins && i == 0, last = t + i == hi - 1;
        sts128(info, rec.y, rec.z, d, key0);
        sts128(info + 16,
               (first ? kInfoFirst : 0u) | (last ? kInfoLast : 0u) |
                   (p0 >= t0 && p1 <= t1 ? kInfoComplete : 0u),
               window_first_key(rec.z - 1, a.window), (int)p0, (int)p1);
        mbar_arrive_expect_tx(full, n_runs * run_bytes);
      }
      __syncwarp();
      const uint32_t kst = sbase + stage * SM::kStageBytes, vst = kst + SM::kKVBytes;
      const uint32_t sst = sbase + SM::kScales + stage * SM::kScaleBytes;
      auto copy_run_of = [&](int run, int token) {
        tma_load_3d_hint(kst + run * run_stride, kmap, full, 0, token, head0, policy);
        tma_load_3d_hint(vst + run * run_stride, vmap, full, 0, token, head0, policy);
        if (qa.copy == 0)
          bulk_load(sst + run * scale_run, qa.scales + (size_t)token * row_bytes, scale_run, full);
      };
      if (runs <= 32) {
        if (tok >= 0) copy_run_of(lane, tok);
      } else {
        for (int run = lane; run < runs; run += 32)
          if (tokens[run] >= 0) copy_run_of(run, tokens[run]);
      }
      if (qa.copy > 0) {
        int run = copy_run;
        long long from = copy_src;
        for (int u0 = 0; u0 < copies; u0 += 32) {
          const int u = u0 + lane;
          if (u0 > 0) from = copy_at(u < copies ? u : 0, run);
          const int tk = runs <= 32 ? __shfl_sync(0xffffffffu, tok, run & 31) : u < copies ? tokens[run] : -1;
          if (u >= copies || tk < 0) continue;
          const uint8_t* src = qa.scales + (size_t)tk * a.Hkv * 2 + from;
          const uint32_t dst = sst + u * qa.copy;
          if (qa.copy == 16) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
          } else if (qa.copy == 8) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
          } else if (qa.copy == 4) {
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
          } else {
            const unsigned short v = __ldg(reinterpret_cast<const unsigned short*>(src));
            asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst), "h"(v) : "memory");
          }
        }
        // one arrival per lane, once its copies are there
        if (qa.copy == 2)
          mbar_arrive(full);
        else
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(full) : "memory");
        __syncwarp();
      }
      if (++stage == SM::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) {
      if (lane == 0) report(a.err, kErrTimeout);
      break;
    }
    t += nb;
    begins = t >= p1;
    if (begins) {
      ++d;
      rec = next;
      next = after;
      after = dec_rec[min(d + 2, n_dec)];
    }
    e = e_n;
    off = off_n;
  }
}

constexpr float kFp16Room = 7.f;  // log2 of the largest p where the running maximum is up to date

// Consumer warp: KV head h of the CTA's HB, query heads qoff .. qoff + 7 of its G, keys
// 32 slice .. 32 slice + 31 of every tile.  As in the decode pass the keys are the M side of the score
// product and the head dim that of the output product, 8 query heads the N side.  Lane (g, tq):
//   scores: keys g and g + 8 of a 16-key group (rows), query heads 2 tq and 2 tq + 1 (columns); of each
//           key's row it feeds codes tq D/4 .. (tq + 1) D/4 - 1;
//   output: codes g D/8 .. (g + 1) D/8 - 1 of the group's keys 2tq, 2tq + 1, 2tq + 8, 2tq + 9, so that
//           it holds D/8 consecutive values of query heads 2 tq and 2 tq + 1.
template <int D, int QS, bool kMod>
__device__ __forceinline__ void quant_consume(const AttnArgs& a, const QuantArgs& qa,
                                              const ScoreArgs& sc, uint32_t sbase,
                                              int c, int hg, int HB, int slices, int warp,
                                              long long n_my, long long ntiles, int N,
                                              const WsLayout& L, int lane) {
  using SM = QDecodeSmem<D, QS>;
  constexpr int KS = D / 16, MT = D / 16;   // steps over the head dim
  constexpr int W = D / 32;                 // 32-bit words of a lane's part of a V row
  const uint32_t bar_full = sbase + SM::kBar, bar_empty = bar_full + 8 * SM::kStages;
  const int sub = warp % QS, h = warp / QS % HB, slice = warp / QS / HB;
  const int qoff = sub * 8, kvh = hg * (8 / QS) + h;
  const int g = lane >> 2, tq = lane & 3;
  const float sl2 = a.scale_log2;
  const __nv_bfloat16* qg = static_cast<const __nv_bfloat16*>(a.q);
  __nv_bfloat16* outg = static_cast<__nv_bfloat16*>(a.out);
  float2* part_ml = reinterpret_cast<float2*>(a.ws + L.part_ml);
  float* part_o = reinterpret_cast<float*>(a.ws + L.part_o);
  int32_t* merge_cnt = reinterpret_cast<int32_t*>(a.ws + L.merge_cnt);

  // byte offsets of this lane's pieces in a stage
  const int KB = qa.KB, run_stride = quant_run_stride<D>(HB, KB);
  auto row_of = [&](int k) { return (uint32_t)(k / KB * run_stride + (h * KB + k % KB) * D); };
  uint32_t k_at[4], v_at[8], s_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = slice * kQTileKeys + 8 * i + g;
    k_at[i] = quant_swizzle<D>(row_of(key) + tq * (D / 4));
    s_at[i] = (uint32_t)(2 * (key * HB + h));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int key = slice * kQTileKeys + 16 * (i >> 2) + 2 * tq + 8 * ((i >> 1) & 1) + (i & 1);
    v_at[i] = quant_swizzle<D>(row_of(key) + g * (D / 8));
  }

  uint32_t qb[KS][2];
  float cq[2];          // per column: 2^eq, times scale log2(e) unless the scores are changed
  float slope[2];
  float o[MT][4];
  float m[2], l[2];
  uint32_t sync_phase = 0;

  uint32_t stage = SM::kStages - 1, phase = 1;
  for (long long it = 0; it < n_my; ++it) {
    if (++stage == SM::kStages) {
      stage = 0;
      phase ^= 1;
    }
    if (!mbar_wait(bar_full + 8 * stage, phase)) {
      if (lane == 0) report(a.err, kErrTimeout);
      break;
    }
    const QuantStage si = quant_stage(sbase + SM::kInfo + stage * (uint32_t)sizeof(QuantStage));
    if (si.flags & kInfoFirst) {
      // the query row of column g, scaled so that its largest value is in [1, 2) (exact in fp16 but
      // for values 2^-14 smaller, which are off by 2^-25 at most)
      const int hl = qoff + g;
      uint4 raw[D / 32];
      float top = 0.f;
      const uint4* src = reinterpret_cast<const uint4*>(
          qg + ((size_t)si.tok * a.Hq + kvh * a.G + (hl < a.G ? hl : 0)) * D + tq * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        raw[i] = hl < a.G ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        float x[8];
        unpack8(raw[i], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int eq = min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126);
      const float inv = __int_as_float((127 - eq) << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float x[8];
        unpack8(raw[i], x);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          qb[2 * i + j][0] = pack_f16x2(x[4 * j] * inv, x[4 * j + 1] * inv);
          qb[2 * i + j][1] = pack_f16x2(x[4 * j + 2] * inv, x[4 * j + 3] * inv);
        }
      }
      const float up = __int_as_float((127 + eq) << 23);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        cq[j] = __shfl_sync(0xffffffffu, up, 4 * (2 * tq + j)) * (kMod ? 1.f : sl2);
        if constexpr (kMod) {
          const int hc = qoff + 2 * tq + j;
          slope[j] = hc < a.G ? slope_of(sc, kvh * a.G + hc) : 0.f;
        }
        m[j] = -INFINITY;
        l[j] = 0.f;
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    }
    const uint32_t kst = sbase + stage * SM::kStageBytes, vst = kst + SM::kKVBytes;
    const uint32_t sst = sbase + SM::kScales + stage * SM::kScaleBytes;
    const int key0 = si.key0 + slice * kQTileKeys;
    const bool edge = key0 + kQTileKeys > si.kv || key0 < si.lo;

    // ---- everything of the stage into registers, then the stage is released
    uint32_t kr[4][KS];
    uint32_t vr[8][W];
    uint32_t ex[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unsigned short v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(sst + s_at[i]));
      ex[i] = v;
      const uint4 x = lds128(kst + k_at[i]);
      kr[i][0] = x.x; kr[i][1] = x.y; kr[i][2] = x.z; kr[i][3] = x.w;
      if constexpr (D == 128) {
        const uint4 y = lds128(kst + (k_at[i] ^ 16u));
        kr[i][4] = y.x; kr[i][5] = y.y; kr[i][6] = y.z; kr[i][7] = y.w;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (D == 128) {
        const uint4 x = lds128(vst + v_at[i]);
        vr[i][0] = x.x; vr[i][1] = x.y; vr[i][2] = x.z; vr[i][3] = x.w;
      } else {
        const uint2 x = lds64(vst + v_at[i]);
        vr[i][0] = x.x; vr[i][1] = x.y;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_empty + 8 * stage);

    // ---- scores
    float s[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float s1[4] = {0.f, 0.f, 0.f, 0.f};  // (two chains of products)
      s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t af[4];
        e4m3x4_to_f16(kr[2 * j][ks], af[0], af[2]);
        e4m3x4_to_f16(kr[2 * j + 1][ks], af[1], af[3]);
        mma_f16_16816(ks & 1 ? s1 : s[j], af, qb[ks][0], qb[ks][1]);
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) s[j][x] += s1[x];
    }
    // Rows that are NaN: a key's scores, and all of a value's codes (its p is that of a finite row).
    if (__any_sync(0xffffffffu, max(max(ex[0] & 255u, ex[0] >> 8), max(ex[1] & 255u, ex[1] >> 8)) == kQuantNan ||
                                    max(max(ex[2] & 255u, ex[2] >> 8), max(ex[3] & 255u, ex[3] >> 8)) == kQuantNan)) {
      uint32_t vn = 0;  // bit i: the value of key 8 i + g is NaN
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((ex[i] & 255u) == kQuantNan) s[i >> 1][2 * (i & 1)] = s[i >> 1][2 * (i & 1) + 1] = __int_as_float(0x7fffffff);
        if ((ex[i] >> 8) == kQuantNan) {
          vn |= 1u << i;
          ex[i] = (ex[i] & 255u) | (uint32_t)kQuantBias << 8;
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = 16 * (i >> 2) + 2 * tq + 8 * ((i >> 1) & 1) + (i & 1);
        const uint32_t bits = __shfl_sync(0xffffffffu, vn, 4 * (key & 7));
        if (bits >> (key >> 3) & 1) {
#pragma unroll
          for (int w = 0; w < W; ++w) vr[i][w] = 0x7f7f7f7fu;
        }
      }
    }
    // y = x + ev; the weights of l
    float wl[4], ev[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float fk = __uint_as_float((ex[i] & 255u) << 23);
      ev[i] = (float)(int)(ex[i] >> 8) - 127.f;
      wl[i] = __uint_as_float((254u - (ex[i] >> 8)) << 23);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float& x = s[i >> 1][2 * (i & 1) + j];
        x = kMod ? x * fk * cq[j] : fmaf(x * fk, cq[j], ev[i]);
      }
    }
    if constexpr (kMod) {
      change_scores<8>(&s[0][0], sl2, slope, key0 + g - (si.kv - 1), sc);
#pragma unroll
      for (int x = 0; x < 8; ++x) s[x >> 2][x & 3] += ev[x >> 1];
    }
    if (edge) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key0 + 8 * i + g;
        if (key >= si.kv || key < si.lo) {
          s[i >> 1][2 * (i & 1)] = s[i >> 1][2 * (i & 1) + 1] = -INFINITY;
          wl[i] = 0.f;
        }
      }
      // (what stands in other slots may be a NaN code, and 0 * NaN is NaN)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = key0 + 16 * (i >> 2) + 2 * tq + 8 * ((i >> 1) & 1) + (i & 1);
        if (key >= si.kv || key < si.lo) {
#pragma unroll
          for (int w = 0; w < W; ++w) vr[i][w] = 0u;
        }
      }
    }
    // ---- the running maximum follows where a score exceeds it by more than 2^8
    const float ta = fmaxf(fmaxf(s[0][0], s[0][2]), fmaxf(s[1][0], s[1][2]));
    const float tb = fmaxf(fmaxf(s[0][1], s[0][3]), fmaxf(s[1][1], s[1][3]));
    if (__any_sync(0xffffffffu, ta > m[0] + 8.f || tb > m[1] + 8.f)) {
      float ma = ta, mb = tb;
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, x));
        mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, x));
      }
      float al = 1.f, be = 1.f;
      if (ma > m[0] + 8.f) {
        al = fast_exp2(m[0] - ma);
        m[0] = ma;
      }
      if (mb > m[1] + 8.f) {
        be = fast_exp2(m[1] - mb);
        m[1] = mb;
      }
      l[0] *= al;
      l[1] *= be;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        o[mt][0] *= al;
        o[mt][1] *= be;
        o[mt][2] *= al;
        o[mt][3] *= be;
      }
    }
    // (a warp whose keys so far are all masked has m = -inf: 0 is subtracted instead)
    const float sa = m[0] == -INFINITY ? 0.f : m[0] - kFp16Room, sb = m[1] == -INFINITY ? 0.f : m[1] - kFp16Room;
    uint32_t pb[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float p0 = fast_exp2(s[j][0] - sa), p1 = fast_exp2(s[j][1] - sb);
      const float p2 = fast_exp2(s[j][2] - sa), p3 = fast_exp2(s[j][3] - sb);
      l[0] = fmaf(p0, wl[2 * j], fmaf(p2, wl[2 * j + 1], l[0]));
      l[1] = fmaf(p1, wl[2 * j], fmaf(p3, wl[2 * j + 1], l[1]));
      pb[j][0] = movm_trans(pack_f16x2(p0, p1));  // keys 0-7 of the group: B[k = 2tq, 2tq+1][n = g]
      pb[j][1] = movm_trans(pack_f16x2(p2, p3));  // keys 8-15
    }
    // ---- O^T += V^T P^T: row g of m-tile mt is the lane's value 2 mt, row g + 8 its value 2 mt + 1
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int w = mt >> 1;
        const uint32_t sel = mt & 1 ? 0x7362u : 0x5140u;
        uint32_t vf[4];
        e4m3x4_to_f16(__byte_perm(vr[4 * j][w], vr[4 * j + 1][w], sel), vf[0], vf[1]);
        e4m3x4_to_f16(__byte_perm(vr[4 * j + 2][w], vr[4 * j + 3][w], sel), vf[2], vf[3]);
        mma_f16_16816(o[mt], vf, pb[j][0], pb[j][1]);
      }

    if (!(si.flags & kInfoLast)) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) m[j] -= kFp16Room;  // what was subtracted
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[j] += __shfl_xor_sync(0xffffffffu, l[j], x);
    // ---- the head's warps together, halving their number each time
    bool lost = false;
    for (int half = slices >> 1; half > 0; half >>= 1) {
      const uint32_t mbar = sbase + SM::kBar + 8 * (2 * SM::kStages + h * QS + sub);
      const int pair = slice & (half - 1);
      const uint32_t buf = sbase + SM::kMerge + ((h * QS + sub) * (slices >> 1) + pair) * SM::kMergeWarp;
      if (slice >= half && slice < 2 * half) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(buf + (mt * 32 + lane) * 16),
                       "f"(o[mt][0]), "f"(o[mt][1]), "f"(o[mt][2]), "f"(o[mt][3]) : "memory");
        asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(buf + (MT * 32 + lane) * 16),
                     "f"(m[0]), "f"(m[1]), "f"(l[0]), "f"(l[1]) : "memory");
      }
      // every warp of the head arrives twice per halving: written, read
#pragma unroll 1
      for (int step = 0; step < 2; ++step) {
        if (step == 1 && slice < half) {
          float v[4], x[2], y[2];
          asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(buf + (MT * 32 + lane) * 16) : "memory");
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float top = fmaxf(m[j], v[j]);
            x[j] = m[j] == -INFINITY ? 0.f : fast_exp2(m[j] - top);
            y[j] = v[j] == -INFINITY ? 0.f : fast_exp2(v[j] - top);
            m[j] = top;
            l[j] = l[j] * x[j] + v[2 + j] * y[j];
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                         : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(buf + (mt * 32 + lane) * 16) : "memory");
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mt][i] = o[mt][i] * x[i & 1] + v[i] * y[i & 1];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(mbar);
        if (!mbar_wait(mbar, sync_phase & 1)) lost = true;
        __syncwarp();
        ++sync_phase;
      }
    }
    if (lost) {
      if (lane == 0) report(a.err, kErrTimeout);
      break;
    }
    if (slice > 0) continue;

    // ---- the result, or this CTA's part of it: D / 8 values of heads qoff + 2 tq and the next
    const bool complete = si.flags & kInfoComplete;
    int peek = -1;
    int32_t* count = merge_cnt + ((size_t)si.dec * a.Hkv + kvh) * QS + sub;
    if (!complete && lane == 0)
      asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(peek) : "l"(count) : "memory");
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int hl = qoff + 2 * tq + j;
      if (hl >= a.G) continue;
      const int head = kvh * a.G + hl;
      if (complete) {
        const float inv = 1.f / l[j];
        uint4* dst = reinterpret_cast<uint4*>(outg + ((size_t)si.tok * a.Hq + head) * D + g * (D / 8));
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint32_t r[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            r[k] = pack_bf16x2(o[4 * i + k][j] * inv, o[4 * i + k][2 + j] * inv);
          dst[i] = make_uint4(r[0], r[1], r[2], r[3]);
        }
        if (g == 0 && a.lse != nullptr)
          a.lse[(size_t)si.tok * a.Hq + head] = (m[j] + __log2f(l[j])) * 0.6931471805599453f;
      } else {
        const size_t row = ((size_t)c + si.dec) * a.Hq + head;
        float4* dst = reinterpret_cast<float4*>(part_o + row * D + g * (D / 8));
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          dst[i] = make_float4(o[2 * i][j], o[2 * i][2 + j], o[2 * i + 1][j], o[2 * i + 1][2 + j]);
        if (g == 0) part_ml[row] = make_float2(m[j], l[j]);
      }
    }
    if (!complete) {
      // the last warp to finish this (sequence, KV head, group of 8 query heads) merges its parts
      const int cf = cta_of_tile(si.p0, ntiles, N), cl = cta_of_tile(si.p1 - 1, ntiles, N);
      __threadfence();
      __syncwarp();
      int last = __shfl_sync(0xffffffffu, peek, 0) == cl - cf ? 1 : 0;
      if (!last) {
        if (lane == 0) last = atomicAdd(count, 1) == cl - cf;
        last = __shfl_sync(0xffffffffu, last, 0);
        if (last) __threadfence();
      }
      if (last)
        merge_parts<D, false>(a, part_ml, part_o, si.dec, si.tok, kvh, cf, cl, qoff,
                              qoff + 8 < a.G ? qoff + 8 : a.G, lane);
    }
  }
}

// The kernel's 512 threads are launched with 128 registers each.
constexpr int kRegsQuantConsume = 176, kRegsQuantRest = 80;
constexpr int kQuantProducer = 8;  // the producer warp (consumers are warps 0 .. 7 at most)
static_assert(2 * kRegsQuantConsume + 2 * kRegsQuantRest <= 4 * 128, "register split exceeds the launch");

// One CTA of the pass, number b of a.decode_grid: one of the N ranges of each KV-head group; beside chunk
// items the one that it takes by its SM, and where it arrived last those that are left (cb_place.cuh).
template <int D, int QS, bool kMod>
__device__ __forceinline__ void quant_decode_cta(const AttnArgs& a, const QuantArgs& qa,
                                                 const ScoreArgs& sc, const CUtensorMap* kmap,
                                                 const CUtensorMap* vmap, uint8_t* smem_raw, int b) {
  using SM = QDecodeSmem<D, QS>;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int HB = a.Hkv < 8 / QS ? a.Hkv : 8 / QS;
  const int slices = 1 << (qa.tile_log2 - 5);
  const int n_cons = QS * HB * slices;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WsLayout L = ws_layout(a.R, a.T, a.Hq, a.D, a.pack);
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(a.ws + L.header);
  const int4* dec_rec = reinterpret_cast<const int4*>(a.ws + L.dec_rec);
  const int32_t* cta_first = reinterpret_cast<const int32_t*>(a.ws + L.cta_first);
  const long long ntiles = hdr->dec_tiles;
  const int N = hdr->decode_ctas, n_dec = hdr->n_dec;
  if (ntiles == 0) return;
  const int total = N * (a.decode_grid / a.decode_ctas);
  int* shared = reinterpret_cast<int*>(smem + SM::kRange);  // this CTA's ranges
  if (threadIdx.x == 0) {
    const int c = decode_cta_index(b % a.decode_ctas, N, a.decode_ctas), mine = b / a.decode_ctas * N + c;
    RangeClaim r = {mine, c < 0 ? mine : mine + 1};
    if (total < a.decode_grid && hdr->pf_qtiles > 0 && a.prefill_ctas > 0)
      r = claim_range(hdr, total, a.decode_grid, a.chunk_ctas);
    shared[0] = r.first;
    shared[1] = r.end;
  }
  const uint32_t bars = sbase + SM::kBar;
  auto init = [&]() {
    for (int i = 0; i < SM::kStages; ++i) {
      // the bytes announced, and each producer lane's small copies
      mbar_init(bars + 8 * i, qa.copy == 0 ? 1 : 1 + 32);
      mbar_init(bars + 8 * (SM::kStages + i), n_cons);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bars + 8 * (2 * SM::kStages + i), slices);
    fence_barrier_init();
  };
  if (threadIdx.x == 0) init();
  __syncthreads();
  const int first = shared[0], end = shared[1];
  if (first >= end) {
    __syncthreads();
    if (threadIdx.x == 0)
      for (int i = 0; i < 2 * SM::kStages + 4; ++i) mbar_inval(bars + 8 * i);
    return;
  }
  // A role's work on every range of this CTA.
  auto ranges = [&](auto&& work) {
    for (int range = first;;) {
      const int hg = range / N, c = range - hg * N;
      const long long t0 = ntiles * c / N, t1 = ntiles * (c + 1) / N;
      const int d_first = cta_first[c];
      if (t0 < t1 && d_first >= 0 && d_first < n_dec) work(c, hg, d_first, t0, t1);
      __syncthreads();
      const bool more = ++range < end;
      if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * SM::kStages + 4; ++i) mbar_inval(bars + 8 * i);
        if (more) init();
      }
      if (!more) break;
      __syncthreads();
    }
  };
  auto produce = [&](int c, int hg, int d_first, long long t0, long long t1) {
    quant_produce<D, QS>(a, qa, kmap, vmap, sbase, reinterpret_cast<int*>(smem + SM::kTokens), n_dec,
                         dec_rec, d_first, hg, HB, t0, t1, lane);
  };
  auto consume = [&](int c, int hg, int, long long t0, long long t1) {
    quant_consume<D, QS, kMod>(a, qa, sc, sbase, c, hg, HB, slices, warp, t1 - t0, ntiles, N, L, lane);
  };
  // The consumers hold a whole stage in registers: they take what the warps behind them leave, of which
  // one works: the producer.
  if (warp < 8) {
    regs_inc<kRegsQuantConsume>();
    if (warp < n_cons)
      ranges(consume);
    else
      ranges([](int, int, int, long long, long long) {});
    regs_dec<128>();  // as launched
  } else {
    regs_dec<kRegsQuantRest>();
    if (warp == kQuantProducer)
      ranges(produce);
    else
      ranges([](int, int, int, long long, long long) {});
    regs_inc<128>();
  }
}

}  // namespace cb

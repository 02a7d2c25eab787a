// The chunk pass's K and V tiles from the quantised cache: the two roles that take the place of its TMA
// producer.
//
// The tensor cores read bf16 tiles with the 128-byte swizzle, the pass's usual operands, and everything
// behind them is the usual pass (cb_prefill.cuh).  A tile is made from codes on the way from L2 to
// shared memory: c * 2^e is exact in bf16, so nothing is lost and no scale is left to the products.
// (The tensor cores' own 8-bit products would take the codes as they are, but need the queries and the
// probabilities in 8 bits too, which costs either accuracy or a second product and more work in the
// softmax warps.)  What bounds the pass is this part's instructions, four per two values on the
// converting warps: 8 chunks of 512 tokens on up to 4096 keys (32 query, 8 KV heads of 128) take 152 us,
// 754 TFLOP/s, on a bf16 cache 150; on up to 8192 keys 230 and 218.
#pragma once

#include <cstddef>

#include "cb_prefill.cuh"
#include "cb_quant.cuh"

namespace cb {

// Warp 0: the Q tiles of each item by TMA, and per K/V tile every key's row in the pool with its scales,
// into a ring of kRowSlots slots.  It runs ahead of the converting warps, so the chain block table ->
// scale is off their path.
template <int D, bool kMod>
__device__ __forceinline__ void quant_rows(const AttnArgs& a, const QuantArgs& qa,
                                           const CUtensorMap* qmap, uint8_t* smem, uint32_t sbase,
                                           int lane) {
  using SM = PrefillSmem<D>;
  using QM = QuantPrefillSmem<D>;
  auto bar = [&](int i) -> uint32_t { return sbase + SM::kBar + 8 * i; };
  const uint32_t row_full = sbase + QM::kBar, row_empty = row_full + 8 * kRowSlots;
  RowSlot* ring = reinterpret_cast<RowSlot*>(smem + QM::kRows);
  if (lane == 0) tma_prefetch_desc(qmap);
  const int whole = kChunkKeys / a.bs, rest = kChunkKeys - whole * a.bs;  // a tile in blocks
  uint32_t n = 0;  // tiles so far
  bool ok = true;
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (!__all_sync(0xffffffffu, mbar_wait(b, parity))) {
      if (lane == 0) report(a.err, kErrTimeout);
      ok = false;
    }
  };
  for (uint32_t k = 0; ok; ++k) {
    const int slot = k & 1;
    wait(bar(SM::bItemFull + slot), (k >> 1) & 1);
    if (!ok) break;
    const PfItemOf<kMod> it =
        *reinterpret_cast<const PfItemOf<kMod>*>(smem + SM::kItems + slot * SM::kItemSlot);
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(SM::bItemEmpty + slot));
    if (it.item < 0) break;
    const int m_claim = max(0, it.nt_all - it.j0 - 3);  // (cb_prefill.cuh: when to claim the next item)
    wait(bar(SM::bQEmpty), (k & 1) ^ 1);
    if (!ok) break;
    if (lane == 0) {
      mbar_arrive_expect_tx(bar(SM::bQFull), (it.hasB ? 2 : 1) * SM::kQTile);
#pragma unroll
      for (int half = 0; half < SM::kHalves; ++half)
        tma_load_3d(sbase + SM::kQ0 + half * SM::kQHalf, qmap, bar(SM::bQFull), half * 64, it.head[0],
                    it.tok[0]);
      if (it.hasB) {
#pragma unroll
        for (int half = 0; half < SM::kHalves; ++half)
          tma_load_3d(sbase + SM::kQ0 + SM::kQTile + half * SM::kQHalf, qmap, bar(SM::bQFull),
                      half * 64, it.head[1], it.tok[1]);
      }
    }
    const int32_t* table = a.block_table + (size_t)it.s * a.max_blocks;
    // Three tiles are in work: one's factors are written, the next one's scales and the block ids of the
    // one behind it are on their way (with the chain of both loads per tile the pass waited for this warp at
    // times: 8 chunks of 512 tokens on up to 4096 keys 169 us, so 166).
    int lb[4], off[4];  // the block and the offset in it of this lane's keys, in the tile of `ent`
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pos = it.j0 * kChunkKeys + 32 * i + lane;
      lb[i] = pos / a.bs;
      off[i] = pos - lb[i] * a.bs;
    }
    int ent[4], tok[4];
    unsigned short sc[4];
    // keys before the earliest query's window are not read: the table's entries may name no block any more
    const int lo = kMod ? window_first_key(it.ctx + it.qoff[0], a.window) : 0;
    auto has_key = [&](int j, int i) {
      const int pos = j * kChunkKeys + 32 * i + lane;
      return pos < it.nk_all && (!kMod || pos >= lo);
    };
    auto fetch = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ent[i] = -1;
        if (has_key(j, i) && lb[i] < a.max_blocks) ent[i] = __ldg(table + lb[i]);
      }
    };
    auto resolve = [&](int j) {  // ent's tokens, of tile j, and their scales
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tok[i] = -1;
        if (ent[i] >= 0 && ent[i] < a.P)
          tok[i] = ent[i] * a.bs + off[i];
        else if (has_key(j, i))
          report(a.err, kErrOutOfRange);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[i] = 0;
        if (tok[i] >= 0)
          sc[i] = __ldg(reinterpret_cast<const unsigned short*>(qa.scales) + (size_t)tok[i] * a.Hkv + it.kvh);
      }
    };
    auto advance = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        off[i] += rest;
        lb[i] += whole;
        if (off[i] >= a.bs) {
          off[i] -= a.bs;
          ++lb[i];
        }
      }
    };
    fetch(it.j0);
    resolve(it.j0);
    advance();
    fetch(it.j0 + 1);
    for (int j = it.j0; j < it.nt_all && ok; ++j, ++n) {
      int tok_j[4];
      unsigned short sc_j[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tok_j[i] = tok[i];
        sc_j[i] = sc[i];
      }
      resolve(j + 1);
      advance();
      fetch(j + 2);
      RowSlot& rs = ring[n % kRowSlots];
      wait(row_empty + 8 * (n % kRowSlots), ((n / kRowSlots) & 1) ^ 1);
      // The factors: 2^120 (codes_to_bf16x4) times the scale, which bf16 holds for scales up to 2^7; the
      // rest of a larger one is a second factor.
      bool more = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ek = (int)(sc_j[i] & 255) - kQuantBias, ev = (int)(sc_j[i] >> 8) - kQuantBias;
        const uint32_t fk = ek == kQuantNan - kQuantBias ? 0x7fffu : (uint32_t)(247 + min(ek, 7)) << 7;
        const uint32_t fv = ev == kQuantNan - kQuantBias ? 0x7fffu : (uint32_t)(247 + min(ev, 7)) << 7;
        // (where there is no key: the pool's first row, times 0)
        const int at = row_place<D>(32 * i + lane);
        rs.row[at] = tok_j[i] < 0 ? 0u : (uint32_t)tok_j[i] * a.Hkv + it.kvh;
        rs.factor[at] = tok_j[i] < 0 ? 0u : fk | fv << 16;
        rs.more[at] = (uint32_t)(127 + max(ek - 7, 0)) << 7 | (uint32_t)(127 + max(ev - 7, 0)) << 23;
        more = more || (tok_j[i] >= 0 && max(ek, ev) > 7);
      }
      more = __any_sync(0xffffffffu, more);
      if (lane == 0) {
        rs.flags = (j == it.nt_all - 1 ? kRowLast : 0) | (more ? kRowMore : 0);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(row_full + 8 * (n % kRowSlots));
        if (j - it.j0 == m_claim) mbar_arrive(bar(SM::bClaim));
      }
    }
  }
  if (ok) {  // no more tiles
    wait(row_empty + 8 * (n % kRowSlots), ((n / kRowSlots) & 1) ^ 1);
    if (lane == 0) {
      ring[n % kRowSlots].flags = kRowEnd;
      mbar_arrive(row_full + 8 * (n % kRowSlots));
    }
  }
}

// Four codes to bf16 (two words), times f (2^120 times a row's scale, as bf16 twice).  A code's bits
// s eeee mmm moved to bf16's sign, low exponent and high mantissa bits are its value times 2^-120 (its
// exponent's bias is 7, bf16's 127), subnormal codes included, so one product makes it the stored value.
__device__ __forceinline__ void codes_to_bf16x4(uint32_t w, uint32_t f, uint32_t& lo, uint32_t& hi) {
  uint32_t x, y;
  // each code as 16 bits with its sign above it
  asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(x) : "r"(w));
  asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(y) : "r"(w));
  x = (x << 4) & 0x87f087f0u;
  y = (y << 4) & 0x87f087f0u;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(x), "r"(f));
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(y), "r"(f));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t x, uint32_t f) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(f));
  return r;
}

// Warps 12-15: K and V tiles of the ring's stages.  Stage m of an item holds K tile m and V tile m - 1,
// as in cb_prefill.cuh, so an item's order is K(0) | K(1) V(0) | ... | K(n-1) V(n-2) | V(n-1), stages
// between the bars.  A thread makes the same 16 columns of D / 16 rows of every tile.  Its codes wait in
// shared memory, in pieces of 16 bytes that only this thread copies and reads; the next tile's in that
// order are copied behind the conversion of this one's.
//   What one warp per scheduler executes for a stage is what bounds the pass (its copies are there in
// time), beside softmax warps whose code displaces its own from the nearest instruction cache: so few
// instructions in one small loop count for more than few loads or dependences.  4 chunks of 2048 tokens on
// up to 16384 keys (32 query, 8 KV heads of 128) took 1262 us with the next tile's codes in registers,
// loaded between the conversions, all unrolled; 1072 with the codes here; 1024 with a loop over four rows;
// 967 with the order's decisions once a stage and rows without a predicate; 956 with the next rows read
// beside the codes; 947 with a thread's rows and factors side by side.  (Two rows at a time 993, eight 1020,
// one 1326.  On a bf16 cache 855.)
template <int D>
__device__ __forceinline__ void quant_convert(const AttnArgs& a, const QuantArgs& qa, uint8_t* smem,
                                              uint32_t sbase) {
  using SM = PrefillSmem<D>;
  using QM = QuantPrefillSmem<D>;
  constexpr int NS = SM::kStages, NR = QM::kRowsPerThread;
  constexpr int kGroup = 4;  // rows at a time
  constexpr uint32_t kFactors = offsetof(RowSlot, factor), kMore = offsetof(RowSlot, more);
  auto bar = [&](int i) -> uint32_t { return sbase + SM::kBar + 8 * i; };
  const uint32_t row_full = sbase + QM::kBar, row_empty = row_full + 8 * kRowSlots;
  const uint32_t rings = sbase + QM::kRows;
  const int t = threadIdx.x - 384, lane = threadIdx.x & 31;
  // Columns 16 c .. 16 c + 15 of rows r0 + 128 / NR * i.  Eight neighbouring threads (one pass of a
  // 16-byte access) have four columns of two rows, so that their swizzled stores meet no bank twice.
  const int c = D == 128 ? (t & 3) + 4 * ((t >> 3) & 1) : t & 3;
  const int r0 = D == 128 ? ((t >> 2) & 1) + 2 * (t >> 4) : t >> 2;
  constexpr int kStep = 128 / NR;  // (a multiple of 8: all rows of a thread have one swizzle)
  static_assert(kStep % 8 == 0, "rows of a thread share their swizzle");
  const uint32_t at0 = sw128((c >> 2) * SM::kKVHalf, r0, 2 * (c & 3));
  const uint32_t at1 = sw128((c >> 2) * SM::kKVHalf, r0, 2 * (c & 3) + 1);
  const uint32_t codes = sbase + QM::kCodes + t * 16;  // this thread's pieces of a tile, 2 KB apart
  bool ok = true;
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (ok && !mbar_wait(b, parity)) {
      if (lane == 0) report(a.err, kErrTimeout);
      ok = false;
    }
  };
  auto slot = [&](uint32_t i) -> uint32_t { return rings + (i % kRowSlots) * (uint32_t)sizeof(RowSlot); };
  auto ready = [&](uint32_t i) { wait(row_full + 8 * (i % kRowSlots), (i / kRowSlots) & 1); };
  auto flags_of = [&](uint32_t i) -> int {
    int f;
    asm volatile("ld.shared.s32 %0, [%1];" : "=r"(f) : "r"(slot(i) + (uint32_t)offsetof(RowSlot, flags)));
    return f;
  };
  const uint8_t* kp = qa.k_pages + 16 * c;
  const uint8_t* vp = qa.v_pages + 16 * c;
  // This thread's piece of a row to shared memory.
  auto copy = [&](const uint8_t* pages, uint32_t row, int k) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(codes + 2048 * k), "l"(pages + (size_t)row * D)
                 : "memory");
  };
  auto copy4 = [&](const uint8_t* pages, const uint4& row, int k0) {
    copy(pages, row.x, k0);
    copy(pages, row.y, k0 + 1);
    copy(pages, row.z, k0 + 2);
    copy(pages, row.w, k0 + 3);
  };
  auto commit = [&]() { asm volatile("cp.async.commit_group;" ::: "memory"); };
  auto convert = [&](const uint4& x, uint32_t f, uint32_t dst, int k) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) codes_to_bf16x4(w[i], f, y[2 * i], y[2 * i + 1]);
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + at0 + kStep * 128 * k), "r"(y[0]),
                 "r"(y[1]), "r"(y[2]), "r"(y[3]));
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(dst + at1 + kStep * 128 * k), "r"(y[4]),
                 "r"(y[5]), "r"(y[6]), "r"(y[7]));
  };
  uint32_t n = 0;        // the tile of this stage's keys, of all tiles so far; its values are tile n - 1
  bool has_v = false;    // not an item's first stage
  int flags = 0, before = 0;  // of tiles n and n - 1
  bool loaded = false;   // the codes of tile n's keys are on their way although its item has not begun
  for (uint32_t g = 0;; ++g) {
    uint32_t at = slot(n) + 4 * NR * r0;  // this thread's first row in tile n's slot
    if (!has_v) {          // an item begins
      ready(n);
      if (!ok) break;
      flags = flags_of(n);
      if (flags & kRowEnd) break;
      if (!loaded) {
#pragma unroll 1
        for (int k0 = 0; k0 < NR; k0 += kGroup) {
          const uint4 row = lds128(at + 4 * k0);
          copy4(kp, row, k0);
          commit();
        }
      }
    }
    const bool has_k = !has_v || !(before & kRowLast);
    // The tile that the next stage begins with: keys, an item's last values, or the next item's first
    // keys where its rows are known already.
    const bool nv = has_k && (flags & kRowLast);
    uint32_t nn = n;
    loaded = true;
    if (has_k && !nv)
      ready(++nn);
    else if (!has_k)
      loaded = __all_sync(0xffffffffu, mbar_test(row_full + 8 * (n % kRowSlots), (n / kRowSlots) & 1)) &&
               !(flags_of(n) & kRowEnd);
    const int flags_n = flags_of(nn);
    wait(bar(SM::bEmpty + g % NS), ((g / NS) & 1) ^ 1);
    if (!ok) break;
    const uint32_t at_n = slot(nn) + 4 * NR * r0, at_v = slot(n - 1) + 4 * NR * r0;
    uint32_t dst = sbase + SM::kStage0 + (g % NS) * SM::kStageBytes, pick = 0x1010u;
    if (!has_k) {
      dst += SM::kKVTile;
      pick = 0x3232u;
      at = at_v;
    }
    // keys, then values; copies of what comes behind each
#pragma unroll 1
    for (int tiles = has_k && has_v ? 2 : 1; tiles > 0; --tiles) {
      const bool more = (has_k && tiles == (has_v ? 2 : 1) ? flags : before) & kRowMore;
      const bool values_next = tiles == 2 || nv;
      const uint8_t* next = values_next ? vp : kp;
      const uint32_t at_next = tiles == 2 ? at_v : at_n;
#pragma unroll 1
      for (int k0 = 0; k0 < NR; k0 += kGroup) {
        // (this tile's later pieces may still be on their way)
        asm volatile("cp.async.wait_group %0;" ::"n"(NR / kGroup - 1) : "memory");
        const uint4 row = lds128(at_next + 4 * k0), fs = lds128(at + kFactors + 4 * k0);
        uint4 x[kGroup];
#pragma unroll
        for (int k = 0; k < kGroup; ++k) x[k] = lds128(codes + 2048 * (k0 + k));
        convert(x[0], __byte_perm(fs.x, 0, pick), dst, k0);
        convert(x[1], __byte_perm(fs.y, 0, pick), dst, k0 + 1);
        convert(x[2], __byte_perm(fs.z, 0, pick), dst, k0 + 2);
        convert(x[3], __byte_perm(fs.w, 0, pick), dst, k0 + 3);
        if (loaded || tiles == 2) copy4(next, row, k0);
        commit();
      }
      if (more) {  // the second factors: over what this thread has just written
#pragma unroll 1
        for (int i = 0; i < 2 * NR; ++i) {
          const uint32_t to = dst + (i & 1 ? at1 : at0) + kStep * 128 * (i >> 1);
          uint32_t m;
          asm volatile("ld.shared.u32 %0, [%1];"
                       : "=r"(m)
                       : "r"(at + kMore + 4 * (i >> 1)));
          m = __byte_perm(m, 0, pick);
          uint32_t y[4];
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]) : "r"(to));
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = mul_bf16x2(y[k], m);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(to), "r"(y[0]), "r"(y[1]), "r"(y[2]),
                       "r"(y[3]));
        }
      }
      dst += SM::kKVTile;
      pick = 0x3232u;
      at = at_v;
    }
    // the stage is complete
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(bar(SM::bFull + g % NS));
      if (has_v) mbar_arrive(row_empty + 8 * ((n - 1) % kRowSlots));
    }
    has_v = has_k;
    if (has_k) {
      before = flags;
      flags = flags_n;
      ++n;
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace cb

// The chunk pass's K and V tiles from the quantised cache: the two roles that take the place of its TMA
// producer.
//
// The tensor cores read bf16 tiles with the 128-byte swizzle, the pass's usual operands, and everything
// behind them is the usual pass (cb_prefill.cuh).  A tile is made from codes on the way from L2 to
// shared memory: c * 2^e is exact in bf16, so nothing is lost and no scale is left to the products.
// (The tensor cores' own 8-bit products would take the codes as they are, but need the queries and the
// probabilities in 8 bits too, which costs either accuracy or a second product and more work in the
// softmax warps, which bound the pass.)  What bounds this part is the latency of the codes' loads -- a
// thread has one tile's 16 x D / 16 of them in flight, its registers hold no more -- and four instructions
// per two values on the converting warps, beside the softmax warps of the same schedulers: 8 chunks of 512
// tokens on up to 4096 keys (32 query, 8 KV heads of 128) take 166 us, 690 TFLOP/s, without the loads 141,
// on a bf16 cache 146 to 150.  Codes copied by TMA into a ring of their own, which costs the tiles' ring a
// stage and another pass over shared memory: 174 us.
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
    auto fetch = [&](int j) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ent[i] = -1;  // no key
        if (j * kChunkKeys + 32 * i + lane < it.nk_all)
          ent[i] = lb[i] < a.max_blocks ? __ldg(table + lb[i]) : -2;
      }
    };
    auto resolve = [&]() {  // ent's tokens, and their scales
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tok[i] = -1;
        if (ent[i] >= 0 && ent[i] < a.P)
          tok[i] = ent[i] * a.bs + off[i];
        else if (ent[i] != -1)
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
    resolve();
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
      resolve();
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
        rs.row[32 * i + lane] = make_uint2(tok_j[i] < 0 ? kNoRow : (uint32_t)tok_j[i] * a.Hkv + it.kvh,
                                           tok_j[i] < 0 ? 0u : fk | fv << 16);
        rs.more[32 * i + lane] = (uint32_t)(127 + max(ek - 7, 0)) << 7 | (uint32_t)(127 + max(ev - 7, 0)) << 23;
        more = more || (tok_j[i] >= 0 && max(ek, ev) > 7);
      }
      more = __any_sync(0xffffffffu, more);
      if (lane == 0) {
        rs.flags = (j == it.j0 ? kRowFirst : 0) | (j == it.nt_all - 1 ? kRowLast : 0) | (more ? kRowMore : 0);
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
// shared memory (pieces of 16 bytes that only this thread copies and reads); the next tile's in that order
// are copied behind the conversion of this one's.  In registers they would be taken from the softmax
// warps: those spilled, and as the pass leaves L1 some 20 KB, through which the codes pass, a part of the
// spilled values came from L2, in the chain of every K/V step (4 chunks of 2048 tokens on up to 16384 keys:
// 1262 us, so FIGURE).  One copy of the conversion, in a loop over tiles: written out for each place in the
// order the four warps' code did not stay in the instruction cache beside the softmax warps'.
template <int D>
__device__ __forceinline__ void quant_convert(const AttnArgs& a, const QuantArgs& qa, uint8_t* smem,
                                              uint32_t sbase) {
  using SM = PrefillSmem<D>;
  using QM = QuantPrefillSmem<D>;
  constexpr int NS = SM::kStages, NR = QM::kRowsPerThread;
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
  const uint32_t codes = sbase + QM::kCodes + t * 16;  // this thread's pieces of a V tile, 2 KB apart
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
  // A tile's rows (or factors, at = 4) of this thread.
  auto rows_of = [&](uint32_t i, uint32_t at, uint32_t (&r)[NR]) {
#pragma unroll
    for (int k = 0; k < NR; ++k)
      asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[k]) : "r"(slot(i) + 8 * (r0 + kStep * k) + at));
  };
  // One row's piece to shared memory (zeros where there is no row).
  auto copy = [&](const uint8_t* pages, uint32_t row, int k) {
    const bool none = row == kNoRow;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(codes + 2048 * k),
                 "l"(pages + (none ? 0 : (size_t)row * D + 16 * c)), "r"(none ? 0 : 16)
                 : "memory");
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
  uint32_t g = 0;              // stages so far
  uint32_t n = 0;              // the tile at hand, of all tiles so far
  bool v = false;              // its values
  int flags = 0, flags1 = 0;   // of tile n; v: of tile n + 1, where that is the same item's
  uint32_t kst = 0;
  bool loaded = false;         // its codes are on their way
  while (true) {
    if (!loaded) {             // an item begins
      ready(n);
      if (!ok) break;
      flags = flags_of(n);
      if (flags & kRowEnd) break;
      uint32_t row[NR];
      rows_of(n, 0, row);
#pragma unroll
      for (int k = 0; k < NR; ++k) {
        copy(qa.k_pages, row[k], k);
        if (k % 4 == 3) commit();
      }
    }
    // The next tile in the order.
    uint32_t nn;
    bool nv;
    loaded = true;
    if (!v) {
      const bool first = flags & kRowFirst, last = flags & kRowLast;
      nv = !first || last;
      nn = first ? (last ? n : n + 1) : n - 1;
    } else if (!(flags & kRowLast)) {
      nv = flags1 & kRowLast;
      nn = nv ? n + 1 : n + 2;
    } else {  // the next item's first keys, where its rows are known already
      nv = false;
      nn = n + 1;
      loaded = __all_sync(0xffffffffu, mbar_test(row_full + 8 * (nn % kRowSlots), (nn / kRowSlots) & 1)) &&
               !(flags_of(nn) & kRowEnd);
    }
    if (!nv && loaded) ready(nn);
    const int flags_n = loaded ? (nn == n ? flags : flags_of(nn)) : 0;
    // A stage begins with keys, or with an item's last values.
    if (!v || (flags & kRowLast)) {
      wait(bar(SM::bEmpty + g % NS), ((g / NS) & 1) ^ 1);
      kst = sbase + SM::kStage0 + (g % NS) * SM::kStageBytes;
    }
    if (!ok) break;
    const uint32_t dst = kst + (v ? SM::kKVTile : 0);
    // (all loads of rows and factors ahead of the stores, which the compiler keeps in order with them)
    uint32_t fs[NR], row[NR];
    rows_of(n, 4, fs);
    rows_of(nn, 0, row);
    const uint8_t* next = nv ? qa.v_pages : qa.k_pages;
    const uint32_t pick = v ? 0x3232u : 0x1010u;
#pragma unroll
    for (int k0 = 0; k0 < NR; k0 += 4) {
      // (this tile's later pieces may still be on their way)
      asm volatile("cp.async.wait_group %0;" ::"n"(NR / 4 - 1) : "memory");
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = lds128(codes + 2048 * (k0 + k));
#pragma unroll
      for (int k = 0; k < 4; ++k) convert(x[k], __byte_perm(fs[k0 + k], 0, pick), dst, k0 + k);
      if (loaded) {
#pragma unroll
        for (int k = 0; k < 4; ++k) copy(next, row[k0 + k], k0 + k);
      }
      commit();
    }
    if (flags & kRowMore) {  // the second factors: over what this thread has just written
#pragma unroll 1
      for (int i = 0; i < 2 * NR; ++i) {
        const uint32_t at = dst + (i & 1 ? at1 : at0) + kStep * 128 * (i >> 1);
        uint32_t m;
        asm volatile("ld.shared.u32 %0, [%1];"
                     : "=r"(m)
                     : "r"(slot(n) + (uint32_t)offsetof(RowSlot, more) + 4 * (r0 + kStep * (i >> 1))));
        m = __byte_perm(m, 0, pick);
        uint32_t y[4];
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]) : "r"(at));
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = mul_bf16x2(y[k], m);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(y[0]), "r"(y[1]), "r"(y[2]),
                     "r"(y[3]));
      }
    }
    if (v || (flags & kRowFirst)) {  // the stage is complete
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(SM::bFull + g % NS));
        if (v) mbar_arrive(row_empty + 8 * (n % kRowSlots));
      }
      ++g;
    }
    if (!v && nv && nn + 1 == n) flags1 = flags;  // (the values before these keys)
    flags = flags_n;
    n = nn;
    v = nv;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

}  // namespace cb

// The chunk pass's K and V tiles from the quantised cache: the two roles that take the place of its TMA
// producer.
//
// The tensor cores read bf16 tiles with the 128-byte swizzle, the pass's usual operands, and everything
// behind them is the usual pass (cb_prefill.cuh).  A tile is made from codes on the way from L2 to
// shared memory: c * 2^e is exact in bf16, so nothing is lost and no scale is left to the products.
// (The tensor cores' own 8-bit products would take the codes as they are, but need the queries and the
// probabilities in 8 bits too, which costs either accuracy or a second product and more work in the
// softmax warps, which bound the pass.)  What bounds this part is instructions: four per two values on
// the converting warps, beside the softmax warps of the same schedulers.
#pragma once

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
    for (int j = it.j0; j < it.nt_all && ok; ++j, ++n) {
      int tok[4];
      unsigned short sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pos = j * kChunkKeys + 32 * i + lane;
        tok[i] = -1;
        sc[i] = 0;
        if (pos < it.nk_all) {
          const int lb = pos / a.bs;
          const int e = lb < a.max_blocks ? __ldg(table + lb) : -1;
          if (e >= 0 && e < a.P)
            tok[i] = e * a.bs + (pos - lb * a.bs);
          else
            report(a.err, kErrOutOfRange);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (tok[i] >= 0)
          sc[i] = __ldg(reinterpret_cast<const unsigned short*>(qa.scales) + (size_t)tok[i] * a.Hkv + it.kvh);
      RowSlot& rs = ring[n % kRowSlots];
      wait(row_empty + 8 * (n % kRowSlots), ((n / kRowSlots) & 1) ^ 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) rs.row[32 * i + lane] = make_int2(tok[i], sc[i]);
      if (lane == 0) {
        rs.kvh = it.kvh;
        rs.flags = (j == it.j0 ? kRowFirst : 0) | (j == it.nt_all - 1 ? kRowLast : 0);
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
// Not for NaN codes.
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
// as in cb_prefill.cuh.  A thread makes the same 16 columns of D / 16 rows of every tile; the codes of
// the next tile are loaded while this one's are converted, each into the register that just became free.
template <int D>
__device__ __forceinline__ void quant_convert(const AttnArgs& a, const QuantArgs& qa, uint8_t* smem,
                                              uint32_t sbase) {
  using SM = PrefillSmem<D>;
  using QM = QuantPrefillSmem<D>;
  constexpr int NS = SM::kStages, NR = D / 16;  // rows per thread
  auto bar = [&](int i) -> uint32_t { return sbase + SM::kBar + 8 * i; };
  const uint32_t row_full = sbase + QM::kBar, row_empty = row_full + 8 * kRowSlots;
  const RowSlot* ring = reinterpret_cast<const RowSlot*>(smem + QM::kRows);
  const int t = threadIdx.x - 384, lane = threadIdx.x & 31;
  // Columns 16 c .. 16 c + 15 of rows r0 + 128 / NR * i.  Eight neighbouring threads (one pass of a
  // 16-byte access) have four columns of two rows, so that their swizzled stores meet no bank twice.
  const int c = D == 128 ? (t & 3) + 4 * ((t >> 3) & 1) : t & 3;
  const int r0 = D == 128 ? ((t >> 2) & 1) + 2 * (t >> 4) : t >> 2;
  constexpr int kStep = 128 / NR;
  bool ok = true;
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (ok && !mbar_wait(b, parity)) {
      if (lane == 0) report(a.err, kErrTimeout);
      ok = false;
    }
  };
  uint4 raw[NR];
  auto load = [&](const uint8_t* pages, const RowSlot& rs, int i) {
    const int token = rs.row[r0 + kStep * i].x;
    raw[i] = make_uint4(0, 0, 0, 0);
    if (token >= 0)
      raw[i] = __ldg(reinterpret_cast<const uint4*>(pages + ((size_t)token * a.Hkv + rs.kvh) * D) + c);
  };
  // Converts the codes in raw (rows of rs; v: values) into the tile at dst, and loads the next ones.
  auto convert = [&](const RowSlot& rs, bool v, uint32_t dst, const uint8_t* next, const RowSlot& nrs) {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int row = r0 + kStep * i;
      const int e = (rs.row[row].y >> (v ? 8 : 0) & 255) - kQuantBias;
      const uint4 x = raw[i];
      if (next != nullptr) load(next, nrs, i);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t y[8];
      // bf16's exponent ends at 127: a scale above 2^7 is applied in two steps
      const uint32_t f1 = (uint32_t)(127 + 120 + min(e, 7)) << 7, f = f1 | f1 << 16;
      uint32_t nan = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        codes_to_bf16x4(w[k], f, y[2 * k], y[2 * k + 1]);
        nan |= (w[k] & 0x7f7f7f7fu) + 0x01010101u;
      }
      if (e > 7) {
        const uint32_t g1 = (uint32_t)(127 + e - 7) << 7, g = g1 | g1 << 16;
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = mul_bf16x2(y[k], g);
      }
      if (nan & 0x80808080u) {  // a NaN code (0x7f with either sign) among them
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t pair = w[k >> 1] >> (16 * (k & 1));
          if ((pair & 0x7fu) == 0x7fu) y[k] |= 0x7fffu;
          if ((pair & 0x7f00u) == 0x7f00u) y[k] |= 0x7fff0000u;
        }
      }
      const uint32_t tile = dst + (c >> 2) * SM::kKVHalf;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t addr = sw128(tile, row, 2 * (c & 3) + k);
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(y[4 * k]),
                     "r"(y[4 * k + 1]), "r"(y[4 * k + 2]), "r"(y[4 * k + 3]) : "memory");
      }
    }
  };
  uint32_t g = 0;  // stages so far
  auto begin = [&]() -> uint32_t {  // the next stage, once it is free
    wait(bar(SM::bEmpty + g % NS), ((g / NS) & 1) ^ 1);
    return sbase + SM::kStage0 + (g % NS) * SM::kStageBytes;
  };
  auto finish = [&]() {  // the stage is written
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(SM::bFull + g % NS));
    ++g;
  };
  uint32_t n = 0;       // tiles so far
  bool loaded = false;  // raw holds tile n's keys
  auto tile_ready = [&](uint32_t i) { wait(row_full + 8 * (i % kRowSlots), (i / kRowSlots) & 1); };
  auto release = [&](uint32_t i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(row_empty + 8 * (i % kRowSlots));
  };
  while (ok) {
    tile_ready(n);
    if (!ok || (ring[n % kRowSlots].flags & kRowEnd)) break;
    // ---- an item: K of its first tile, then per tile K and the V before it, then the last V
    if (!loaded) {
#pragma unroll
      for (int i = 0; i < NR; ++i) load(qa.k_pages, ring[n % kRowSlots], i);
    }
    loaded = false;
    bool last = ring[n % kRowSlots].flags & kRowLast;
    uint32_t kst = begin();
    if (!last) tile_ready(n + 1);
    if (!ok) break;
    convert(ring[n % kRowSlots], false, kst, last ? qa.v_pages : qa.k_pages, ring[(n + (last ? 0 : 1)) % kRowSlots]);
    finish();
    while (!last && ok) {
      ++n;  // this stage: K of tile n, V of tile n - 1
      const RowSlot &cur = ring[n % kRowSlots], &prev = ring[(n - 1) % kRowSlots];
      last = cur.flags & kRowLast;
      kst = begin();
      if (!ok) break;
      convert(cur, false, kst, qa.v_pages, prev);
      if (!last) tile_ready(n + 1);
      if (!ok) break;
      convert(prev, true, kst + SM::kKVTile, last ? qa.v_pages : qa.k_pages,
              ring[(n + (last ? 0 : 1)) % kRowSlots]);
      finish();
      release(n - 1);
    }
    if (!ok) break;
    kst = begin();
    if (!ok) break;
    // the next item's first keys, where its rows are known already
    const uint32_t i = (n + 1) % kRowSlots;
    loaded = __all_sync(0xffffffffu, mbar_test(row_full + 8 * i, ((n + 1) / kRowSlots) & 1)) &&
             !(ring[i].flags & kRowEnd);
    convert(ring[n % kRowSlots], true, kst + SM::kKVTile, loaded ? qa.k_pages : nullptr, ring[i]);
    finish();
    release(n);
    ++n;
  }
}

}  // namespace cb

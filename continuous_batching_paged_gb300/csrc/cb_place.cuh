// Where the decode ranges run when some SMs run chunk items meanwhile.
//
// The two SMs of a TPC share instruction-cache capacity: a decode CTA beside a chunk CTA of its TPC runs at
// half its speed where the two roles' loops do not fit together (over the 8-bit cache, 12 decode CTAs
// beside 8 chunks of 512 tokens: 364 us, on TPCs of their own 159 us, alone 159 us).  The grid's order
// does not say which SM a CTA gets (a planner that still runs when the CTAs are placed shifts them), so a
// decode CTA looks at its SM: those on the chosen TPCs take the ranges, from a counter; the others leave
// their SMs to the chunk CTAs behind them.  Which CTA computes a range changes no result.
#pragma once

#include "cb_common.cuh"
#include "cb_launch.h"

namespace cb {

// Of one thread of each of the `grid` decode CTAs: the ranges (of `total` < grid) that it takes, first to
// end - 1; most often one or none.  The CTA that arrives last also takes those that are left, if any: the
// chosen SMs may have had too few CTAs, for instance where another launch holds some.  (One atomic per
// CTA, for the claim and the arrival.)
struct RangeClaim {
  int first, end;
};
__device__ __forceinline__ RangeClaim claim_range(PlanHeader* hdr, int total, int grid, int sms) {
  unsigned sm;
  asm("mov.u32 %0, %%smid;" : "=r"(sm));
  const int tpcs = (sms + 1) / 2, pairs = (total + 1) / 2, tpc = (int)(sm >> 1) % tpcs;
  // every tpcs / pairs-th TPC, spread evenly
  const int chosen = (tpc + 1) * pairs / tpcs > tpc * pairs / tpcs;
  const unsigned long long old = atomicAdd(&hdr->dec_claims, (1ull << 32) | (unsigned)chosen);
  const int taken = min((int)(old & 0xffffffffu), total);
  const bool last = (int)(old >> 32) == grid - 1;
  return {taken, last ? total : min(taken + chosen, total)};
}

}  // namespace cb

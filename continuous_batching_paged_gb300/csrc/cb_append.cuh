// Device code of the paged KV-append: a token's cache slot, and the copy of its K/V rows
// (cb_append.cu; the rotary append, cb_rope.cuh, finds its slots the same way).
#pragma once

#include "cb_common.cuh"
#include "cb_launch.h"

namespace cb {

// One warp per new token: the warp finds the token's sequence with 32-way probes of
// cu_seqlens_q (a few rounds instead of a binary search per 16-byte chunk), then each lane
// moves its share of the token's K row and V row (all KV heads: Hkv * D bf16, contiguous in
// both the input and the token-major pool), issuing every load before the first store.
constexpr int kAppendThreads = 256;
constexpr int kAppendMaxChunks = 8;  // 16-byte chunks per lane and tensor in flight

// Cache slot (row of the flattened [P * bs, Hkv, D] pool) of packed token t < cu_seqlens_q[S], and
// its position; -1, after a report, where the metadata is bad.  Called by one full warp.  kPadding: t
// may lie behind the last sequence (-1 then, without a report).
template <bool kPadding = false>
__device__ __forceinline__ long long token_slot(const AppendArgs& a, int t, int lane, int& pos) {
  // Sequence of token t: the last s with cu[s] <= t (cu is non-decreasing).  Each round
  // probes 32 increasing positions in (lo, hi]; the lanes whose probe is <= t form a prefix.
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int span = hi - lo;
    const int p = lo + 1 + (int)((long long)(span - 1) * lane / 31);
    const unsigned le = __ballot_sync(0xffffffffu, __ldg(a.cu_seqlens_q + p) <= t);
    const int k = le ? 31 - __clz(le) : -1;
    const int pk = __shfl_sync(0xffffffffu, p, k < 0 ? 0 : k);
    const int pn = __shfl_sync(0xffffffffu, p, k < 31 ? k + 1 : 31);
    if (k < 0) {
      hi = pk - 1;
    } else {
      lo = pk;
      if (k < 31 && pn - 1 < hi) hi = pn - 1;
    }
  }
  const int s = lo;
  if (s >= a.S) {
    if (!kPadding && lane == 0) report(a.err, kErrOutOfRange);
    return -1;
  }
  const int c0 = __ldg(a.cu_seqlens_q + s), c1 = __ldg(a.cu_seqlens_q + s + 1);
  const int q_len = c1 - c0;
  const int kv = __ldg(a.kv_lens + s);
  if (c0 < 0 || t < c0 || t >= c1 || c1 > a.T || kv < q_len) {
    if (lane == 0) report(a.err, kErrOutOfRange);
    return -1;
  }
  pos = kv - q_len + (t - c0);
  const int lb = pos / a.bs;
  if (lb >= a.max_blocks) {
    if (lane == 0) report(a.err, kErrOutOfRange);
    return -1;
  }
  const int blk = __ldg(a.block_table + (size_t)s * a.max_blocks + lb);
  if (blk < 0 || blk >= a.P) {
    if (lane == 0) report(a.err, kErrOutOfRange);
    return -1;
  }
  return (long long)blk * a.bs + (pos - lb * a.bs);
}

// Tokens handled by warps first_warp, first_warp + nwarps, ...  kMaxChunks: 16-byte chunks per
// lane and tensor in flight (registers: 8 per chunk pair).
template <int kMaxChunks>
__device__ __forceinline__ void append_tokens(const AppendArgs& a, int first_warp, int nwarps) {
  const int lane = threadIdx.x & 31;
  const int cpr = a.Hkv * a.D / 8;  // 16-byte chunks per token row
  const uint4* kn = static_cast<const uint4*>(a.k_new);
  const uint4* vn = static_cast<const uint4*>(a.v_new);
  uint4* kp = static_cast<uint4*>(a.k_pages);
  uint4* vp = static_cast<uint4*>(a.v_pages);
  // Rows at or past cu_seqlens_q[S] are padding of the token tensors: left untouched.
  const int t_end = min(a.T, __ldg(a.cu_seqlens_q + a.S));
  for (int t = first_warp; t < t_end; t += nwarps) {
    int pos;
    const long long slot = token_slot(a, t, lane, pos);
    if (slot < 0) continue;
    const uint4* ks = kn + (size_t)t * cpr;
    const uint4* vs = vn + (size_t)t * cpr;
    uint4* kd = kp + (size_t)slot * cpr;
    uint4* vd = vp + (size_t)slot * cpr;
    for (int base = 0; base < cpr; base += 32 * kMaxChunks) {
      uint4 kr[kMaxChunks], vr[kMaxChunks];
#pragma unroll
      for (int i = 0; i < kMaxChunks; ++i) {
        const int c = base + lane + 32 * i;
        if (c < cpr) {
          kr[i] = __ldg(ks + c);
          vr[i] = __ldg(vs + c);
        }
      }
#pragma unroll
      for (int i = 0; i < kMaxChunks; ++i) {
        const int c = base + lane + 32 * i;
        if (c < cpr) {
          kd[c] = kr[i];
          vd[c] = vr[i];
        }
      }
    }
  }
}

// Checks of cu_seqlens_q that no token's own search sees (cu[0] = 0, non-decreasing,
// cu[S] <= T), spread over the grid's threads: a token of a malformed range may land in a
// neighbouring sequence's range, so the stand-alone append reports the metadata itself.  (The
// append + planner launch leaves this to the planner, which makes the same checks.)
__device__ __forceinline__ void check_cu_seqlens(const AppendArgs& a) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < a.S; i += gridDim.x * blockDim.x) {
    const int c0 = __ldg(a.cu_seqlens_q + i), c1 = __ldg(a.cu_seqlens_q + i + 1);
    if (c1 < c0 || (i == 0 && c0 != 0) || (i == a.S - 1 && c1 > a.T)) report(a.err, kErrOutOfRange);
  }
}

}  // namespace cb

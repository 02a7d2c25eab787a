// Whole-block moves of the paged KV cache: copy-on-write block copies inside the pools, and
// the batched offload (gather to host) / restore (scatter from host) of a list of blocks.
// HBM (or CPU-GPU link) bound: 16-byte vector loads, four per thread in flight before the
// stores, K and V of the same chunk together; grid = a few waves of the SMs.  The quantised cache's scales, 2 of
// 2 D + 2 bytes of a row, go in the same launch.
#include "cb_common.cuh"
#include "cb_launch.h"

namespace cb {

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// Source and destination block of pair i (linear host position for the host side); false: out of range.
__device__ __forceinline__ bool move_pair(const BlockMoveArgs& a, int i, long long& sblk, long long& dblk) {
  sblk = dblk = i;
  if (a.mode != kMoveRestore) sblk = a.src_idx[i];
  if (a.mode != kMoveOffload) dblk = a.dst_idx[i];
  return (a.mode == kMoveRestore || (sblk >= 0 && sblk < a.P)) &&
         (a.mode == kMoveOffload || (dblk >= 0 && dblk < a.P));
}

// The blocks' scales in words of type W, which divides a block's scale bytes (bad ids are reported with the
// codes).
template <typename W>
__device__ __forceinline__ void move_scales(const BlockMoveArgs& a) {
  const int wpb = a.scale_bytes / (int)sizeof(W);
  const long long total = (long long)a.n * wpb;
  for (long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x; idx < total;
       idx += (long long)gridDim.x * blockDim.x) {
    const int i = (int)(idx / wpb);
    const long long w = idx - (long long)i * wpb;
    long long sblk, dblk;
    if (!move_pair(a, i, sblk, dblk) || (a.mode == kMoveCopy && sblk == dblk)) continue;
    reinterpret_cast<W*>(a.dst_scales)[dblk * wpb + w] = reinterpret_cast<const W*>(a.src_scales)[sblk * wpb + w];
  }
}

template <bool kScales>
__global__ void __launch_bounds__(kMoveThreads) block_move_kernel(BlockMoveArgs a) {
  if constexpr (kScales) {
    if (a.scale_bytes % 16 == 0) move_scales<uint4>(a);
    else if (a.scale_bytes % 8 == 0) move_scales<uint2>(a);
    else if (a.scale_bytes % 4 == 0) move_scales<uint32_t>(a);
    else move_scales<uint16_t>(a);
  }
  const long long cpb = a.block_bytes / 16;  // 16-byte chunks per block and pool
  const long long total = (long long)a.n * cpb;
  const long long stride = (long long)gridDim.x * blockDim.x;
  for (long long base = (long long)blockIdx.x * blockDim.x + threadIdx.x; base < total;
       base += stride * kMoveUnroll) {
    uint4 kv[kMoveUnroll][2];
    long long doff[kMoveUnroll];
    bool ok[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      const long long idx = base + u * stride;
      ok[u] = false;
      if (idx >= total) continue;
      const int i = (int)(idx / cpb);
      const long long c = idx - (long long)i * cpb;
      long long sblk, dblk;
      if (!move_pair(a, i, sblk, dblk)) {
        if (c == 0) report(a.err, kErrOutOfRange);
        continue;
      }
      if (a.mode == kMoveCopy && sblk == dblk) continue;
      const long long soff = sblk * a.block_bytes + c * 16;
      doff[u] = dblk * a.block_bytes + c * 16;
      kv[u][0] = *reinterpret_cast<const uint4*>(a.src[0] + soff);
      kv[u][1] = *reinterpret_cast<const uint4*>(a.src[1] + soff);
      ok[u] = true;
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      if (!ok[u]) continue;
      *reinterpret_cast<uint4*>(a.dst[0] + doff[u]) = kv[u][0];
      *reinterpret_cast<uint4*>(a.dst[1] + doff[u]) = kv[u][1];
    }
  }
}

cudaError_t launch_block_move(const BlockMoveArgs& a, int sm_count, cudaStream_t stream) {
  if (a.n <= 0) return cudaSuccess;
  const long long total = (long long)a.n * (a.block_bytes / 16);
  long long blocks = (total + (long long)kMoveThreads * kMoveUnroll - 1) / ((long long)kMoveThreads * kMoveUnroll);
  const long long cap = (long long)sm_count * 8;
  if (blocks > cap) blocks = cap;
  if (blocks < 1) blocks = 1;
  if (a.scale_bytes > 0)
    block_move_kernel<true><<<(unsigned)blocks, kMoveThreads, 0, stream>>>(a);
  else
    block_move_kernel<false><<<(unsigned)blocks, kMoveThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// Self-test of the bounded wait every kernel of the library uses: one thread waits on an
// mbarrier phase that nothing completes; after limit_ns it gives up, records the timeout in
// the error word and returns, leaving the context usable.
__global__ void wait_selftest_kernel(uint32_t* err, uint64_t limit_ns, uint64_t* waited_ns) {
  __shared__ __align__(8) uint64_t bar;
  const uint32_t b = smem_u32(&bar);
  mbar_init(b, 1);
  fence_barrier_init();
  const uint64_t t0 = globaltimer_ns();
  if (!mbar_wait_for(b, 0, limit_ns)) report(err, kErrTimeout);
  if (waited_ns != nullptr) *waited_ns = globaltimer_ns() - t0;
}

cudaError_t launch_wait_selftest(uint32_t* err, uint64_t limit_ns, uint64_t* waited_ns,
                                 cudaStream_t stream) {
  wait_selftest_kernel<<<1, 1, 0, stream>>>(err, limit_ns, waited_ns);
  return cudaGetLastError();
}

}  // namespace cb

// The quantising KV-append and the read-back of a quantised cache (the arithmetic: cb_quant.cuh).
#include "cb_quant.cuh"

namespace cb {

constexpr int kQuantThreads = 128;
constexpr int kQuantUnroll = 4;

__global__ void __launch_bounds__(kQuantThreads) quant_append_kernel(const QuantAppendArgs x) {
  // Launched as a programmatic dependent of whatever precedes it, and lets such a launch behind it
  // start early.
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  check_cu_seqlens(x.r.ap);
  quant_tokens<kQuantUnroll>(x, (long long)blockIdx.x * (kQuantThreads / 32) + (threadIdx.x >> 5),
                             (long long)gridDim.x * (kQuantThreads / 32));
}

// Warps per token, as for the rotary append.
int quant_parts(const RopeArgs& r, int sm_count) {
  const int per_warp = 32 / (r.ap.D / 16);
  const int heads = (r.q != nullptr ? r.Hq : 0) + 2 * r.ap.Hkv;
  const int groups = (heads + per_warp - 1) / per_warp;
  const long long want = ((long long)sm_count * 8 + r.ap.T - 1) / r.ap.T;
  return (int)(want < groups ? want : groups);
}

cudaError_t launch_quant_append(QuantAppendArgs x, int sm_count, cudaStream_t stream) {
  if (x.r.ap.T == 0) return cudaSuccess;
  x.r.parts = quant_parts(x.r, sm_count);
  const int warps = kQuantThreads / 32;
  long long blocks = ((long long)x.r.ap.T * x.r.parts + warps - 1) / warps;
  if (blocks > (long long)sm_count * 64) blocks = (long long)sm_count * 64;
  return launch_dependent(quant_append_kernel, (unsigned)blocks, kQuantThreads, 0, stream, x);
}

constexpr int kGatherThreads = 128;
constexpr int kGatherUnroll = 4;

__global__ void __launch_bounds__(kGatherThreads) quant_gather_kernel(const GatherArgs g) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = blockIdx.x * kGatherThreads + threadIdx.x; i < g.S; i += gridDim.x * kGatherThreads) {
    const int c0 = __ldg(g.cu_seqlens_k + i), c1 = __ldg(g.cu_seqlens_k + i + 1);
    if (c1 < c0 || (i == 0 && c0 != 0) || (i == g.S - 1 && c1 > g.T)) report(g.err, kErrOutOfRange);
  }
  gather_rows<kGatherUnroll>(g, (long long)blockIdx.x * (kGatherThreads / 32) + (threadIdx.x >> 5));
}

cudaError_t launch_quant_gather(GatherArgs g, int sm_count, cudaStream_t stream) {
  if (g.T == 0) return cudaSuccess;
  // Rows per warp: as many as leave 32 warps to every SM (one row each for small ranges), and as make 512
  // pieces of 8 values: more leave the last wave of warps long (95859 rows of 8 heads of 128: 32 rows 97
  // us, 8 rows 95, 4 rows 89, 2 rows 89), and fewer search the metadata more often.
  const int per_row = g.Hkv * g.D / 8;
  g.rows = 1;
  while (g.rows < 32 && (long long)g.rows * 2 * sm_count * 32 <= g.T && g.rows * 2 * per_row <= 512)
    g.rows *= 2;
  const int per_block = kGatherThreads / 32 * g.rows;
  const unsigned blocks = (unsigned)(((long long)g.T + per_block - 1) / per_block);
  return launch_dependent(quant_gather_kernel, blocks, kGatherThreads, 0, stream, g);
}

}  // namespace cb

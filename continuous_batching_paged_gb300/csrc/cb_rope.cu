// The rotary KV-append as a launch of its own (the arithmetic and the lane layout: cb_rope.cuh).
#include "cb_rope.cuh"

namespace cb {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;  // head groups in flight: 8 16-byte loads per lane

__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs r) {
  check_cu_seqlens(r.ap);
  rope_tokens<kRopeUnroll>(r, (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5),
                           (long long)gridDim.x * (kRopeThreads / 32));
}

cudaError_t launch_rope_append(RopeArgs r, int sm_count, cudaStream_t stream) {
  const AppendArgs& a = r.ap;
  if (a.T == 0) return cudaSuccess;
  const int per_warp = 32 / (a.D / 16);
  const int heads = (r.q != nullptr ? r.Hq : 0) + 2 * a.Hkv;
  const int groups = (heads + per_warp - 1) / per_warp;
  // Warps per token: enough that the step's warps fill the SMs (32 warps each).
  const long long want = ((long long)sm_count * 32 + a.T - 1) / a.T;
  r.parts = (int)(want < groups ? want : groups);
  const int warps = kRopeThreads / 32;
  long long blocks = ((long long)a.T * r.parts + warps - 1) / warps;
  if (blocks > (long long)sm_count * 64) blocks = (long long)sm_count * 64;
  rope_append_kernel<<<(unsigned)blocks, kRopeThreads, 0, stream>>>(r);
  return cudaGetLastError();
}

}  // namespace cb

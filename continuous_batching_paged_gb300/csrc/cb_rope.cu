// The rotary KV-append as a launch of its own, and with the attention planner beside it (the
// arithmetic and the lane layout: cb_rope.cuh).
#include "cb_plan.cuh"
#include "cb_rope.cuh"

namespace cb {

// Blocks of 4 warps and 4 head groups in flight (8 16-byte loads per lane, 96 registers): blocks of 8
// leave a quarter of the registers unused and were slower at every size (8208 tokens of 64 heads 59
// us, now 52 us, 6.07 TB/s; 2048 tokens of 32 heads 13.7 us, now 11.5 us), 2 or 6 groups too.
constexpr int kRopeThreads = 128;
constexpr int kRopeUnroll = 4;

__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs r) {
  // Launched as a programmatic dependent of whatever precedes it on the stream, and lets such a
  // launch behind it start early: the launch latency of calls in a row overlaps.
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  check_cu_seqlens(r.ap);
  rope_tokens<kRopeUnroll>(r, (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5),
                           (long long)gridDim.x * (kRopeThreads / 32));
}

// Warps per token: enough that every SM has 8 (one token a warp from 1216 tokens on), at most one per
// group of heads.  With few tokens the loads' latency counts, with many every further warp on a token
// looks its slot up once more (256 decodes: 3.9 us with 5 warps a token, 5.6 with 12, 6.4 with 1).
static int rope_parts(const RopeArgs& r, int sm_count) {
  const int per_warp = 32 / (r.ap.D / 16);
  const int heads = (r.q != nullptr ? r.Hq : 0) + 2 * r.ap.Hkv;
  const int groups = (heads + per_warp - 1) / per_warp;
  const long long want = ((long long)sm_count * 8 + r.ap.T - 1) / r.ap.T;
  return (int)(want < groups ? want : groups);
}

cudaError_t launch_rope_append(RopeArgs r, int sm_count, cudaStream_t stream) {
  if (r.ap.T == 0) return cudaSuccess;
  r.parts = rope_parts(r, sm_count);
  const int warps = kRopeThreads / 32;
  long long blocks = ((long long)r.ap.T * r.parts + warps - 1) / warps;
  if (blocks > (long long)sm_count * 64) blocks = (long long)sm_count * 64;
  return launch_dependent(rope_append_kernel, (unsigned)blocks, kRopeThreads, 0, stream, r);
}

// CTA 0 plans the attention pass (it reads only the metadata); CTAs 1.. rotate and append.
template <bool kPre>
__global__ void __launch_bounds__(plan_threads<kPre>(), 1) rope_plan_kernel(const RopeArgs r,
                                                                            AttnArgs a) {
  allow_dependent_launch();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0) {
    plan_cta<kPre>(a);
  } else {
    constexpr int kWarps = plan_threads<kPre>() / 32;
    constexpr int kUnroll = kPre ? kRopeUnroll : 2;  // (2 fits the 64 registers of 1024 threads)
    rope_tokens<kUnroll>(r, (long long)(blockIdx.x - 1) * kWarps + (threadIdx.x >> 5),
                         (long long)(gridDim.x - 1) * kWarps);
  }
}

template <bool kPre>
static cudaError_t launch_rope_plan_t(const RopeArgs& r, const AttnArgs& a, int sm_count,
                                      cudaStream_t stream) {
  constexpr int kWarps = plan_threads<kPre>() / 32;
  long long blocks = ((long long)r.ap.T * r.parts + kWarps - 1) / kWarps;
  const long long most = (long long)sm_count * 512 / kWarps;
  if (blocks > most) blocks = most;
  return launch_dependent(rope_plan_kernel<kPre>, (unsigned)(1 + blocks), kWarps * 32, 0, stream, r, a);
}

cudaError_t launch_rope_plan(RopeArgs r, const AttnArgs& a, int sm_count, cudaStream_t stream) {
  r.parts = rope_parts(r, sm_count);
  return a.NG > 0 ? launch_rope_plan_t<true>(r, a, sm_count, stream)
                  : launch_rope_plan_t<false>(r, a, sm_count, stream);
}

}  // namespace cb

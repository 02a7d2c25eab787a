// Paged KV-append: scatter this step's K/V rows into their cache slots, and the batch planner
// of the attention pass.
//
// Slot rule ("LLM learning path 3.3 Batching & Memory Management", section "PagedAttention:
// block tables"): token position p of a sequence lives in physical block table[p / bs] at
// offset p % bs; with the token-major pool of "Continuous batching in transformers"
// (paged-cache section) that is row table[p / bs] * bs + p % bs of the flattened
// [P * bs, Hkv, D] tensor.  Token i of sequence s has position kv_len_s - q_len_s + i.
#include "cb_append.cuh"
#include "cb_plan.cuh"

namespace cb {

__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(AppendArgs a) {
  check_cu_seqlens(a);
  append_tokens<kAppendMaxChunks>(a, blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5),
                                  gridDim.x * (kAppendThreads / 32));
}

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const int warps = kAppendThreads / 32;
  long long blocks = ((long long)a.T + warps - 1) / warps;
  if (blocks > 8192) blocks = 8192;
  kv_append_kernel<<<(unsigned)blocks, kAppendThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(AttnArgs a) {
  allow_dependent_launch();
  plan_cta<false>(a);
}

cudaError_t launch_plan(const AttnArgs& a, cudaStream_t stream) {
  plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// CTA 0 plans the attention pass (it reads only the metadata); CTAs 1.. append this step's
// K/V rows, one warp per token, 32 tokens per CTA at a time.
constexpr int kAppendPlanMaxChunks = 4;  // fits the 64 registers of a 1024-thread CTA
__global__ void __launch_bounds__(kPlanThreads, 1) append_plan_kernel(AppendArgs ap, AttnArgs a) {
  allow_dependent_launch();
  if (blockIdx.x == 0) {
    plan_cta<false>(a);
  } else {
    constexpr int kWarps = kPlanThreads / 32;
    append_tokens<kAppendPlanMaxChunks>(ap, (blockIdx.x - 1) * kWarps + (threadIdx.x >> 5),
                                        (gridDim.x - 1) * kWarps);
  }
}

cudaError_t launch_append_plan(const AppendArgs& ap, const AttnArgs& a, cudaStream_t stream) {
  constexpr int kWarps = kPlanThreads / 32;
  long long blocks = ((long long)ap.T + kWarps - 1) / kWarps;
  if (blocks > 2048) blocks = 2048;
  if (blocks < 1) blocks = 1;
  append_plan_kernel<<<(unsigned)(1 + blocks), kPlanThreads, 0, stream>>>(ap, a);
  return cudaGetLastError();
}

}  // namespace cb

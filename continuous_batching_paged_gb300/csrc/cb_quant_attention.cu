// Attention over the quantised cache (cb_quant_attention.cuh): its planner, alone and beside the
// quantising append, and the kernels without changed scores.
#include "cb_plan.cuh"
#include "cb_quant_attention.cuh"

namespace cb {

__global__ void __launch_bounds__(kPlanThreads, 1) quant_plan_kernel(AttnArgs a, int tile_log2) {
  allow_dependent_launch();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the workspace may still be in use)
  plan_cta<false, true>(a, tile_log2);
}

cudaError_t launch_quant_plan(const AttnArgs& a, const QuantArgs& qa, cudaStream_t stream) {
  return launch_dependent(quant_plan_kernel, 1, kPlanThreads, 0, stream, a, qa.tile_log2);
}

// CTA 0 plans the attention pass (it reads only the metadata); CTAs 1.. quantise and append.
constexpr int kQuantPlanUnroll = 1;  // (what the 64 registers of a 1024-thread CTA hold)
__global__ void __launch_bounds__(kPlanThreads, 1)
    quant_append_plan_kernel(const QuantAppendArgs x, AttnArgs a, int tile_log2) {
  allow_dependent_launch();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blockIdx.x == 0) {
    plan_cta<false, true>(a, tile_log2);
  } else {
    constexpr int kWarps = kPlanThreads / 32;
    quant_tokens<kQuantPlanUnroll>(x, (long long)(blockIdx.x - 1) * kWarps + (threadIdx.x >> 5),
                                   (long long)(gridDim.x - 1) * kWarps);
  }
}

cudaError_t launch_quant_append_plan(QuantAppendArgs x, const AttnArgs& a, const QuantArgs& qa,
                                     int sm_count, cudaStream_t stream) {
  x.r.parts = quant_parts(x.r, sm_count);
  constexpr int kWarps = kPlanThreads / 32;
  long long blocks = ((long long)x.r.ap.T * x.r.parts + kWarps - 1) / kWarps;
  const long long most = (long long)sm_count * 512 / kWarps;
  if (blocks > most) blocks = most;
  return launch_dependent(quant_append_plan_kernel, (unsigned)(1 + blocks), kPlanThreads, 0, stream, x,
                          a, qa.tile_log2);
}

cudaError_t launch_quant_attention(const AttnArgs& a, const QuantArgs& qa, const ScoreArgs* sc,
                                   const QuantMaps& m, cudaStream_t stream) {
  if (a.decode_grid + a.prefill_ctas == 0) return cudaSuccess;
  if (sc != nullptr) return launch_quant_scored(a, qa, *sc, m, stream);
  const ScoreArgs none = {};
  return a.D == 128 ? launch_quant_heads<128, false>(a, qa, none, m, stream)
                    : launch_quant_heads<64, false>(a, qa, none, m, stream);
}

}  // namespace cb

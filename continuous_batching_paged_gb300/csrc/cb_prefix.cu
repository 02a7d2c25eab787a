// Attention over batches whose sequences share prefixes: each group's prefix is computed once for
// all its query rows, every other key by the sequence it belongs to.
//
//   out = sum_c w_c o_c / sum_c w_c l_c over the parts c of a row's keys (w_c = 2^(m_c - max m)):
// the parts of the prefix, and the parts of the sequence's own keys.  The softmax over all keys is
// the same sum in another order, so a row's result is that of cb_ragged_paged_attention within
// rounding.
//
// Own keys are streamed by the decode pass (cb_decode.cuh), as ever, from the prefix's end on; a
// member with up to kPreMaxQ query tokens has one record per token.  The prefix is a dense
// contraction (all rows of the group see all its keys), so it runs on the 5th-generation tensor
// cores, in the chunk pass (cb_prefill.cuh): tiles of 128 rows = 128 / G query tokens with the G
// heads of one KV head, gathered by TMA, two tiles per work item against the same K/V tiles, no
// mask but the prefix's end, O and (m, l) left unnormalised in fp32.  K/V of the prefix are read
// once per 2 x 128 rows (by L2 at most once from HBM) instead of once per query token, which is
// what bounds the batch otherwise.  Both kinds of parts count up one counter per (record, KV head,
// 8 query heads); whoever counts last merges, so the two passes run side by side in one launch and
// no part waits for another.
#include "cb_attention.cuh"
#include "cb_plan.cuh"

namespace cb {

__global__ void __launch_bounds__(kPlanThreads, 1) prefix_plan_kernel(AttnArgs a) {
  allow_dependent_launch();
  plan_cta<true>(a);
}

cudaError_t launch_prefix_plan(const AttnArgs& a, cudaStream_t stream) {
  prefix_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, int QS>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prefix_attention_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap qmap_tok,
                            const __grid_constant__ CUtensorMap kmap_dec,
                            const __grid_constant__ CUtensorMap vmap_dec,
                            const __grid_constant__ CUtensorMap kmap_chunk,
                            const __grid_constant__ CUtensorMap vmap_chunk) {
  extern __shared__ uint8_t smem_raw[];
  attention_cta<D, QS, false, true>(a, &qmap, &qmap_tok, &kmap_dec, &vmap_dec, &kmap_chunk,
                                    &vmap_chunk, smem_raw);
}

template <int D, int QS>
static cudaError_t launch_instance(const AttnArgs& a, const AttnMaps& m, const CUtensorMap& q_tok,
                                   cudaStream_t stream) {
  constexpr int kSmem = AttnSmem<D, QS>::kTotal;
  // a setting of the context, as for the attention kernel without prefixes
  static unsigned long long configured_ctx = 0;
  const unsigned long long ctx = launch_context_id();
  if (ctx == 0 || configured_ctx != ctx) {
    const cudaError_t e = cudaFuncSetAttribute(
        prefix_attention_kernel<D, QS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured_ctx = ctx;
  }
  // may start before the planner ends, and waits for it (griddepcontrol.wait)
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.decode_grid + a.prefill_ctas);
  cfg.blockDim = dim3(kAttnThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_attention_kernel<D, QS>, a, m.q, q_tok, m.k_dec, m.v_dec,
                            m.k_chunk, m.v_chunk);
}

cudaError_t launch_prefix_attention(const AttnArgs& a, const AttnMaps& m, const CUtensorMap& q_tok,
                                    cudaStream_t stream) {
  if (a.D == 128)
    return a.G <= 8 ? launch_instance<128, 1>(a, m, q_tok, stream)
                    : launch_instance<128, 2>(a, m, q_tok, stream);
  return a.G <= 8 ? launch_instance<64, 1>(a, m, q_tok, stream)
                  : launch_instance<64, 2>(a, m, q_tok, stream);
}

}  // namespace cb

// Attention with changed scores and masks (cb_score.cuh) on the bf16 cache: the attention kernel's two
// passes (cb_attention.cu) with the change between the product and the softmax.
#include "cb_attention.cuh"

namespace cb {

template <int D, int QS>
__global__ void __launch_bounds__(kAttnThreads, 1)
    scored_attention_kernel(const AttnArgs a, const ScoreArgs sc,
                            const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap kmap_dec,
                            const __grid_constant__ CUtensorMap vmap_dec,
                            const __grid_constant__ CUtensorMap kmap_chunk,
                            const __grid_constant__ CUtensorMap vmap_chunk) {
  extern __shared__ uint8_t smem_raw[];
  attention_cta<D, QS, true, false, true>(a, &qmap, nullptr, nullptr, &kmap_dec, &vmap_dec,
                                          &kmap_chunk, &vmap_chunk, smem_raw, sc);
}

template <int D, int QS>
static cudaError_t launch_instance(const AttnArgs& a, const ScoreArgs& sc, const AttnMaps& m,
                                   cudaStream_t stream) {
  constexpr int kSmem = AttnSmem<D, QS, false>::kTotal;
  // a setting of the context, as for the attention kernel
  static unsigned long long configured_ctx = 0;
  const unsigned long long ctx = launch_context_id();
  if (ctx == 0 || configured_ctx != ctx) {
    const cudaError_t e = cudaFuncSetAttribute(
        scored_attention_kernel<D, QS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured_ctx = ctx;
  }
  return launch_dependent(scored_attention_kernel<D, QS>, (unsigned)launch_ctas(a),
                          kAttnThreads, kSmem, stream, a, sc, m.q, m.k_dec, m.v_dec, m.k_chunk,
                          m.v_chunk);
}

cudaError_t launch_scored_attention(const AttnArgs& a, const ScoreArgs& sc, const AttnMaps& maps,
                                    cudaStream_t stream) {
  if (a.decode_grid + a.prefill_ctas == 0) return cudaSuccess;
  if (a.D == 128)
    return a.G <= 8 ? launch_instance<128, 1>(a, sc, maps, stream)
                    : launch_instance<128, 2>(a, sc, maps, stream);
  return a.G <= 8 ? launch_instance<64, 1>(a, sc, maps, stream)
                  : launch_instance<64, 2>(a, sc, maps, stream);
}

}  // namespace cb

// Attention over the quantised cache with changed scores, masks or a sliding window.
#include "cb_quant_attention.cuh"

namespace cb {

cudaError_t launch_quant_scored(const AttnArgs& a, const QuantArgs& qa, const ScoreArgs& sc,
                                const QuantMaps& m, cudaStream_t stream) {
  return a.D == 128 ? launch_quant_heads<128, true>(a, qa, sc, m, stream)
                    : launch_quant_heads<64, true>(a, qa, sc, m, stream);
}

}  // namespace cb

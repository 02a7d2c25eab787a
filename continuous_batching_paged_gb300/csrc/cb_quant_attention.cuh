// The attention kernel over the quantised cache: the decode pass (cb_quant_decode.cuh) and the chunk
// pass (cb_prefill.cuh, cb_quant_prefill.cuh) in one launch.  Its first a.decode_grid CTAs take the decode
// ranges, and every CTA then takes chunk items while there are any: an SM that the planner leaves to the
// chunk pass begins with it at once, and one whose range is done goes on without another CTA's launch
// (beside CTAs that only leave their SM: 64 decodes on up to 4000 keys 63 us, so 62; those and a chunk
// 148 us, so 144).
#pragma once

#include "cb_quant_decode.cuh"
#include "cb_quant_prefill.cuh"

namespace cb {

template <int D, int QS>
constexpr int quant_attention_smem() {
  return QDecodeSmem<D, QS>::kTotal > QuantPrefillSmem<D>::kTotal ? QDecodeSmem<D, QS>::kTotal
                                                                  : QuantPrefillSmem<D>::kTotal;
}

// kMod: with changed scores, masks or a sliding window.
template <int D, int QS, bool kMod>
__global__ void __launch_bounds__(kQuantPrefillThreads, 1)
    quant_attention_kernel(const AttnArgs a, const QuantArgs qa, const ScoreArgs sc,
                           const __grid_constant__ CUtensorMap qmap,
                           const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ uint8_t smem_raw[];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = (int)blockIdx.x;
  if (b < a.decode_grid) {
    PlanHeader* hdr = reinterpret_cast<PlanHeader*>(a.ws + ws_layout(a.R, a.T, a.Hq, a.D, a.pack).header);
    const bool busy = hdr->dec_tiles > 0;
    if (threadIdx.x == 0 && busy) atomicMin(&hdr->t_dec_start, global_ns());
    quant_decode_cta<D, QS, kMod>(a, qa, sc, &kmap, &vmap, smem_raw, b);
    if ((threadIdx.x & 31) == 0 && busy) atomicMax(&hdr->t_dec_end, global_ns());
    if (a.prefill_ctas == 0 || hdr->pf_qtiles == 0) return;
    fence_proxy_async_smem();  // (the chunk pass's copies into what the decode role wrote)
    __syncthreads();
  }
  prefill_cta<D, kMod, kMod, true>(a, &qmap, nullptr, nullptr, smem_raw, sc, qa);
}

template <int D, int QS, bool kMod>
static cudaError_t launch_quant_instance(const AttnArgs& a, const QuantArgs& qa, const ScoreArgs& sc,
                                         const QuantMaps& m, cudaStream_t stream) {
  constexpr int kSmem = quant_attention_smem<D, QS>();
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  // a setting of the context, as for the attention kernel
  static unsigned long long configured_ctx = 0;
  const unsigned long long ctx = launch_context_id();
  if (ctx == 0 || configured_ctx != ctx) {
    const cudaError_t e = cudaFuncSetAttribute(
        quant_attention_kernel<D, QS, kMod>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    // both passes hand registers from one warpgroup to another (setmaxnreg), which waits for ever where
    // the launch brings fewer than their split
    cudaFuncAttributes f;
    const cudaError_t g = cudaFuncGetAttributes(&f, quant_attention_kernel<D, QS, kMod>);
    if (g != cudaSuccess) return g;
    if (f.numRegs < 121) return cudaErrorInvalidConfiguration;  // (allocated in eights: 128)
    configured_ctx = ctx;
  }
  return launch_dependent(quant_attention_kernel<D, QS, kMod>, (unsigned)launch_ctas(a),
                          kQuantPrefillThreads, kSmem, stream, a, qa, sc, m.q, m.k, m.v);
}

template <int D, bool kMod>
static cudaError_t launch_quant_heads(const AttnArgs& a, const QuantArgs& qa, const ScoreArgs& sc,
                                      const QuantMaps& m, cudaStream_t stream) {
  return a.G <= 8 ? launch_quant_instance<D, 1, kMod>(a, qa, sc, m, stream)
                  : launch_quant_instance<D, 2, kMod>(a, qa, sc, m, stream);
}

}  // namespace cb

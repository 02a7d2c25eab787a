// One CTA of an attention kernel: a decode-role CTA, with shared prefixes a prefix-role CTA, or a
// chunk-role CTA, by its index in the grid (cb_attention.cu says how they share the GPU).
#pragma once

#include "cb_decode.cuh"
#include "cb_prefill.cuh"
#include "cb_prefix.cuh"

namespace cb {

constexpr int kAttnThreads = kPrefillThreads;
static_assert(32 * (kMaxDecodeHeadsPerCta + 1) <= kAttnThreads,
              "the decode role fits in the chunk role's CTA");

template <int D, int QS, bool kPre>
struct AttnSmem {
  static constexpr int kBoth = DecodeSmem<D, QS>::kTotal > PrefillSmem<D>::kTotal
                                   ? DecodeSmem<D, QS>::kTotal
                                   : PrefillSmem<D>::kTotal;
  static constexpr int kTotal = kPre && PreSmem<D>::kTotal > kBoth ? PreSmem<D>::kTotal : kBoth;
};

// kPre: the batch's shared prefixes are computed once per group (cb_prefix.cu); qmap_tok and
// qmap_run are the tensor maps of a group's query rows, token by token and a tile of tokens (unused
// otherwise).
template <int D, int QS, bool kWin, bool kPre>
__device__ __forceinline__ void attention_cta(const AttnArgs& a, const CUtensorMap* qmap,
                                              const CUtensorMap* qmap_tok,
                                              const CUtensorMap* qmap_run,
                                              const CUtensorMap* kmap_dec,
                                              const CUtensorMap* vmap_dec,
                                              const CUtensorMap* kmap_chunk,
                                              const CUtensorMap* vmap_chunk, uint8_t* smem_raw) {
  // Launched as a programmatic dependent of the planner: CTAs may start while the planner's
  // launch still runs; everything below reads the plan (and the appended K/V), so wait here
  // for that launch to complete and its writes to be visible.  A no-op without the attribute.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the merge of the prefixes' parts may start once every CTA of this kernel has (it waits itself)
  if constexpr (kPre) asm volatile("griddepcontrol.launch_dependents;");
  const int b = (int)blockIdx.x;
  PlanHeader* hdr = reinterpret_cast<PlanHeader*>(a.ws + ws_layout(a.R, a.T, a.Hq, a.D, a.pack).header);
  if constexpr (kPre) {
    // The decode CTAs that the planner leaves without work are the first prefix CTAs; where those
    // are too few, some of the chunk CTAs are the others.
    const int N = hdr->decode_ctas;
    const int c = b < a.decode_grid
                      ? pre_idle_index(b % a.decode_ctas, b / a.decode_ctas, N, a.decode_ctas)
                      : pre_idle_count(pre_head_groups(a.Hkv, a.G), N, a.decode_ctas) + b -
                            a.decode_grid;
    if (c >= 0 && c < hdr->pre_ctas) {
      prefix_cta<D>(a, qmap_tok, qmap_run, kmap_chunk, vmap_chunk, smem_raw, c);
      return;
    }
  }
  if (b < a.decode_grid) {
    // Span of the decode role: first start and last end of any warp of a CTA with work (the
    // chunk role stamps its own span inside prefill_cta).
    const bool busy = hdr->dec_tiles > 0;
    if (threadIdx.x == 0 && busy) atomicMin(&hdr->t_dec_start, global_ns());
    decode_cta<D, QS, kPre>(a, kmap_dec, vmap_dec, smem_raw, b % a.decode_ctas, b / a.decode_ctas);
    if ((threadIdx.x & 31) == 0 && busy) atomicMax(&hdr->t_dec_end, global_ns());
    return;
  }
  prefill_cta<D, kWin>(a, qmap, kmap_chunk, vmap_chunk, smem_raw);
}

}  // namespace cb

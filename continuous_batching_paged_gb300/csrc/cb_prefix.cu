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
// what bounds the batch otherwise.  The two passes run side by side in one launch, no part waits
// for another, and a last small launch merges the parts, a warp per (token, query head).  (Merged by
// whoever counted last, as the decode pass merges its own splits, the prefix's few warps merged
// a tile's tokens one after the other: 64 sequences sharing 1024 keys took 96 us.)
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

// One warp per (query token, query head) of the shared prefixes: M = max m_c, w_c = 2^(m_c - M),
// out = sum_c w_c o_c / sum_c w_c l_c, lse = (M + log2 sum_c w_c l_c) ln 2 over the prefix's parts,
// then the parts of the own keys that decode CTAs cf .. cl left.  Every part holds at least one
// key, so its m is finite.  Bound by the latency of its loads: kC parts at a time, all loaded
// before any is used.
constexpr int kMergeThreads = 256;
template <int D>
__global__ void __launch_bounds__(kMergeThreads) prefix_merge_kernel(const AttnArgs a) {
  constexpr int PER = D / 32, kC = 4;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const WsLayout L = ws_layout(a.R, a.T, a.Hq, a.D);
  const PreLayout PL = pre_layout(a.R, a.T, a.Hq, a.Hkv, a.D, a.NG);
  const PlanHeader* hdr = reinterpret_cast<const PlanHeader*>(a.ws + L.header);
  const int2* pre_tok = reinterpret_cast<const int2*>(a.ws + PL.tok);
  const int4* pre_rec = reinterpret_cast<const int4*>(a.ws + PL.rec);
  const int4* dec_rec = reinterpret_cast<const int4*>(a.ws + L.dec_rec);
  const float2* pre_ml = reinterpret_cast<const float2*>(a.ws + PL.part_ml);
  const float* pre_o = reinterpret_cast<const float*>(a.ws + PL.part_o);
  const float2* own_ml = reinterpret_cast<const float2*>(a.ws + L.part_ml);
  const float* own_o = reinterpret_cast<const float*>(a.ws + L.part_o);
  __nv_bfloat16* outg = static_cast<__nv_bfloat16*>(a.out);
  const long long rows = (long long)hdr->pre_tokens * a.Hq;
  const long long ntiles = hdr->dec_tiles;
  const int N = hdr->decode_ctas;
  for (long long row = (long long)blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5); row < rows;
       row += (long long)gridDim.x * (kMergeThreads / 32)) {
    const int i = (int)(row / a.Hq), head = (int)(row - (long long)i * a.Hq);
    const int2 tr = pre_tok[i];
    const int4 rec = pre_rec[tr.y];  // prefix length, first slot, slots between parts, parts
    const int cf = cta_of_tile(dec_rec[tr.y].w, ntiles, N);
    const int cl = cta_of_tile(dec_rec[tr.y + 1].w - 1, ntiles, N);
    const int nparts = rec.w + cl - cf + 1;
    float M = -INFINITY, l = 0.f, acc[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = 0.f;
    for (int c0 = 0; c0 < nparts; c0 += kC) {
      float2 ml[kC];
      float v[kC][PER];
#pragma unroll
      for (int cc = 0; cc < kC; ++cc) {
        const int c = c0 + cc;
        ml[cc] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int k = 0; k < PER; ++k) v[cc][k] = 0.f;
        if (c < nparts) {
          const bool pre = c < rec.w;
          const size_t at = (pre ? (size_t)rec.y + (size_t)c * rec.z
                                 : (size_t)(cf + c - rec.w) + tr.y) * a.Hq + head;
          ml[cc] = (pre ? pre_ml : own_ml)[at];
          const float* po = (pre ? pre_o : own_o) + at * D + lane * PER;
          if constexpr (PER == 4) {
            const float4 x = *reinterpret_cast<const float4*>(po);
            v[cc][0] = x.x; v[cc][1] = x.y; v[cc][2] = x.z; v[cc][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(po);
            v[cc][0] = x.x; v[cc][1] = x.y;
          }
        }
      }
      float mn = M;
#pragma unroll
      for (int cc = 0; cc < kC; ++cc) mn = fmaxf(mn, ml[cc].x);
      const float sc = fast_exp2(M - mn);
      l *= sc;
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[k] *= sc;
#pragma unroll
      for (int cc = 0; cc < kC; ++cc) {
        const float w = fast_exp2(ml[cc].x - mn);  // 0 past the last part
        l += w * ml[cc].y;
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[k] += w * v[cc][k];
      }
      M = mn;
    }
    const float inv = 1.f / l;
    uint32_t* dst = reinterpret_cast<uint32_t*>(outg + ((size_t)tr.x * a.Hq + head) * D + lane * PER);
    if constexpr (PER == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                  pack_bf16x2(acc[2] * inv, acc[3] * inv));
    else
      dst[0] = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    if (lane == 0 && a.lse != nullptr)
      a.lse[(size_t)tr.x * a.Hq + head] = (M + __log2f(l)) * 0.6931471805599453f;
  }
}

cudaError_t launch_prefix_merge(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  const long long warps = (long long)a.R * a.Hq;
  long long blocks = (warps + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
  if (blocks > (long long)sm_count * 8) blocks = (long long)sm_count * 8;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.D == 128 ? cudaLaunchKernelEx(&cfg, prefix_merge_kernel<128>, a)
                    : cudaLaunchKernelEx(&cfg, prefix_merge_kernel<64>, a);
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

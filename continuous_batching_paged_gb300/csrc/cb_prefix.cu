// Attention over batches whose sequences share prefixes: each group's prefix is computed once for
// all its query rows, every other key by the sequence it belongs to.
//
//   out = sum_c w_c o_c / sum_c w_c l_c over the parts c of a row's keys (w_c = 2^(m_c - max m)):
// the parts of the prefix, and the parts of the sequence's own keys.  The softmax over all keys is
// the same sum in another order, so a row's result is that of cb_ragged_paged_attention within
// rounding.
//
// Own keys are streamed by the decode pass (cb_decode.cuh), as ever, from the prefix's end on (or,
// for several query tokens, are a group of their own: PreGroup).  The prefix is a dense
// contraction (all rows of the group see all its keys) and runs on the 5th-generation tensor cores
// (cb_prefix.cuh): its K/V are read once per 2 x 128 rows (from HBM at most once) instead of once
// per query token, which is what bounds the batch otherwise.  The passes run side by side in one
// launch, each on the SMs that the planner gives it, no part of either waits for another, and a
// last small launch merges the parts, a warp per (token, query head) or four heads.  (Merged by whoever counted
// last, as the decode pass merges its own splits, a tile's tokens were merged one after the other
// by the few warps that finished last: 64 sequences sharing 1024 keys took 96 us, now 45.)
#include "cb_attention.cuh"
#include "cb_plan.cuh"

namespace cb {

__global__ void __launch_bounds__(kPrePlanThreads, 1) prefix_plan_kernel(AttnArgs a) {
  allow_dependent_launch();
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (the workspace may still be in use)
  plan_cta<true>(a);
}

cudaError_t launch_prefix_plan(const AttnArgs& a, cudaStream_t stream) {
  return launch_dependent(prefix_plan_kernel, 1, kPrePlanThreads, 0, stream, a);
}

template <int D, int QS>
__global__ void __launch_bounds__(kAttnThreads, 1)
    prefix_attention_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap qmap,
                            const __grid_constant__ CUtensorMap qmap_tok,
                            const __grid_constant__ CUtensorMap qmap_run,
                            const __grid_constant__ CUtensorMap kmap_dec,
                            const __grid_constant__ CUtensorMap vmap_dec,
                            const __grid_constant__ CUtensorMap kmap_chunk,
                            const __grid_constant__ CUtensorMap vmap_chunk) {
  extern __shared__ uint8_t smem_raw[];
  attention_cta<D, QS, false, true>(a, &qmap, &qmap_tok, &qmap_run, &kmap_dec, &vmap_dec,
                                    &kmap_chunk, &vmap_chunk, smem_raw);
}

template <int D, int QS>
static cudaError_t launch_instance(const AttnArgs& a, const AttnMaps& m, const PrefixMaps& p,
                                   cudaStream_t stream) {
  constexpr int kSmem = AttnSmem<D, QS, true>::kTotal;
  // a setting of the context, as for the attention kernel without prefixes
  static unsigned long long configured_ctx = 0;
  const unsigned long long ctx = launch_context_id();
  if (ctx == 0 || configured_ctx != ctx) {
    const cudaError_t e = cudaFuncSetAttribute(
        prefix_attention_kernel<D, QS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    configured_ctx = ctx;
  }
  return launch_dependent(prefix_attention_kernel<D, QS>, a.decode_grid + a.prefill_ctas, kAttnThreads,
                          kSmem, stream, a, m.q, p.q_tok, p.q_run, m.k_dec, m.v_dec, m.k_chunk,
                          m.v_chunk);
}

// One warp per (query token, HP query heads of one KV head) of the shared prefixes:
// M = max m_c, w_c = 2^(m_c - M), out = sum_c w_c o_c / sum_c w_c l_c,
// lse = (M + log2 sum_c w_c l_c) ln 2 over the parts c of its chains and of its decode record.  Some
// part holds a key that the token sees, so M is finite (a part without one has m = -inf, w = 0).  A lane
// finds a part and loads its (m, l), so all are there after one trip to L2, and the rows of O follow kC
// at a time.  Finding the parts is what costs instructions, so with many rows a warp does HP = 4 heads;
// with few, where only the latency of its loads counts, one (launch_prefix_merge).
constexpr int kMergeThreads = 256;
template <int D, int HP, int kC>
__global__ void __launch_bounds__(kMergeThreads, HP * kC > 16 ? 1 : 2)
    prefix_merge_kernel(const AttnArgs a) {
  constexpr int PER = D / 32;  // columns per lane
  allow_dependent_launch();
  const int lane = threadIdx.x & 31;
  const WsLayout L = ws_layout(a.R, a.T, a.Hq, a.D, a.pack);
  const PreLayout PL = pre_layout(a.S, a.R, a.LT, a.T, a.Hq, a.D, a.NG, a.pack);
  const PlanHeader* hdr = reinterpret_cast<const PlanHeader*>(a.ws + L.header);
  const int4* list = reinterpret_cast<const int4*>(a.ws + PL.tok);
  __nv_bfloat16* outg = static_cast<__nv_bfloat16*>(a.out);
  // The plan is read before the wait for the attention kernel: that kernel's CTAs let this one
  // start only after their own wait for the planner, so the plan is complete and in L2 (ld.cg).
  // (An entry behind the list's end is read before the end is known, inside the workspace.)
  const int per_kvh = (a.G + HP - 1) / HP, per_tok = per_kvh * a.Hkv;
  long long job = (long long)blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
  const int i0 = (int)(job / per_tok);
  int4 e[3] = {};
  auto entry = [&](int i) {
#pragma unroll
    for (int k = 0; k < 3; ++k) e[k] = __ldcg(list + 3 * (size_t)i + k);
  };
  if (i0 < a.LT) entry(i0);
  const long long jobs = (long long)__ldcg(&hdr->pre_tokens) * per_tok;
  const long long ntiles = __ldcg(&hdr->dec_tiles), Wh = __ldcg(&hdr->pre_cost), W = Wh * a.Hkv;
  const int N = __ldcg(&hdr->decode_ctas), NP = __ldcg(&hdr->pre_ctas);
  const int per_tile = pre_tile_tokens(a.G);
  bool waited = false;
  for (; job < jobs; job += (long long)gridDim.x * (kMergeThreads / 32)) {
    const int i = (int)(job / per_tok), in_tok = (int)(job - (long long)i * per_tok);
    const int kvh = in_tok / per_kvh, h0 = (in_tok - kvh * per_kvh) * HP;
    const int nh = a.G - h0 < HP ? a.G - h0 : HP, head0 = kvh * a.G + h0;
    if (waited) entry(i);
    const int token = e[0].x, rec = e[0].y;
    // own keys' parts: decode CTAs df .. dl of the record
    const int df = rec < 0 ? 0 : cta_of_tile(e[0].z, ntiles, N);
    const int n_own = rec < 0 ? 0 : cta_of_tile(e[0].w - 1, ntiles, N) - df + 1;
    // a chain's parts: prefix CTAs pf ..., its place, and this token's first head's row in its tile
    struct Chain {
      long long cs;
      int w, nt, pf, n, tile, row;
    } ch[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int4 c = e[1 + k];  // place, tokens, tiles, cost0
      ch[k] = {0, 1, 0, 0, 0, 0, 0};
      if (c.z > 0) {
        const PreShape sh = pre_shape(c.y, c.z, a.G);
        ch[k].tile = c.x / per_tile;
        ch[k].w = (ch[k].tile >> 1) < sh.full ? kPreCost2 : kPreCost1;
        ch[k].nt = c.z;
        ch[k].cs = kvh * Wh + c.w + (ch[k].tile >> 1) * kPreCost2 * c.z;
        ch[k].pf = cta_of_tile(ch[k].cs, W, NP);
        ch[k].n = cta_of_tile(ch[k].cs + (long long)ch[k].w * c.z - 1, W, NP) - ch[k].pf + 1;
        ch[k].row = (c.x - ch[k].tile * per_tile) * a.G + h0;
      }
    }
    const int n_pre = ch[0].n + ch[1].n, nparts = n_pre + n_own;
    float M[HP], l[HP], acc[HP][PER];
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      M[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int k = 0; k < PER; ++k) acc[h][k] = 0.f;
    }
    for (int p0 = 0; p0 < nparts; p0 += 32) {
      // this lane's part: its first head's row of (m, l) and of O (the heads' rows follow it)
      const int p = p0 + lane;
      const float2* pml = nullptr;
      unsigned long long po = 0;
      if (p < n_pre) {
        const int k = p < ch[0].n ? 0 : 1;
        const Chain x = k ? ch[1] : ch[0];
        const int c = x.pf + (k ? p - ch[0].n : p);
        const int j0 = pre_step(x.cs, x.w, x.nt, pre_bound(W, c, NP));
        const int j1 = pre_step(x.cs, x.w, x.nt, pre_bound(W, c + 1, NP));
        const bool cut = j0 > 0;
        const size_t at = cut ? ((size_t)c * 2 + (x.tile & 1)) * kPrefillTileM + x.row
                              : ((size_t)i + (size_t)k * a.LT) * a.Hq + head0;
        if (j0 < j1) {  // (a range may end before the step that its last unit of cost lies in)
          pml = reinterpret_cast<const float2*>(a.ws + (cut ? PL.cut_ml : PL.base_ml)) + at;
          po = (unsigned long long)(reinterpret_cast<const float*>(
                                        a.ws + (cut ? PL.cut_o : PL.base_o)) + at * D);
        }
      } else if (p < nparts) {
        const size_t at = (((size_t)(df + p - n_pre) + (rec >> 3)) * a.pack + (rec & 7)) * a.Hq + head0;
        pml = reinterpret_cast<const float2*>(a.ws + L.part_ml) + at;
        po = (unsigned long long)(reinterpret_cast<const float*>(a.ws + L.part_o) + at * D);
      }
      if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
      float2 ml[HP];
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        ml[h] = make_float2(-INFINITY, 0.f);
        if (pml != nullptr && h < nh) ml[h] = pml[h];
      }
      float wt[HP];
#pragma unroll
      for (int h = 0; h < HP; ++h) {
        float mn = ml[h].x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mn = fmaxf(mn, M[h]);
        const float mx = mn;
        if (h >= nh || mn == -INFINITY) mn = 0.f;  // (no such head, or no key yet: every weight 0)
        const float sc = fast_exp2(M[h] - mn);
        wt[h] = fast_exp2(ml[h].x - mn);
        float ls = wt[h] * ml[h].y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, o);
        l[h] = l[h] * sc + ls;
        M[h] = mx;
#pragma unroll
        for (int k = 0; k < PER; ++k) acc[h][k] *= sc;
      }
      unsigned left = __ballot_sync(0xffffffffu, pml != nullptr);
      while (left) {
        float v[kC][HP][PER], wc[kC][HP];
#pragma unroll
        for (int cc = 0; cc < kC; ++cc) {
          const int src = left ? __ffs(left) - 1 : -1;
          left &= left - 1;  // (0 stays 0)
          const float* o = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, po, src & 31)) +
                           lane * PER;
#pragma unroll
          for (int h = 0; h < HP; ++h) {
            const float wx = __shfl_sync(0xffffffffu, wt[h], src & 31);
            wc[cc][h] = src < 0 ? 0.f : wx;
#pragma unroll
            for (int k = 0; k < PER; ++k) v[cc][h][k] = 0.f;
            if (src >= 0 && h < nh) {
              if constexpr (PER == 4) {
                const float4 x = *reinterpret_cast<const float4*>(o + h * D);
                v[cc][h][0] = x.x; v[cc][h][1] = x.y; v[cc][h][2] = x.z; v[cc][h][3] = x.w;
              } else {
                const float2 x = *reinterpret_cast<const float2*>(o + h * D);
                v[cc][h][0] = x.x; v[cc][h][1] = x.y;
              }
            }
          }
        }
#pragma unroll
        for (int cc = 0; cc < kC; ++cc)
#pragma unroll
          for (int h = 0; h < HP; ++h)
#pragma unroll
            for (int k = 0; k < PER; ++k) acc[h][k] += wc[cc][h] * v[cc][h][k];
      }
    }
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      if (h >= nh) continue;
      const float inv = 1.f / l[h];
      const size_t row = (size_t)token * a.Hq + head0 + h;
      uint32_t* dst = reinterpret_cast<uint32_t*>(outg + row * D + lane * PER);
      if constexpr (PER == 4)
        *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[h][0] * inv, acc[h][1] * inv),
                                                    pack_bf16x2(acc[h][2] * inv, acc[h][3] * inv));
      else
        dst[0] = pack_bf16x2(acc[h][0] * inv, acc[h][1] * inv);
      if (lane == 0 && a.lse != nullptr) a.lse[row] = (M[h] + __log2f(l[h])) * 0.6931471805599453f;
    }
  }
  // (without a row too: work behind this launch on the stream must not overtake the attention)
  if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
}

cudaError_t launch_prefix_merge(const AttnArgs& a, int sm_count, cudaStream_t stream) {
  // Four heads per warp where that leaves every SM two warps or more (32 sequences under 8 KV heads 27.6
  // us with one, 30.6 with four; 64 sequences 47.5 and 45.4).  8 parts of four heads in flight take all
  // registers of an SM for 8 warps, so with more blocks than SMs 4 (128 sequences on 4096 keys 57.4 us
  // with 4, 56.0 with 8; 256 on 8192 100.2 and 102.7).
  const bool four = (long long)a.LT * a.Hkv >= (long long)sm_count * 2 && a.G >= 4;
  const long long warps = (long long)a.LT * a.Hkv * (four ? (a.G + 3) / 4 : a.G);
  long long blocks = (warps + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
  const bool one_each = blocks <= sm_count;
  if (blocks > (long long)sm_count * 8) blocks = (long long)sm_count * 8;
  auto* kernel = a.D == 128 ? (!four      ? prefix_merge_kernel<128, 1, 8>
                               : one_each ? prefix_merge_kernel<128, 4, 8>
                                          : prefix_merge_kernel<128, 4, 4>)
                            : (!four      ? prefix_merge_kernel<64, 1, 8>
                               : one_each ? prefix_merge_kernel<64, 4, 8>
                                          : prefix_merge_kernel<64, 4, 4>);
  return launch_dependent(kernel, (unsigned)blocks, kMergeThreads, 0, stream, a);
}

cudaError_t launch_prefix_attention(const AttnArgs& a, const AttnMaps& m, const PrefixMaps& p,
                                    cudaStream_t stream) {
  if (a.D == 128)
    return a.G <= 8 ? launch_instance<128, 1>(a, m, p, stream)
                    : launch_instance<128, 2>(a, m, p, stream);
  return a.G <= 8 ? launch_instance<64, 1>(a, m, p, stream)
                  : launch_instance<64, 2>(a, m, p, stream);
}

}  // namespace cb

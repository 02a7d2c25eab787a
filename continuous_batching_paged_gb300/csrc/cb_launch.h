// Internal launch interface between the C ABI (cb_api.cu) and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace cb {

// Launch `kernel` as a programmatic dependent of the launch before it on the stream: it may start
// before that one ends (once all of its CTAs have allowed that, or ended), and waits for it with
// griddepcontrol.wait before it touches memory, so its launch latency overlaps.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned blocks, unsigned threads,
                             size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct AppendArgs {
  const void* k_new;
  const void* v_new;
  void* k_pages;
  void* v_pages;
  const int32_t* block_table;
  const int32_t* cu_seqlens_q;
  const int32_t* kv_lens;
  int S, T, Hkv, D, bs, max_blocks, P;
  uint32_t* err;
};

// The rotary append: what the plain append takes, plus q, its rotation, and the angles' table.
// Token rows of q / k_new / v_new are q_stride / k_stride / v_stride elements apart.
struct RopeArgs {
  AppendArgs ap;
  const void* q;     // NULL: keys are rotated and appended only
  void* q_out;       // [T, Hq, D]; may be q itself where q is contiguous
  const float* cos_sin;
  int Hq, max_positions, rot_dim, interleaved;
  long long q_stride, k_stride, v_stride;
  int parts;         // warps that share one token's heads
};

struct AttnArgs {
  const void* q;
  void* out;
  float* lse;
  const int32_t* block_table;
  const int32_t* cu_seqlens_q;
  const int32_t* kv_lens;
  char* ws;
  uint32_t* err;
  int S, T, Hq, Hkv, G, D, bs, max_blocks, P;
  int KB;              // rows per TMA box on the page pool, decode pass: gcd(bs, 16)
  int KBp;             // rows per TMA box on the page pool, chunk pass: gcd(bs, 128)
  int decode_ctas;     // CTAs of the decode pass per KV-head group (<= CB_MAX_DECODE_CTAS)
  int decode_grid;     // decode-role CTAs of this attention launch (decode_ctas x head groups;
                       // 0 when the launch runs the chunk pass only)
  int decode_auto;     // 1: the planner picks how many of them work (decode / chunk balance)
  int prefill_ctas;    // persistent CTAs of the chunk pass (0 when the launch runs decode only)
  int chunk_ctas;      // the same, whatever this launch runs (for the planner)
  int R;               // decode records the workspace is laid out for (S; pre_records with shared
                       // prefixes)
  int pack;            // most query tokens of a decode record (1; pre_pack(G) with shared prefixes)
  const int32_t* prefix_group;  // [S]: the group whose prefix a sequence shares, or -1
  const int32_t* prefix_lens;   // [NG]: keys of each group's prefix
  int NG;                       // groups (0 without shared prefixes)
  int window;          // > 0: query at position p sees keys (p - window, p]; 0: all <= p
  float scale_log2;    // softmax scale * log2(e)
  int LT;              // query tokens whose keys may be computed apart (0; pre_tokens).  Here, where it moves
                       // no other argument: two more in front of the others cost the chunk pass 0.6 %
};

// Block moves: copy (pool -> pool), offload (pool -> linear host buffer), restore (host ->
// pool).  Per pool (K, V) one block is block_bytes contiguous bytes.
enum BlockMoveMode { kMoveCopy = 0, kMoveOffload = 1, kMoveRestore = 2 };
struct BlockMoveArgs {
  const char* src[2];   // K, V: pool (copy, offload) or host buffer (restore)
  char* dst[2];         // K, V: pool (copy, restore) or host buffer (offload)
  const int32_t* src_idx;  // block ids read (copy, offload)
  const int32_t* dst_idx;  // block ids written (copy, restore)
  int n, P, mode;
  long long block_bytes;
  uint32_t* err;
};

// Id of the CUDA context the calling thread's next launch goes to (set by every API entry
// point before it launches; 0 if unknown).
unsigned long long launch_context_id();

cudaError_t launch_kv_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_rope_append(RopeArgs r, int sm_count, cudaStream_t stream);
cudaError_t launch_block_move(const BlockMoveArgs& a, int sm_count, cudaStream_t stream);
cudaError_t launch_wait_selftest(uint32_t* err, uint64_t limit_ns, uint64_t* waited_ns,
                                 cudaStream_t stream);
cudaError_t launch_plan(const AttnArgs& a, cudaStream_t stream);
// The append of a step and the planner of its attention pass in one launch (CTA 0 plans, the
// other CTAs append).
cudaError_t launch_append_plan(const AppendArgs& ap, const AttnArgs& a, cudaStream_t stream);
// Tensor maps of the attention pass: Q, and the page pools as the decode pass reads them
// (box of a page run of all KV heads of a group) and as the chunk pass reads them (one head).
struct AttnMaps {
  CUtensorMap q, k_dec, v_dec, k_chunk, v_chunk;
};
// The rotary append and the planner in one launch (with shared prefixes where a.NG > 0).
cudaError_t launch_rope_plan(RopeArgs r, const AttnArgs& a, int sm_count, cudaStream_t stream);
// The attention kernel: a.decode_grid decode-role CTAs, then a.prefill_ctas chunk-role CTAs.
cudaError_t launch_attention(const AttnArgs& a, const AttnMaps& maps, cudaStream_t stream);
// The planner and the attention kernel for a batch with shared prefixes (a.NG > 0).  Q as boxes of the
// query heads of one KV head: of one token, and of as many tokens as a tile of rows holds.
struct PrefixMaps {
  CUtensorMap q_tok, q_run;
};
cudaError_t launch_prefix_plan(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_prefix_attention(const AttnArgs& a, const AttnMaps& maps,
                                    const PrefixMaps& p, cudaStream_t stream);
// After it: merges the parts of the shared prefixes' rows.
cudaError_t launch_prefix_merge(const AttnArgs& a, int sm_count, cudaStream_t stream);

}  // namespace cb

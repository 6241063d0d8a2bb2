// serving_internal.h -- declarations shared between the entry points of jf_serving.h (serving_api.cu) and their
// kernels.
#pragma once

#include "../../include/jf_serving.h"
#include "jf_internal.h"

namespace jf {

// ---- sampling
constexpr int kMaxSampleVocab = 1 << 19;
constexpr int kMaxSampleRows = 1 << 24;

struct SampleParams {  // one entry per row (jf_sample) or sequence (jf_accept_sampled)
  const float* temperature;
  const int32_t* top_k;  // each of the three may be null: off
  const float* top_p;
  const float* min_p;
};

cudaError_t launch_sample(const void* logits, bool bf16, long long row_stride, int rows, int vocab, const float* u,
                          const SampleParams& sp, int32_t* token, float* logprob, int32_t* status,
                          cudaStream_t stream);
cudaError_t launch_accept_sampled(const int32_t* token, const int32_t* parent, const void* logits, bool bf16,
                                  const float* u, const SampleParams& sp, int batch, int num_nodes, int vocab,
                                  int max_depth, int32_t* accepted_len, int32_t* path, int32_t* bonus, float* logprob,
                                  int32_t* status, cudaStream_t stream);

#ifdef JF_DEBUG
cudaError_t hold_sample(int on);  // whether the kernels leave out the copies that they wait for (jf_debug_hold)
cudaError_t hold_accept_sampled(int on);
#endif

// ---- tree attention over a shared prefix
enum RowState : int { kRowBad = 0, kRowWhole = 1, kRowSplit = 2, kRowShares = 4 };

// Sequences whose own keys a kernel of their own takes (shared_small.cu): few rows and few keys.
constexpr int kSmallRows = 16, kSmallKeys = 1024;
__host__ __device__ inline bool small_sequence(int nodes, int group, int keys) {
  return nodes * group <= kSmallRows && keys <= kSmallKeys;
}

// Block-table entries a sequence: the kernels count its slots, rounded up to a tile, in 32 bits.
constexpr int kMaxSharedPages = (1 << 27) - 16;

struct SharedAttnParams : AttnParams {
  const int32_t* group_offsets;  // [num_groups + 1] sequences
  const int32_t* shared_lens;    // [num_groups]
  int num_groups;
  int small;        // whether that kernel runs
  int32_t* cta_ok;  // [kMaxGrid] 0 = the CTA gave up, or the batch's metadata are malformed
  // Softmax states of the rows, kind 0 from their own keys, kind 1 from the shared ones.  A row's place is
  // (node * group + head in the group) within its kv head, in which order an M tile's rows lie too.
  float4* rows_o;  // [2][hkv][32 column quads][rows]
  float2* rows_ml; // [2][hkv][rows] (running max in log2 units, row sum)
  int4* rows_at;   // [2][hkv][rows] RowState and, for a split unit, its first and last CTA and the row in its tiles

  __host__ __device__ long long rows() const { return static_cast<long long>(total_nodes) * group; }
  __device__ __forceinline__ float4* row_o(int kind, int kvh, int quad) const {
    return rows_o + ((static_cast<long long>(kind) * hkv + kvh) * 32 + quad) * rows();
  }
  __device__ __forceinline__ float2* row_ml(int kind, int kvh) const {
    return rows_ml + (static_cast<long long>(kind) * hkv + kvh) * rows();
  }
  __device__ __forceinline__ int4* row_at(int kind, int kvh) const {
    return rows_at + (static_cast<long long>(kind) * hkv + kvh) * rows();
  }
};

struct SharedArgs {  // what jf_tree_attention_shared takes beyond jf_tree_attention's arguments
  const int32_t* group_offsets;
  const int32_t* shared_lens;
  int num_groups;
};

struct SharedAttnWorkspace {  // byte offsets, each 256-aligned; the partials' part is AttnWorkspace's
  size_t ok_off, o_off, ml_off, at_off, total;
  SharedAttnWorkspace(int total_nodes, int num_q_heads) {
    auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t n = 2 * static_cast<size_t>(total_nodes) * num_q_heads;
    ok_off = up(AttnWorkspace::total);
    o_off = up(ok_off + kMaxGrid * sizeof(int32_t));
    ml_off = up(o_off + n * kHeadDim * sizeof(float));
    at_off = up(ml_off + n * sizeof(float2));
    total = up(at_off + n * sizeof(int4));
  }
};

// Validation, tensor maps, workspace carving and launch of the four attention entry points; shared is null for those of
// jf.h.
jf_status attention_call(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                         int max_pages_per_seq, const int32_t* prefix_lens, const int32_t* tree_offsets,
                         const int32_t* parent, const SharedArgs* shared, int batch, int total_nodes, int num_q_heads,
                         int num_kv_heads, int head_dim, int page_size, int num_pages, float sm_scale, bool fp8,
                         float k_scale, float v_scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                         int32_t* dev_status, jf_stream_t stream);

cudaError_t launch_shared_small(const void* q, const void* k_cache, const void* v_cache, const SharedAttnParams& p,
                                bool fp8_cache, cudaStream_t stream);
cudaError_t launch_tree_attention_shared(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                         const SharedAttnParams& p, int grid, bool fp8_cache, cudaStream_t stream);

}  // namespace jf

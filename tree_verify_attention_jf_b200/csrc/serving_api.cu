// serving_api.cu -- the C ABI of include/jf_serving.h: argument validation and kernel launches.  As in jf_api.cu, every
// check that needs no device data runs before the first CUDA call.
#include "serving_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace

extern "C" {

size_t jf_tree_attention_shared_workspace_size(int total_nodes, int num_q_heads) {
  return jf::SharedAttnWorkspace(total_nodes > 0 ? total_nodes : 0, num_q_heads > 0 ? num_q_heads : 0).total;
}

jf_status jf_tree_attention_shared(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                   int max_pages_per_seq, const int32_t* prefix_lens, const int32_t* tree_offsets,
                                   const int32_t* parent, const int32_t* group_offsets, const int32_t* shared_lens,
                                   int num_groups, int batch, int total_nodes, int num_q_heads, int num_kv_heads,
                                   int head_dim, int page_size, int num_pages, float sm_scale, void* out, float* lse,
                                   void* workspace, size_t workspace_bytes, int32_t* dev_status, jf_stream_t stream) {
  const jf::SharedArgs sh{group_offsets, shared_lens, num_groups};
  return jf::attention_call(q, k_cache, v_cache, block_table, max_pages_per_seq, prefix_lens, tree_offsets, parent, &sh,
                            batch, total_nodes, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, sm_scale,
                            false, 1.f, 1.f, out, lse, workspace, workspace_bytes, dev_status, stream);
}

jf_status jf_tree_attention_shared_fp8(const void* q, const void* k_cache, const void* v_cache, float k_scale,
                                       float v_scale, const int32_t* block_table, int max_pages_per_seq,
                                       const int32_t* prefix_lens, const int32_t* tree_offsets, const int32_t* parent,
                                       const int32_t* group_offsets, const int32_t* shared_lens, int num_groups,
                                       int batch, int total_nodes, int num_q_heads, int num_kv_heads, int head_dim,
                                       int page_size, int num_pages, float sm_scale, void* out, float* lse,
                                       void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                       jf_stream_t stream) {
  const jf::SharedArgs sh{group_offsets, shared_lens, num_groups};
  return jf::attention_call(q, k_cache, v_cache, block_table, max_pages_per_seq, prefix_lens, tree_offsets, parent, &sh,
                            batch, total_nodes, num_q_heads, num_kv_heads, head_dim, page_size, num_pages, sm_scale,
                            true, k_scale, v_scale, out, lse, workspace, workspace_bytes, dev_status, stream);
}

jf_status jf_sample(const void* logits, int logits_type, long long row_stride, int rows, int vocab, const float* u,
                    const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                    int32_t* token, float* logprob, int32_t* dev_status, jf_stream_t stream) {
  using namespace jf;
  if (rows < 0 || vocab <= 0 || row_stride < vocab) return JF_ERR_INVALID_ARG;
  if (logits_type != JF_LOGITS_F32 && logits_type != JF_LOGITS_BF16) return JF_ERR_INVALID_ARG;
  if (vocab > kMaxSampleVocab || rows > kMaxSampleRows) return JF_ERR_UNSUPPORTED;
  if (rows == 0) return JF_OK;
  if (!logits || !u || !temperature || !token) return JF_ERR_INVALID_ARG;
  if (!aligned(logits, 16)) return JF_ERR_INVALID_ARG;
  const SampleParams sp{temperature, top_k, top_p, min_p};
  if (launch_sample(logits, logits_type == JF_LOGITS_BF16, row_stride, rows, vocab, u, sp, token, logprob, dev_status,
                    reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return JF_ERR_CUDA;
  return JF_OK;
}

jf_status jf_accept_sampled(const int32_t* token, const int32_t* parent, const void* target_logits, int logits_type,
                            const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                            const float* min_p, int batch, int num_nodes, int vocab, int max_depth,
                            int32_t* accepted_len, int32_t* path, int32_t* bonus_token, float* logprob,
                            int32_t* dev_status, jf_stream_t stream) {
  using namespace jf;
  if (batch < 0 || num_nodes <= 0 || vocab <= 0 || max_depth < 0) return JF_ERR_INVALID_ARG;
  if (logits_type != JF_LOGITS_F32 && logits_type != JF_LOGITS_BF16) return JF_ERR_INVALID_ARG;
  if (num_nodes > kMaxAcceptNodes || max_depth >= kMaxAcceptNodes || vocab > kMaxSampleVocab || batch > kMaxSampleRows)
    return JF_ERR_UNSUPPORTED;
  if (batch == 0) return JF_OK;
  if (!token || !parent || !target_logits || !u || !temperature || !accepted_len || !path || !bonus_token)
    return JF_ERR_INVALID_ARG;
  if (!aligned(target_logits, 16)) return JF_ERR_INVALID_ARG;
  const SampleParams sp{temperature, top_k, top_p, min_p};
  if (launch_accept_sampled(token, parent, target_logits, logits_type == JF_LOGITS_BF16, u, sp, batch, num_nodes, vocab,
                            max_depth, accepted_len, path, bonus_token, logprob, dev_status,
                            reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return JF_ERR_CUDA;
  return JF_OK;
}

}  // extern "C"

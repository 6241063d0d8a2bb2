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

}  // namespace jf

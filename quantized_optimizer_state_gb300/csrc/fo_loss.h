// fo_loss.h -- interface between the C-ABI layer of the loss operators
// (fo_loss_api.cu) and their kernels (fo_logprobs.cu, fo_distill.cu). Not
// installed; not part of the ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fo {

// Rows of logits and their temperature, as the kernels see them.
struct LogitRows {
    const void *data;
    int64_t rows, vocab, row_stride, inner_rows, outer_stride;
    float inv_t;   // 1 / T
    float c;       // log2(e) / T: exp((x - m) / T) = 2^((x - m) c)
    float c_lo;    // what the rounding of c left
    float d_min;   // -160 / c: 2^((x - m) c) is 0 in FP32 from there on
};

// The gradient's rows (inner_rows is the logits').
struct GradRows {
    void *data;
    int64_t row_stride, outer_stride;
};

// Statistics by row, saved for the gradients:
//   log probabilities: {m, Z, H, unused}
//   distillation:      {m, Z, m_r, F}: m_r the largest logit that is not listed,
//                      F 2^((x_j - m_r) c) the gradient of KL by s_j at such a j
struct LogprobArgs {
    LogitRows in;
    const int64_t *tokens;   // may be null (then logp is)
    int32_t k;
    float *logp, *entropy;   // each may be null
    int32_t *top_ids;        // [rows, k]
    float *top_logp;
    float4 *stats;           // may be null
    int32_t ahead;           // set by the launch (fo_logprobs.cu)
};

struct LogprobGradArgs {
    LogitRows in;
    GradRows out;
    const int64_t *tokens;
    int32_t k;
    const int32_t *top_ids;
    const float4 *stats;
    const float *g_logp, *g_entropy, *g_top;   // null: 0
};

struct Teacher {
    const int32_t *ids;
    const void *logits;
    const float *lse;        // may be null
    float inv_t, inv_t_lo;   // 1 / its temperature, in two parts
    int32_t k, dtype, tail;
};

struct DistillArgs {
    LogitRows in;
    Teacher teacher;
    const float *weight;     // may be null: 1
    float *loss;             // may be null
    float4 *stats;           // may be null
    GradRows grad;           // data may be null
    int32_t mark_words;      // set by the launch: shared memory for marks (fo_distill.cu)
};

struct DistillGradArgs {
    LogitRows in;
    GradRows out;
    Teacher teacher;
    const float4 *stats;
    const float *g_loss;
};

cudaError_t launch_token_logprobs(int dtype, const LogprobArgs &a, cudaStream_t stream);
cudaError_t launch_token_logprobs_grad(int dtype, const LogprobGradArgs &a, cudaStream_t stream);
cudaError_t launch_distill(int dtype, const DistillArgs &a, cudaStream_t stream);
cudaError_t launch_distill_grad(int dtype, const DistillGradArgs &a, cudaStream_t stream);

}  // namespace fo

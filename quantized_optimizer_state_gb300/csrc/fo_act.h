// fo_act.h -- interface between the C-ABI layer of the operators on activations
// (fo_act_api.cu) and their kernels (fo_compress.cu, fo_activation.cu,
// fo_norm.cu). Not installed; not part of the ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace fo {

// Rows of `width` contiguous elements, `stride` elements apart.
struct RowsIn {
    const void *data;
    int64_t stride;
};
struct RowsOut {
    void *data;
    int64_t stride;
};

// What is kept of a matrix: codes[rows, 32 groups], steps[rows, groups].
struct KeptIn {
    const int8_t *codes;
    const uint16_t *steps;
};
struct KeptOut {
    int8_t *codes;     // null: nothing is kept
    uint16_t *steps;
};

struct CompressArgs {
    int64_t rows, width, groups;
    RowsIn x;
    KeptOut kept;
};
struct ExpandArgs {
    int64_t rows, width, groups;
    KeptIn kept;
    RowsOut x;
};

// up: data null for the kinds that are not gated.
struct ActivationArgs {
    int64_t rows, width, groups;
    RowsIn x, up;
    RowsOut y;
    KeptOut kept, kept_up;
};
struct ActivationGradArgs {
    int64_t rows, width, groups;
    KeptIn kept, kept_up;
    RowsIn grad_y;
    RowsOut grad, grad_up;
};

struct NormArgs {
    int64_t rows, width, groups;
    RowsIn x;
    const void *weight;     // may be null: 1
    int32_t weight_dtype;
    float eps;
    RowsOut y;
    float *inv_rms;
    KeptOut kept;           // inv_rms is null where it is
    float inv_width;        // these two are set by the launch
    bool weight_aligned;
};
struct NormGradArgs {
    int64_t rows, width, groups;
    KeptIn kept;
    const float *inv_rms;
    const void *weight;     // may be null: 1
    int32_t weight_dtype;
    RowsIn grad_y;
    RowsOut grad;
    void *grad_weight;      // may be null
    float *parts;           // [norm_parts, 32 groups] partial sums of grad_weight
    float inv_width;        // these two are set by the launch
    bool weight_aligned;
};

// Rows of partial sums that the norm's gradient leaves at most, by the sizes alone, so
// that a workspace can be made without asking the device: 1024 for rows held in
// registers (more of short rows, whose CTAs are small), fewer of longer rows, whose
// columns fill the device by themselves. A bound: the present launches leave one or
// two a multiprocessor of rows of 1024 elements and more, 304 at 4096 columns (5 of
// the 17 MB are touched), 152 at 16384 (10 of 67).
inline int64_t norm_parts(int64_t rows, int64_t groups)
{
    const int64_t least = groups <= 512 ? 1024 : 64, most = ((int64_t)1 << (groups <= 512 ? 17 : 19)) / groups;
    const int64_t parts = most < least ? least : most;
    return rows < parts ? rows : parts;
}

cudaError_t launch_compress(int dtype, const CompressArgs &a, cudaStream_t stream);
cudaError_t launch_expand(int dtype, const ExpandArgs &a, cudaStream_t stream);
cudaError_t launch_activation(int dtype, int kind, const ActivationArgs &a, cudaStream_t stream);
cudaError_t launch_activation_grad(int dtype, int kind, const ActivationGradArgs &a, cudaStream_t stream);
cudaError_t launch_norm(int dtype, const NormArgs &a, cudaStream_t stream);
cudaError_t launch_norm_grad(int dtype, const NormGradArgs &a, cudaStream_t stream);

}  // namespace fo

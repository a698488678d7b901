// qk_rope.cuh -- launch interface of the query/key norm and rotation (qk_rope.cu).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace gdn2 {

struct QkRopeArgs {
    gdn2_dtype dt;
    long long tokens;                 // B * T
    int Hq, Hk, D;
    const void *q, *k;                // heads of a token contiguous, tokens q_stride / k_stride elements apart
    long long q_stride, k_stride;
    const void* positions;            // [num_axes, tokens] int32 or int64
    int pos64, num_axes;
    const float* inv_freq;            // [pairs]
    const int* axes;                  // [pairs] or null: every pair turns by axis 0
    int pairs, interleaved, norm;
    float eps;
    const float *q_weight, *k_weight; // [D] or null
    void *q_out, *k_out;              // forward
    const void *dq_out, *dk_out;      // backward
    void *dq, *dk;
    float *dq_weight, *dk_weight;     // or null
};
constexpr int QK_ROPE_BLOCKS = 148 * 2;   // blocks of the backward at most: each leaves one weight's partial gradient
cudaError_t qk_rope_launch(const QkRopeArgs& a, float* ws, cudaStream_t s);
cudaError_t qk_rope_error_word(unsigned int** word);

}  // namespace gdn2

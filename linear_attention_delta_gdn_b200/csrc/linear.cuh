// linear.cuh -- pieces shared by the kernels of linear attention with one fixed decay per head,
//     S_t = a_h S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a_h = exp(log_decay_h).
//
// One pass serves the forward and the three token gradients. With row operand x, column operand y and values z,
//     out_i = sum_{j <= i} a^{i-j} (x_i . y_j) z_j + a^{i+1} R^T x_i           (forwards in time, R the start state)
//     out_i = sum_{j >= i} a^{j-i} (x_i . y_j) z_j + a^{T-1-i} R^T x_i         (backwards, R the state behind the end)
//   o  : x = q,    y = k,    z = v,    forwards,  R = S_0      (state sum a^. k v^T)
//   dq : x = dout, y = v,    z = k,    forwards,  R = S_0^T    (the same state, transposed)
//   dk : x = v,    y = dout, z = q,    backwards, R = dS_T^T   (state sum a^. q dout^T, transposed)
//   dv : x = k,    y = q,    z = dout, backwards, R = dS_T
// and the two states' ends are S_T = a^T S_0 + sum_j a^{T-1-j} k_j v_j^T and dS_0 = a^T dS_T + sum_i a^{i+1} q_i
// dout_i^T. Every power of a has an exponent >= 0, so nothing grows for log_decay <= 0.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "linear_cut.h"

namespace gdn2 {
namespace linear {

// The sequences of a call: dense [N, T, H, D] (cu null) or packed [Ttot, H, D] with cu_seqlens on the device.
struct Seqs {
    const int* cu;       // [N + 1] or null
    int N, T;            // sequences; their length, or the bound Tmax on it
    long long Ttot;      // rows of the token tensors
    int H, Dk, Dv;
};

// First token row and length of sequence n; records an inconsistent cu_seqlens.
__device__ __forceinline__ int seq_span(const Seqs& s, int n, long long* begin, unsigned int* err) {
    if (!s.cu) {
        *begin = (long long)n * s.T;
        return s.T;
    }
    const int b = s.cu[n], e = s.cu[n + 1];
    *begin = b;
    if (b < 0 || e < b || e > s.Ttot) {
        if ((threadIdx.x & 31) == 0) atomicOr(err, ERR_OUTSIDE);
        *begin = 0;
        return 0;
    }
    if (e - b > s.T) {
        if ((threadIdx.x & 31) == 0) atomicOr(err, ERR_LONG);
        return s.T;
    }
    return e - b;
}

// log2 of a head's decay factor. Below e^-200 per token a^1 is already 0 in 32 bits, so a stronger decay
// (-inf too) is the same as e^-200, and a^0 stays 1. A NaN stays a NaN.
__device__ __forceinline__ float log2_decay(const float* log_decay, int h) {
    const float g = log_decay[h];
    return (g < -200.f ? -200.f : g) * 1.4426950408889634f;
}
// a^n from log2(a); n >= 0
__device__ __forceinline__ float decay_pow(float l2, int n) { return exp2f(l2 * (float)n); }

}  // namespace linear

struct LinearArgs {
    linear::Seqs seq;
    gdn2_dtype dt;
    const void *q, *k, *v, *dout;
    const float *log_decay, *S0, *dST;
    void *o, *dq, *dk, *dv;
    float *ST, *dS0;
    void* ws;
};
// fp32 (linear_f32.cu); packed: a varlen call with s.Ttot rows
size_t linear32_workspace(const linear::Seqs& s, bool packed, bool backward);
cudaError_t linear32_launch(const LinearArgs& a, bool backward, cudaStream_t s);
cudaError_t linear32_error_word(unsigned int** word);

// bf16 on tensor cores (linear_chunk.cu)
size_t linear_chunk_workspace(const linear::Seqs& s, bool backward);
cudaError_t linear_chunk_launch(const LinearArgs& a, bool backward, cudaStream_t s);
cudaError_t linear_chunk_error_word(unsigned int** word);

struct LinearStepArgs {
    gdn2_dtype dt;
    const void *q, *k, *v;
    const float* log_decay;
    float* S;
    const int* slots;   // null: row b's state is S[b]
    int num_slots;
    void* o;
    int B, H, Dk, Dv;
};
cudaError_t linear_step_launch(const LinearStepArgs& a, cudaStream_t s);
cudaError_t linear_step_error_word(unsigned int** word);

}  // namespace gdn2

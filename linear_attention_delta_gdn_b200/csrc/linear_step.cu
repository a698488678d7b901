// linear_step.cu -- one token of linear attention with a decay per head for every request of a batch:
//     S <- a_h S + k v^T,   o = S^T q,   on the states of a pool that the requests' slots name.
//
// The state is read and written once, 8 Dk Dv bytes a request and head, against 5 Dk Dv operations: the memory bound.
// A block a state and all its rows in flight: 256 requests of 16 heads of 128 x 128 take 83 us, 6.4 TB/s (97% of the copy
// rate); one request, its states spread over 64 blocks of 32 columns, 3.1 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "linear.cuh"

namespace gdn2 {
namespace {

__device__ unsigned int g_step_error;

// A block owns CS columns of one request's and head's state: thread tid holds the float4 column group tid % C4 of the
// rows tid / C4 + r RSTEP, all of them in flight at once.
template <int DK, int CS>
struct StepLayout {
    static constexpr int C4 = CS / 4;
    static constexpr int NT = DK * C4 >= 256 ? 256 : DK * C4;
    static constexpr int RSTEP = NT / C4;
    static constexpr int RPT = DK / RSTEP;
    static constexpr int WARPS = (NT + 31) / 32;
};

template <typename Tin, int DK, int CS>
__global__ void __launch_bounds__(StepLayout<DK, CS>::NT)
linear_step_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
                   const float* __restrict__ log_decay, float* __restrict__ S, const int* __restrict__ slots, int num_slots,
                   Tin* __restrict__ o, int H, int Dv) {
    using L = StepLayout<DK, CS>;
    __shared__ float red[L::WARPS][CS];
    const int tid = threadIdx.x, c4 = tid % L::C4, r0 = tid / L::C4;
    const int b = blockIdx.x / H, h = blockIdx.x % H;
    const int col = blockIdx.y * CS + 4 * c4;
    const size_t row = blockIdx.x;
    Tin* out = o + row * Dv + blockIdx.y * CS;
    const int slot = slots ? slots[b] : b;
    const bool inside = slot >= 0 && slot < num_slots;
    float4 s[L::RPT];
    float* Sh = S + ((size_t)(inside ? slot : 0) * H + h) * DK * Dv + col;
    if (inside)
#pragma unroll
        for (int r = 0; r < L::RPT; ++r)
            s[r] = __ldcs(reinterpret_cast<const float4*>(Sh + (size_t)(r0 + r * L::RSTEP) * Dv));
    // A slot belongs to the first row that names it; while the state is on its way, look for an earlier one.
    bool mine = inside;
    if (slots && inside) {
        bool earlier = false;
        for (int i = tid; i < b; i += L::NT) earlier |= slots[i] == slot;
        mine = !__syncthreads_or(earlier);
    }
    if (!mine) {
        if (tid == 0 && slot >= 0) atomicOr(&g_step_error, ERR_SLOT);
        for (int j = tid; j < CS; j += L::NT) out[j] = from_f32<Tin>(0.f);
        return;
    }
    const float a = exp2f(linear::log2_decay(log_decay, h));
    const float v0 = to_f32(v[row * Dv + col]), v1 = to_f32(v[row * Dv + col + 1]), v2 = to_f32(v[row * Dv + col + 2]),
                v3 = to_f32(v[row * Dv + col + 3]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int r = 0; r < L::RPT; ++r) {
        const int i = r0 + r * L::RSTEP;
        const float kk = to_f32(k[row * DK + i]), qq = to_f32(q[row * DK + i]);
        s[r].x = fmaf(a, s[r].x, kk * v0);
        s[r].y = fmaf(a, s[r].y, kk * v1);
        s[r].z = fmaf(a, s[r].z, kk * v2);
        s[r].w = fmaf(a, s[r].w, kk * v3);
        acc.x = fmaf(qq, s[r].x, acc.x);
        acc.y = fmaf(qq, s[r].y, acc.y);
        acc.z = fmaf(qq, s[r].z, acc.z);
        acc.w = fmaf(qq, s[r].w, acc.w);
        __stcs(reinterpret_cast<float4*>(Sh + (size_t)i * Dv), s[r]);
    }
    // the lanes of a warp that share a column group, then the warps
#pragma unroll
    for (int m = L::C4; m < 32; m <<= 1) {
        acc.x += __shfl_xor_sync(0xffffffffu, acc.x, m);
        acc.y += __shfl_xor_sync(0xffffffffu, acc.y, m);
        acc.z += __shfl_xor_sync(0xffffffffu, acc.z, m);
        acc.w += __shfl_xor_sync(0xffffffffu, acc.w, m);
    }
    if ((tid & 31) < L::C4) *reinterpret_cast<float4*>(&red[tid >> 5][4 * c4]) = acc;
    __syncthreads();
    for (int j = tid; j < CS; j += L::NT) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < L::WARPS; ++w) x += red[w][j];
        out[j] = from_f32<Tin>(x);
    }
}

template <typename Tin, int DK, int CS>
cudaError_t step(const LinearStepArgs& a, cudaStream_t s) {
    TraceScope trace(K_LINEAR_STEP, s);
    linear_step_kernel<Tin, DK, CS><<<dim3(a.B * a.H, a.Dv / CS), StepLayout<DK, CS>::NT, 0, s>>>(
        static_cast<const Tin*>(a.q), static_cast<const Tin*>(a.k), static_cast<const Tin*>(a.v), a.log_decay, a.S, a.slots,
        a.num_slots, static_cast<Tin*>(a.o), a.H, a.Dv);
    return cudaGetLastError();
}
template <typename Tin, int DK>
cudaError_t step_columns(const LinearStepArgs& a, cudaStream_t s) {
    // Few states: 32 columns a block, so that a small batch's states spread over more SMs. In a replayed graph, states of
    // 128 x 128, 32 columns a block against all of them: 64 states 4.3 against 6.2 us, 128 states 6.3 both, 256 states 8.3
    // against 6.6.
    const bool few = (long long)a.B * a.H * (a.Dv / 32) <= 2 * 148;
    if (a.Dv == 16) return step<Tin, DK, 16>(a, s);
    if (a.Dv == 32 || few) return step<Tin, DK, 32>(a, s);
    if (a.Dv == 64) return step<Tin, DK, 64>(a, s);
    return step<Tin, DK, 128>(a, s);
}
template <typename Tin>
cudaError_t step_rows(const LinearStepArgs& a, cudaStream_t s) {
    switch (a.Dk) {
    case 16: return step_columns<Tin, 16>(a, s);
    case 32: return step_columns<Tin, 32>(a, s);
    case 64: return step_columns<Tin, 64>(a, s);
    default: return step_columns<Tin, 128>(a, s);
    }
}

}  // namespace

cudaError_t linear_step_launch(const LinearStepArgs& a, cudaStream_t s) {
    return a.dt == GDN2_BF16 ? step_rows<__nv_bfloat16>(a, s) : step_rows<float>(a, s);
}

cudaError_t linear_step_error_word(unsigned int** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_step_error);
}

}  // namespace gdn2

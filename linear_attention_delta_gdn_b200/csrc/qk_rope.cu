// qk_rope.cu -- RMS norm of every query and key head and the rotation of its channel pairs by the token's position,
// in one pass, and their backward.
//
// Per head row x of D channels:  n = x w / sqrt(mean(x^2) + eps)   (n = x without a norm), then for pair p < P
//     (y_a, y_b) = (n_a cos t - n_b sin t, n_a sin t + n_b cos t),   t = position[axis_p] * inv_freq_p
// with the pair's channels a = p, b = p + P, or a = 2p, b = 2p + 1 (interleaved); channels behind 2P stay n.
// Backward, with d the gradient turned back by -t and m = x / sqrt(mean(x^2) + eps):
//     dx = (d w - m mean(d w m)) / sqrt(mean(x^2) + eps),   dw = sum over rows of d m
//
// The rows are read and written once (HBM-bound). An angle is the same for all heads of a token: a warp takes a token,
// makes its cosines and sines once, each lane keeps those of its channels in registers, and the token's rows pass by,
// several in flight, 16 bytes a lane at each of a pair's two places. Few tokens: several warps share a token's heads.
// Far positions: the angle is a whole-number product modulo one turn, so a position of millions (or of 2^40) keeps the
// error of a small one (a 32-bit product is off by 0.06 at a million).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "qk_rope.cuh"

namespace gdn2 {
namespace {

constexpr int WARPS = 4;           // warps of a block, one token each

__device__ unsigned int g_rope_error;

// VEC consecutive channels at each of a pair's two places; interleaved pairs lie next to one another.
template <int VEC>
__device__ __forceinline__ void get(const float* p, float* x) {
    if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
            const float4 u = *reinterpret_cast<const float4*>(p + i);
            x[i] = u.x; x[i + 1] = u.y; x[i + 2] = u.z; x[i + 3] = u.w;
        }
    } else {
        x[0] = *p;
    }
}
__device__ __forceinline__ void unpack(uint32_t u, float* x) {
    x[0] = __uint_as_float(u << 16);
    x[1] = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
template <int VEC>
__device__ __forceinline__ void get(const __nv_bfloat16* p, float* x) {
    if constexpr (VEC == 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        unpack(u.x, x); unpack(u.y, x + 2); unpack(u.z, x + 4); unpack(u.w, x + 6);
    } else if constexpr (VEC == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        unpack(u.x, x); unpack(u.y, x + 2);
    } else {
        x[0] = __bfloat162float(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void put(float* p, const float* x) {
    if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
        *p = x[0];
    }
}
template <int VEC>
__device__ __forceinline__ void put(__nv_bfloat16* p, const float* x) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7]));
    } else if constexpr (VEC == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack(x[0], x[1]), pack(x[2], x[3]));
    } else {
        *p = __float2bfloat16_rn(x[0]);
    }
}

// A row's 2 VEC-channel slots: slot s < P / VEC holds VEC pairs, the later ones 2 VEC channels that do not turn.
// LPR lanes share a row, SPL slots each.
template <int D, int VEC>
struct RowLayout {
    static constexpr int SLOTS = D / (2 * VEC);
    static constexpr int LPR = SLOTS < 32 ? SLOTS : 32;
    static constexpr int SPL = SLOTS / LPR;
    static constexpr int RPW = 32 / LPR;                   // rows of a warp
};

template <int VEC, bool IL>
__device__ __forceinline__ void places(int slot, int P, int* a, int* b) {
    const int turning = P / VEC;
    if (IL || slot >= turning) {
        *a = 2 * VEC * slot;   // 2 P = 2 VEC turning: the slots that stay follow the pairs
        *b = *a + VEC;
    } else {
        *a = VEC * slot;
        *b = P + VEC * slot;
    }
}
// One slot's pairs, pair i in (x[i], x[VEC + i]) (interleaved memory order is a0 b0 a1 b1 ...).
template <typename T, int VEC, bool IL>
__device__ __forceinline__ void load_slot(const T* row, int slot, int P, float* x) {
    int a, b;
    places<VEC, IL>(slot, P, &a, &b);
    float y[2 * VEC];
    get<VEC>(row + a, y);
    get<VEC>(row + b, y + VEC);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        x[i] = IL ? y[2 * i] : y[i];
        x[VEC + i] = IL ? y[2 * i + 1] : y[VEC + i];
    }
}
template <typename T, int VEC, bool IL>
__device__ __forceinline__ void store_slot(T* row, int slot, int P, const float* x) {
    int a, b;
    places<VEC, IL>(slot, P, &a, &b);
    float y[2 * VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        if (IL) {
            y[2 * i] = x[i];
            y[2 * i + 1] = x[VEC + i];
        } else {
            y[i] = x[i];
            y[VEC + i] = x[VEC + i];
        }
    }
    put<VEC>(row + a, y);
    put<VEC>(row + b, y + VEC);
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = LPR / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// pos * inv_freq in half turns, in [-1, 1). Turns per position as a 64-bit fraction F (whole turns do not count): the
// product with 1 / 2 pi as a double and its rest, so F is right to its last bit; pos * F then wraps at whole turns by
// itself, and the angle is off by |pos| 2^-64 turns.
__device__ __forceinline__ float position_half_turns(long long pos, float inv_freq) {
    if (!isfinite(inv_freq)) return __int_as_float(0x7fc00000);
    const double f = inv_freq;
    double turns = f * 0.15915494309189535;
    const double rest = fma(f, 0.15915494309189535, -turns) + f * -9.839338337591243e-18;
    turns -= floor(turns);
    const unsigned long long F = __double2ull_rz(turns * 18446744073709551616.0) +
                                 (unsigned long long)__double2ll_rn(rest * 18446744073709551616.0);
    return (float)((double)(long long)((unsigned long long)pos * F) * 0x1p-63);
}

// cos and sin of token t's angles for this lane's slots; `cs` is the warp's own. A pair whose axis does not exist stays.
template <int D, int VEC>
__device__ __forceinline__ void make_angles(const QkRopeArgs& a, long long t, float2* cs,
                                            float2 (&mine)[RowLayout<D, VEC>::SPL][VEC]) {
    using L = RowLayout<D, VEC>;
    const int lane = threadIdx.x & 31;
    __syncwarp();
    for (int p = lane; p < a.pairs; p += 32) {
        const int ax = a.axes ? a.axes[p] : 0;
        float half_turns = 0.f;
        if (ax >= 0 && ax < a.num_axes) {
            const long long at = (long long)ax * a.tokens + t;
            const long long pos = a.pos64 ? static_cast<const long long*>(a.positions)[at] : static_cast<const int*>(a.positions)[at];
            half_turns = position_half_turns(pos, a.inv_freq[p]);
        } else {
            atomicOr(&g_rope_error, 1u);
        }
        float s, c;
        sincospif(half_turns, &s, &c);
        cs[p] = make_float2(c, s);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < L::SPL; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int p = (lane % L::LPR + j * L::LPR) * VEC + i;
            mine[j][i] = p < a.pairs ? cs[p] : make_float2(1.f, 0.f);
        }
}

template <typename T, int D, int VEC, bool IL>
__device__ __forceinline__ void load_weight(const T* w, int sl, int P, float (&g)[RowLayout<D, VEC>::SPL][2 * VEC]) {
    using L = RowLayout<D, VEC>;
#pragma unroll
    for (int j = 0; j < L::SPL; ++j) {
        if (w) load_slot<float, VEC, IL>(w, sl + j * L::LPR, P, g[j]);
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i)
            if (!w) g[j][i] = 1.f;
    }
}

// Rows lo .. hi - 1 of one token and tensor: U rows a lane in flight.
template <typename T, int D, int VEC, bool IL, int U>
__device__ __forceinline__ void rows_fwd(const QkRopeArgs& a, const T* src, T* dst, const float* w, int lo, int hi,
                                         const float2 (&cs)[RowLayout<D, VEC>::SPL][VEC]) {
    using L = RowLayout<D, VEC>;
    const int lane = threadIdx.x & 31, sl = lane % L::LPR;
    float g[L::SPL][2 * VEC];
    if (a.norm) load_weight<float, D, VEC, IL>(w, sl, a.pairs, g);
    for (int r0 = lo + lane / L::LPR; r0 - lane / L::LPR < hi; r0 += U * L::RPW) {
        float x[U][L::SPL][2 * VEC];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < L::SPL; ++j) {
                if (r0 + u * L::RPW < hi) load_slot<T, VEC, IL>(src + (size_t)(r0 + u * L::RPW) * D, sl + j * L::LPR, a.pairs, x[u][j]);
                else
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) x[u][j][i] = 0.f;
            }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (a.norm) {
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < L::SPL; ++j)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) sum = fmaf(x[u][j][i], x[u][j][i], sum);
                const float scale = rsqrtf(row_sum<L::LPR>(sum) * (1.f / D) + a.eps);
#pragma unroll
                for (int j = 0; j < L::SPL; ++j)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) x[u][j][i] *= scale * g[j][i];
            }
            if (r0 + u * L::RPW < hi)
#pragma unroll
                for (int j = 0; j < L::SPL; ++j) {
                    float y[2 * VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {   // slots that do not turn have cosine 1 and sine 0
                        const float2 c = cs[j][i];
                        y[i] = x[u][j][i] * c.x - x[u][j][VEC + i] * c.y;
                        y[VEC + i] = x[u][j][i] * c.y + x[u][j][VEC + i] * c.x;
                    }
                    const bool turns = sl + j * L::LPR < a.pairs / VEC;
                    store_slot<T, VEC, IL>(dst + (size_t)(r0 + u * L::RPW) * D, sl + j * L::LPR, a.pairs, turns ? y : x[u][j]);
                }
        }
    }
}

template <typename T, int D, int VEC, bool IL>
__global__ void __launch_bounds__(32 * WARPS) qk_rope_fwd_kernel(const __grid_constant__ QkRopeArgs a) {
    using L = RowLayout<D, VEC>;
    constexpr int U = VEC == 8 ? 2 : 4;
    __shared__ float2 cs[WARPS][D / 2];
    const long long t = (long long)blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (t >= a.tokens) return;
    float2 mine[L::SPL][VEC];
    make_angles<D, VEC>(a, t, cs[threadIdx.x >> 5], mine);
    const int heads = a.Hq + a.Hk, part = (heads + gridDim.y - 1) / gridDim.y;
    const int lo = blockIdx.y * part, hi = min(heads, lo + part);
    if (lo < a.Hq)
        rows_fwd<T, D, VEC, IL, U>(a, static_cast<const T*>(a.q) + t * a.q_stride, static_cast<T*>(a.q_out) + t * a.Hq * D, a.q_weight,
                                   lo, min(hi, a.Hq), mine);
    if (hi > a.Hq)
        rows_fwd<T, D, VEC, IL, U>(a, static_cast<const T*>(a.k) + t * a.k_stride, static_cast<T*>(a.k_out) + t * a.Hk * D, a.k_weight,
                                   max(0, lo - a.Hq), hi - a.Hq, mine);
}

template <typename T, int D, int VEC, bool IL>
__device__ __forceinline__ void rows_bwd(const QkRopeArgs& a, const T* src, const T* dy, T* dst, const float* w, int n,
                                         const float2 (&cs)[RowLayout<D, VEC>::SPL][VEC], float (&dw)[RowLayout<D, VEC>::SPL][2 * VEC]) {
    using L = RowLayout<D, VEC>;
    const int lane = threadIdx.x & 31, sl = lane % L::LPR;
    float g[L::SPL][2 * VEC];
    if (a.norm) load_weight<float, D, VEC, IL>(w, sl, a.pairs, g);
    for (int r = lane / L::LPR; r - lane / L::LPR < n; r += L::RPW) {
        const bool on = r < n;
        float x[L::SPL][2 * VEC], d[L::SPL][2 * VEC];
#pragma unroll
        for (int j = 0; j < L::SPL; ++j) {
            const int slot = sl + j * L::LPR;
            if (on) {
                load_slot<T, VEC, IL>(dy + (size_t)r * D, slot, a.pairs, d[j]);
                if (a.norm) load_slot<T, VEC, IL>(src + (size_t)r * D, slot, a.pairs, x[j]);
            }
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i) {
                if (!on) d[j][i] = 0.f;
                if (!on || !a.norm) x[j][i] = 0.f;
            }
            if (slot < a.pairs / VEC)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float2 c = cs[j][i];
                    const float da = d[j][i], db = d[j][VEC + i];
                    d[j][i] = da * c.x + db * c.y;
                    d[j][VEC + i] = db * c.x - da * c.y;
                }
        }
        if (a.norm) {
            float sum = 0.f, dot = 0.f;
#pragma unroll
            for (int j = 0; j < L::SPL; ++j)
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) {
                    sum = fmaf(x[j][i], x[j][i], sum);
                    dot = fmaf(d[j][i] * g[j][i], x[j][i], dot);
                }
            const float rs = rsqrtf(row_sum<L::LPR>(sum) * (1.f / D) + a.eps);
            const float mean = row_sum<L::LPR>(dot) * rs * (1.f / D);   // mean(d w m)
#pragma unroll
            for (int j = 0; j < L::SPL; ++j)
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) {
                    const float m = x[j][i] * rs;
                    if (on) dw[j][i] = fmaf(d[j][i], m, dw[j][i]);
                    d[j][i] = (d[j][i] * g[j][i] - m * mean) * rs;
                }
        }
        if (on)
#pragma unroll
            for (int j = 0; j < L::SPL; ++j) store_slot<T, VEC, IL>(dst + (size_t)r * D, sl + j * L::LPR, a.pairs, d[j]);
    }
}

template <typename T, int D, int VEC, bool IL>
__global__ void __launch_bounds__(32 * WARPS) qk_rope_bwd_kernel(const __grid_constant__ QkRopeArgs a, float* __restrict__ partial) {
    using L = RowLayout<D, VEC>;
    __shared__ float2 cs[WARPS][D / 2];
    __shared__ float part[2][WARPS][D];
    const int lane = threadIdx.x & 31, sl = lane % L::LPR, warp = threadIdx.x >> 5;
    float dw[2][L::SPL][2 * VEC] = {};
    for (long long t = (long long)blockIdx.x * WARPS + warp; t < a.tokens; t += (long long)gridDim.x * WARPS) {
        float2 mine[L::SPL][VEC];
        make_angles<D, VEC>(a, t, cs[warp], mine);
        rows_bwd<T, D, VEC, IL>(a, static_cast<const T*>(a.q) + t * a.q_stride, static_cast<const T*>(a.dq_out) + t * a.Hq * D,
                                static_cast<T*>(a.dq) + t * a.Hq * D, a.q_weight, a.Hq, mine, dw[0]);
        rows_bwd<T, D, VEC, IL>(a, static_cast<const T*>(a.k) + t * a.k_stride, static_cast<const T*>(a.dk_out) + t * a.Hk * D,
                                static_cast<T*>(a.dk) + t * a.Hk * D, a.k_weight, a.Hk, mine, dw[1]);
    }
    if (!partial) return;
    // the block's share of the weight gradients: the rows of a warp, then the warps in order
#pragma unroll
    for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int j = 0; j < L::SPL; ++j) {
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i)
#pragma unroll
                for (int m = L::LPR; m < 32; m <<= 1) dw[which][j][i] += __shfl_xor_sync(0xffffffffu, dw[which][j][i], m);
            if (lane < L::LPR) store_slot<float, VEC, IL>(part[which][warp], sl + j * L::LPR, a.pairs, dw[which][j]);
        }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += 32 * WARPS) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s += part[x / D][i][x % D];
        partial[(size_t)blockIdx.x * 2 * D + x] = s;
    }
}

// The weight gradients: one block per channel and tensor sums the blocks' shares in a fixed order.
__global__ void __launch_bounds__(128) qk_rope_weights_kernel(const float* __restrict__ partial, int blocks, int D,
                                                              float* __restrict__ dwq, float* __restrict__ dwk) {
    __shared__ float warps[4];
    float s = 0.f;
    for (int i = threadIdx.x; i < blocks; i += 128) s += partial[(size_t)i * 2 * D + blockIdx.x];
    s = row_sum<32>(s);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x) return;
    s = (warps[0] + warps[1]) + (warps[2] + warps[3]);
    float* out = (int)blockIdx.x < D ? dwq : dwk;
    if (out) out[blockIdx.x % D] = s;
}

template <typename T, int D, int VEC, bool IL>
cudaError_t run(const QkRopeArgs& a, float* ws, cudaStream_t s) {
    const long long blocks = (a.tokens + WARPS - 1) / WARPS;
    if (!a.dq) {
        // few tokens: their heads over several warps, as long as there are SMs without work and rows to share
        const int rows = (a.Hq + a.Hk + RowLayout<D, VEC>::RPW - 1) / RowLayout<D, VEC>::RPW;
        const long long want = (148 * 2 + blocks - 1) / blocks;
        const int parts = (int)(want < rows ? want : rows);
        TraceScope trace(K_QK_ROPE, s);
        qk_rope_fwd_kernel<T, D, VEC, IL><<<dim3((unsigned)blocks, parts), 32 * WARPS, 0, s>>>(a);
        return cudaGetLastError();
    }
    const int grid = (int)(blocks < QK_ROPE_BLOCKS ? blocks : QK_ROPE_BLOCKS);
    const bool weights = a.norm && (a.dq_weight || a.dk_weight);
    {
        TraceScope trace(K_QK_ROPE_BWD, s);
        qk_rope_bwd_kernel<T, D, VEC, IL><<<grid, 32 * WARPS, 0, s>>>(a, weights ? ws : nullptr);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !weights) return e;
    TraceScope trace(K_QK_ROPE_BWD, s);
    qk_rope_weights_kernel<<<2 * D, 128, 0, s>>>(ws, grid, D, a.dq_weight, a.dk_weight);
    return cudaGetLastError();
}
template <typename T, int D>
cudaError_t run_d(const QkRopeArgs& a, float* ws, cudaStream_t s) {
    // as many pairs at a time as 16 bytes hold where the pairs divide so, else four, else one
    if (sizeof(T) == 2 && a.pairs % 8 == 0) {
        if constexpr (sizeof(T) == 2) return a.interleaved ? run<T, D, 8, true>(a, ws, s) : run<T, D, 8, false>(a, ws, s);
    }
    if (a.pairs % 4 == 0) return a.interleaved ? run<T, D, 4, true>(a, ws, s) : run<T, D, 4, false>(a, ws, s);
    return a.interleaved ? run<T, D, 1, true>(a, ws, s) : run<T, D, 1, false>(a, ws, s);
}
template <typename T>
cudaError_t run_t(const QkRopeArgs& a, float* ws, cudaStream_t s) {
    switch (a.D) {
    case 16: return run_d<T, 16>(a, ws, s);
    case 32: return run_d<T, 32>(a, ws, s);
    case 64: return run_d<T, 64>(a, ws, s);
    default: return run_d<T, 128>(a, ws, s);
    }
}

}  // namespace

cudaError_t qk_rope_launch(const QkRopeArgs& a, float* ws, cudaStream_t s) {
    return a.dt == GDN2_BF16 ? run_t<__nv_bfloat16>(a, ws, s) : run_t<float>(a, ws, s);
}

cudaError_t qk_rope_take_errors(unsigned int* bits) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_rope_error, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_rope_error, &zero, sizeof(unsigned int));
}

}  // namespace gdn2

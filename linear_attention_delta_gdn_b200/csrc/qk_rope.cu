// qk_rope.cu -- RMS norm of every query and key head and the rotation of its channel pairs by the token's position,
// in one pass, and their backward.
//
// Per head row x of D channels:  n = x w / sqrt(mean(x^2) + eps)   (n = x without a norm), then for pair p < P
//     (y_a, y_b) = (n_a cos t - n_b sin t, n_a sin t + n_b cos t),   t = position[axis_p] * inv_freq_p
// with the pair's channels a = p, b = p + P, or a = 2p, b = 2p + 1 (interleaved); channels behind 2P stay n.
// Backward, with d the gradient turned back by -t and m = x / sqrt(mean(x^2) + eps):
//     dx = (d w - m mean(d w m)) / sqrt(mean(x^2) + eps),   dw = sum over rows of d m
//
// The rows are read and written once (HBM-bound). An angle is the same for all heads of a token: a block works on a
// few tokens, makes their cosines and sines once in shared memory, and its warps then take the tokens' rows.
// Far positions: the angle is a whole-number product modulo one turn, so a position of millions (or of 2^40) keeps the
// error of a small one (a 32-bit product is off by 0.06 at a million).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "qk_rope.cuh"

namespace gdn2 {
namespace {

constexpr int RT = 256;            // threads of a block
constexpr int TOKENS_MAX = 8;      // tokens of a tile at most

__device__ unsigned int g_rope_error;

// VEC consecutive channels at each of a pair's two places; interleaved pairs lie next to one another.
template <int VEC>
__device__ __forceinline__ void get(const float* p, float* x) {
    if constexpr (VEC == 4) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    } else {
        x[0] = *p;
    }
}
template <int VEC>
__device__ __forceinline__ void get(const __nv_bfloat16* p, float* x) {
    if constexpr (VEC == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
        const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
        x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
    } else {
        x[0] = __bfloat162float(*p);
    }
}
template <int VEC>
__device__ __forceinline__ void put(float* p, const float* x) {
    if constexpr (VEC == 4) *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    else *p = x[0];
}
template <int VEC>
__device__ __forceinline__ void put(__nv_bfloat16* p, const float* x) {
    if constexpr (VEC == 4) {
        uint2 u;
        *reinterpret_cast<__nv_bfloat162*>(&u.x) = __floats2bfloat162_rn(x[0], x[1]);
        *reinterpret_cast<__nv_bfloat162*>(&u.y) = __floats2bfloat162_rn(x[2], x[3]);
        *reinterpret_cast<uint2*>(p) = u;
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
    static constexpr int ROWS = RPW * (RT / 32);           // rows of a block at a time
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

// cos and sin of the tile's angles, [tokens][P]
__device__ __forceinline__ void make_angles(const QkRopeArgs& a, long long t0, int n, float2* cs) {
    for (int x = threadIdx.x; x < n * a.pairs; x += RT) {
        const int p = x % a.pairs;
        const long long t = t0 + x / a.pairs;
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
        cs[x] = make_float2(c, s);
    }
}

template <typename T, int D, int VEC, bool IL>
__global__ void __launch_bounds__(RT) qk_rope_fwd_kernel(const __grid_constant__ QkRopeArgs a, int tile) {
    using L = RowLayout<D, VEC>;
    __shared__ float2 cs[TOKENS_MAX * D / 2];
    const long long t0 = (long long)blockIdx.x * tile;
    const int n = (int)min((long long)tile, a.tokens - t0);
    make_angles(a, t0, n, cs);
    __syncthreads();
    const int heads = a.Hq + a.Hk, rows = n * heads;
    const int lane = threadIdx.x & 31, sl = lane % L::LPR;
    const int turning = a.pairs / VEC;
    for (int r0 = (threadIdx.x >> 5) * L::RPW; r0 < rows; r0 += L::ROWS) {
        const int r = r0 + lane / L::LPR;
        const bool on = r < rows;
        const int tt = on ? r / heads : 0, hd = on ? r % heads : 0;
        const bool isq = hd < a.Hq;
        const T* src = isq ? static_cast<const T*>(a.q) + (t0 + tt) * a.q_stride + hd * D
                           : static_cast<const T*>(a.k) + (t0 + tt) * a.k_stride + (hd - a.Hq) * D;
        T* dst = isq ? static_cast<T*>(a.q_out) + ((t0 + tt) * a.Hq + hd) * D
                     : static_cast<T*>(a.k_out) + ((t0 + tt) * a.Hk + hd - a.Hq) * D;
        const float* w = isq ? a.q_weight : a.k_weight;
        float x[L::SPL][2 * VEC];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < L::SPL; ++j) {
            if (on) load_slot<T, VEC, IL>(src, sl + j * L::LPR, a.pairs, x[j]);
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i) {
                if (!on) x[j][i] = 0.f;
                sum = fmaf(x[j][i], x[j][i], sum);
            }
        }
        if (a.norm) {
            const float scale = rsqrtf(row_sum<L::LPR>(sum) * (1.f / D) + a.eps);
#pragma unroll
            for (int j = 0; j < L::SPL; ++j) {
                float g[2 * VEC];
                if (w) load_slot<float, VEC, IL>(w, sl + j * L::LPR, a.pairs, g);
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) x[j][i] *= w ? scale * g[i] : scale;
            }
        }
#pragma unroll
        for (int j = 0; j < L::SPL; ++j) {
            const int slot = sl + j * L::LPR;
            if (slot < turning)
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float2 c = cs[tt * a.pairs + slot * VEC + i];
                    const float xa = x[j][i], xb = x[j][VEC + i];
                    x[j][i] = xa * c.x - xb * c.y;
                    x[j][VEC + i] = xa * c.y + xb * c.x;
                }
            if (on) store_slot<T, VEC, IL>(dst, slot, a.pairs, x[j]);
        }
    }
}

template <typename T, int D, int VEC, bool IL>
__global__ void __launch_bounds__(RT) qk_rope_bwd_kernel(const __grid_constant__ QkRopeArgs a, int tile, float* __restrict__ partial) {
    using L = RowLayout<D, VEC>;
    __shared__ float2 cs[TOKENS_MAX * D / 2];
    __shared__ float part[2][RT / 32][D];
    const int heads = a.Hq + a.Hk;
    const int lane = threadIdx.x & 31, sl = lane % L::LPR;
    const int turning = a.pairs / VEC;
    float dw[2][L::SPL][2 * VEC] = {};
    for (long long t0 = (long long)blockIdx.x * tile; t0 < a.tokens; t0 += (long long)gridDim.x * tile) {
        const int n = (int)min((long long)tile, a.tokens - t0);
        __syncthreads();
        make_angles(a, t0, n, cs);
        __syncthreads();
        const int rows = n * heads;
        for (int r0 = (threadIdx.x >> 5) * L::RPW; r0 < rows; r0 += L::ROWS) {
            const int r = r0 + lane / L::LPR;
            const bool on = r < rows;
            const int tt = on ? r / heads : 0, hd = on ? r % heads : 0;
            const bool isq = hd < a.Hq;
            const size_t flat = isq ? ((t0 + tt) * a.Hq + hd) * D : ((t0 + tt) * a.Hk + hd - a.Hq) * D;
            const T* src = isq ? static_cast<const T*>(a.q) + (t0 + tt) * a.q_stride + hd * D
                               : static_cast<const T*>(a.k) + (t0 + tt) * a.k_stride + (hd - a.Hq) * D;
            const T* dy = static_cast<const T*>(isq ? a.dq_out : a.dk_out) + flat;
            T* dst = static_cast<T*>(isq ? a.dq : a.dk) + flat;
            const float* w = isq ? a.q_weight : a.k_weight;
            float x[L::SPL][2 * VEC], d[L::SPL][2 * VEC];
#pragma unroll
            for (int j = 0; j < L::SPL; ++j) {
                const int slot = sl + j * L::LPR;
                if (on) {
                    load_slot<T, VEC, IL>(dy, slot, a.pairs, d[j]);
                    if (a.norm) load_slot<T, VEC, IL>(src, slot, a.pairs, x[j]);
                }
#pragma unroll
                for (int i = 0; i < 2 * VEC; ++i) {
                    if (!on) d[j][i] = 0.f;
                    if (!on || !a.norm) x[j][i] = 0.f;
                }
                if (slot < turning)
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float2 c = cs[tt * a.pairs + slot * VEC + i];
                        const float da = d[j][i], db = d[j][VEC + i];
                        d[j][i] = da * c.x + db * c.y;
                        d[j][VEC + i] = db * c.x - da * c.y;
                    }
            }
            if (a.norm) {
                float sum = 0.f, dot = 0.f;
                float g[L::SPL][2 * VEC];
#pragma unroll
                for (int j = 0; j < L::SPL; ++j) {
                    if (w) load_slot<float, VEC, IL>(w, sl + j * L::LPR, a.pairs, g[j]);
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) {
                        if (!w) g[j][i] = 1.f;
                        sum = fmaf(x[j][i], x[j][i], sum);
                        dot = fmaf(d[j][i] * g[j][i], x[j][i], dot);
                    }
                }
                const float rs = rsqrtf(row_sum<L::LPR>(sum) * (1.f / D) + a.eps);
                const float mean = row_sum<L::LPR>(dot) * rs * (1.f / D);   // mean(d w m)
#pragma unroll
                for (int j = 0; j < L::SPL; ++j)
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) {
                        const float m = x[j][i] * rs;
                        const float dm = on ? d[j][i] * m : 0.f;
                        dw[0][j][i] += isq ? dm : 0.f;
                        dw[1][j][i] += isq ? 0.f : dm;
                        d[j][i] = (d[j][i] * g[j][i] - m * mean) * rs;
                    }
            }
            if (on)
#pragma unroll
                for (int j = 0; j < L::SPL; ++j) store_slot<T, VEC, IL>(dst, sl + j * L::LPR, a.pairs, d[j]);
        }
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
            if (lane < L::LPR) store_slot<float, VEC, IL>(part[which][threadIdx.x >> 5], sl + j * L::LPR, a.pairs, dw[which][j]);
        }
    __syncthreads();
    for (int x = threadIdx.x; x < 2 * D; x += RT) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < RT / 32; ++i) s += part[x / D][i][x % D];
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

// Tokens of a tile: enough rows for a block's warps, few enough tiles' worth of tokens that every SM has blocks.
int tile_of(const QkRopeArgs& a) {
    long long t = a.tokens / (148 * 8);
    return (int)(t < 1 ? 1 : t > TOKENS_MAX ? TOKENS_MAX : t);
}

template <typename T, int D, int VEC, bool IL>
cudaError_t run(const QkRopeArgs& a, float* ws, cudaStream_t s) {
    const int tile = tile_of(a);
    const long long tiles = (a.tokens + tile - 1) / tile;
    if (!a.dq) {
        TraceScope trace(K_QK_ROPE, s);
        qk_rope_fwd_kernel<T, D, VEC, IL><<<(unsigned)tiles, RT, 0, s>>>(a, tile);
        return cudaGetLastError();
    }
    const int blocks = (int)(tiles < QK_ROPE_BLOCKS ? tiles : QK_ROPE_BLOCKS);
    const bool weights = a.norm && (a.dq_weight || a.dk_weight);
    {
        TraceScope trace(K_QK_ROPE_BWD, s);
        qk_rope_bwd_kernel<T, D, VEC, IL><<<blocks, RT, 0, s>>>(a, tile, weights ? ws : nullptr);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !weights) return e;
    TraceScope trace(K_QK_ROPE_BWD, s);
    qk_rope_weights_kernel<<<2 * D, 128, 0, s>>>(ws, blocks, D, a.dq_weight, a.dk_weight);
    return cudaGetLastError();
}
template <typename T, int D>
cudaError_t run_d(const QkRopeArgs& a, float* ws, cudaStream_t s) {
    // four pairs at a time where the pairs divide so, else one
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

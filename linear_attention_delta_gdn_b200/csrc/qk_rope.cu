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
// several in flight as they lie in memory, 16 bytes a lane at each of a pair's two places. What an angle needs 64 bits
// for does not depend on the token and is made once a block. Few tokens: several warps share a token's heads.
// Measured: 4 x 4096 tokens of 16 + 16 heads of 128 take 54 us, 4.9 TB/s (76% of the copy rate); 2 x 3999 tokens of 16 + 4
// heads with the backward and both weights' gradients 58 us (the forward 24, the backward 35: loads of few rows a token
// to wait for); 64 tokens of one serving step 3.6 us, the latency of the loads.
// Far positions: the angle is a whole-number product modulo one turn, off by |position| 2^-63 turns at most, whatever the
// sign of the position or the frequency: below a 32-bit angle's own rounding up to 2^38, 7e-7 rad at 2^40 (a 32-bit product
// is off by 0.06 rad at a million).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "qk_rope.cuh"

namespace gdn2 {
namespace {

constexpr int WARPS = 8;           // warps of a block, each with tokens of its own

__device__ unsigned int g_rope_error;

// VEC consecutive channels as they lie in memory, and as floats.
template <int BYTES> struct Piece;
template <> struct Piece<16> { using type = uint4; };
template <> struct Piece<8> { using type = uint2; };
template <> struct Piece<4> { using type = uint32_t; };
template <> struct Piece<2> { using type = unsigned short; };
template <typename T, int VEC>
using piece_t = typename Piece<VEC * (int)sizeof(T)>::type;

__device__ __forceinline__ void widen(uint32_t u, float* x) {
    x[0] = __uint_as_float(u << 16);
    x[1] = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ uint32_t narrow(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void widen(const uint4& u, float (&x)[8], __nv_bfloat16) {
    widen(u.x, x); widen(u.y, x + 2); widen(u.z, x + 4); widen(u.w, x + 6);
}
__device__ __forceinline__ void widen(const uint2& u, float (&x)[4], __nv_bfloat16) { widen(u.x, x); widen(u.y, x + 2); }
__device__ __forceinline__ void widen(unsigned short u, float (&x)[1], __nv_bfloat16) { x[0] = __uint_as_float((uint32_t)u << 16); }
__device__ __forceinline__ void widen(const uint4& u, float (&x)[4], float) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void widen(uint32_t u, float (&x)[1], float) { x[0] = __uint_as_float(u); }
__device__ __forceinline__ void narrow(const float (&x)[8], uint4& u, __nv_bfloat16) {
    u = make_uint4(narrow(x[0], x[1]), narrow(x[2], x[3]), narrow(x[4], x[5]), narrow(x[6], x[7]));
}
__device__ __forceinline__ void narrow(const float (&x)[4], uint2& u, __nv_bfloat16) { u = make_uint2(narrow(x[0], x[1]), narrow(x[2], x[3])); }
__device__ __forceinline__ void narrow(const float (&x)[1], unsigned short& u, __nv_bfloat16) { u = __bfloat16_as_ushort(__float2bfloat16_rn(x[0])); }
__device__ __forceinline__ void narrow(const float (&x)[4], uint4& u, float) {
    u = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
__device__ __forceinline__ void narrow(const float (&x)[1], uint32_t& u, float) { u = __float_as_uint(x[0]); }

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
// One slot as it lies in memory; its pairs, pair i in (x[i], x[VEC + i]) (interleaved memory order is a0 b0 a1 b1 ...).
template <typename T, int VEC>
struct Slot {
    piece_t<T, VEC> a, b;
};
template <typename T, int VEC, bool IL>
__device__ __forceinline__ Slot<T, VEC> load_slot(const T* row, int slot, int P) {
    int a, b;
    places<VEC, IL>(slot, P, &a, &b);
    Slot<T, VEC> s;
    s.a = *reinterpret_cast<const piece_t<T, VEC>*>(row + a);
    s.b = *reinterpret_cast<const piece_t<T, VEC>*>(row + b);
    return s;
}
template <typename T, int VEC, bool IL>
__device__ __forceinline__ void pairs_of(const Slot<T, VEC>& s, float (&x)[2 * VEC]) {
    float y[2][VEC];
    widen(s.a, y[0], T());
    widen(s.b, y[1], T());
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        x[i] = IL ? (&y[0][0])[2 * i] : y[0][i];
        x[VEC + i] = IL ? (&y[0][0])[2 * i + 1] : y[1][i];
    }
}
template <typename T, int VEC, bool IL>
__device__ __forceinline__ void store_slot(T* row, int slot, int P, const float (&x)[2 * VEC]) {
    int a, b;
    places<VEC, IL>(slot, P, &a, &b);
    float y[2][VEC];
#pragma unroll
    for (int i = 0; i < 2 * VEC; ++i) (&y[0][0])[i] = IL ? x[(i & 1) * VEC + (i >> 1)] : x[i];
    Slot<T, VEC> s;
    narrow(y[0], s.a, T());
    narrow(y[1], s.b, T());
    *reinterpret_cast<piece_t<T, VEC>*>(row + a) = s.a;
    *reinterpret_cast<piece_t<T, VEC>*>(row + b) = s.b;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int m = LPR / 2; m >= 1; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Turns per position as a 64-bit fraction (whole turns do not count): the product with 1 / 2 pi as a double and its
// rest, each off by one unit of 2^-64 at most. Of the size, negated as a whole number: a small negative double
// brought to [0, 1) would keep 53 bits of its difference to 1.
__device__ __forceinline__ unsigned long long turns_of(float inv_freq) {
    const double f = fabsf(inv_freq);
    double turns = f * 0.15915494309189535;
    const double rest = fma(f, 0.15915494309189535, -turns) + f * -9.839338337591243e-18;
    turns -= floor(turns);
    const unsigned long long units =
        __double2ull_rz(turns * 18446744073709551616.0) + (unsigned long long)__double2ll_rn(rest * 18446744073709551616.0);
    return inv_freq < 0.f ? 0ull - units : units;
}
// The thread's index, read once (the compiler would read the special register again wherever registers are short, and a
// read takes as long as a shuffle).
__device__ __forceinline__ int thread_index() {
    int t;
    asm volatile("mov.u32 %0, %tid.x;" : "=r"(t));
    return t;
}
// What a block keeps of its pairs: the fraction and the axis (-1: none, the pair stays; -2: not a number).
struct Pairs {
    unsigned long long turns[64];
    int axis[64];
};
__device__ __forceinline__ void make_pairs(const QkRopeArgs& a, Pairs& q) {
    for (int p = threadIdx.x; p < a.pairs; p += 32 * WARPS) {
        const float f = a.inv_freq[p];
        int ax = a.axes ? a.axes[p] : 0;
        if (ax < 0 || ax >= a.num_axes) {
            ax = -1;
            atomicOr(&g_rope_error, 1u);
        } else if (!isfinite(f)) {
            ax = -2;
        }
        q.axis[p] = ax;
        q.turns[p] = ax >= 0 ? turns_of(f) : 0;
    }
    __syncthreads();
}
// cos and sin of token t's angles for this lane's slots; `cs` is the warp's own. pos * turns wraps at whole turns by
// itself, so the angle is off by |pos| times what a turn's fraction is before it rounds to 32 bits.
template <typename T, int D, int VEC>
__device__ __forceinline__ void make_angles(const QkRopeArgs& a, const Pairs& q, long long t, int lane, float2* cs,
                                            float2 (&mine)[RowLayout<D, VEC>::SPL][VEC]) {
    using L = RowLayout<D, VEC>;
    __syncwarp();
    for (int p = lane; p < a.pairs; p += 32) {
        const int ax = q.axis[p];
        float half_turns = ax == -2 ? __int_as_float(0x7fc00000) : 0.f;
        if (ax >= 0) {
            const long long at = (long long)ax * a.tokens + t;
            const long long pos = a.pos64 ? static_cast<const long long*>(a.positions)[at] : static_cast<const int*>(a.positions)[at];
            half_turns = (float)((int)(((unsigned long long)pos * q.turns[p]) >> 32)) * 0x1p-31f;
        }
        float s, c;
        if (sizeof(T) == 2) __sincosf(half_turns * 3.14159265f, &s, &c);   // off by 2^-21 on [-pi, pi]: the outputs have 8 bits
        else sincospif(half_turns, &s, &c);
        cs[p / VEC * (VEC + 2) + p % VEC] = make_float2(c, s);   // 16 bytes of shift a lane's pairs: no bank twice
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < L::SPL; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)   // of slots that do not turn whatever lies there: they are not used
            mine[j][i] = cs[(lane % L::LPR + j * L::LPR) * (VEC + 2) + i];
}

template <int D, int VEC, bool IL>
__device__ __forceinline__ void load_weight(const float* w, int sl, int P, float (&g)[RowLayout<D, VEC>::SPL][2 * VEC]) {
    using L = RowLayout<D, VEC>;
#pragma unroll
    for (int j = 0; j < L::SPL; ++j) {
        int pa, pb;
        places<VEC, IL>(sl + j * L::LPR, P, &pa, &pb);
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i) {
            const int at = i < VEC ? (IL ? pa + 2 * i : pa + i) : (IL ? pa + 2 * (i - VEC) + 1 : pb + i - VEC);
            g[j][i] = w ? w[at] : 1.f;
        }
    }
}

// A token's rows into L2, a 128-byte line a lane: the warp's next token, while it works on this one.
template <typename T>
__device__ __forceinline__ void rows_ahead(const T* p, int elements, int lane) {
    const char* c = reinterpret_cast<const char*>(p);
    for (int at = lane * 128; at < elements * (int)sizeof(T); at += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(c + at));
}

// Rows of both places that a lane has in flight: 64 bytes of bf16 in 16-byte pieces, as much else.
template <typename T, int D, int VEC>
constexpr int rows_in_flight() { return VEC == 1 ? 1 : 64 / (2 * VEC * (int)sizeof(T)); }

// A block works on one of the two tensors, the first q_blocks on q, the others on k, and keeps its weight in registers;
// blockIdx.y takes a part of the heads.
template <typename T, int D, int VEC, bool IL>
__global__ void __launch_bounds__(32 * WARPS, VEC == 1 ? 1 : 3) qk_rope_fwd_kernel(const __grid_constant__ QkRopeArgs a, int q_blocks) {
    using L = RowLayout<D, VEC>;
    constexpr int U = rows_in_flight<T, D, VEC>();
    __shared__ Pairs pairs;
    __shared__ __align__(16) float2 cs[WARPS][D / 2 + 2 * (D / 2 / VEC)];
    make_pairs(a, pairs);
    const int tid = thread_index(), lane = tid & 31, sl = lane % L::LPR, sub = lane / L::LPR, warp = tid >> 5;
    const bool isq = (int)blockIdx.x < q_blocks;
    const int block = isq ? blockIdx.x : blockIdx.x - q_blocks, blocks = isq ? q_blocks : gridDim.x - q_blocks;
    const int n = isq ? a.Hq : a.Hk, part = (n + gridDim.y - 1) / gridDim.y;
    const int lo = blockIdx.y * part, hi = min(n, lo + part);
    if (lo >= hi) return;
    float g[L::SPL][2 * VEC];
    if (a.norm) load_weight<D, VEC, IL>(isq ? a.q_weight : a.k_weight, sl, a.pairs, g);
    for (long long t = (long long)block * WARPS + warp; t < a.tokens; t += (long long)blocks * WARPS) {
        const T* src = isq ? static_cast<const T*>(a.q) + t * a.q_stride : static_cast<const T*>(a.k) + t * a.k_stride;
        T* dst = static_cast<T*>(isq ? a.q_out : a.k_out) + t * n * D;
        const long long next = (long long)blocks * WARPS;
        if (t + next < a.tokens) rows_ahead(src + next * (isq ? a.q_stride : a.k_stride), n * D, lane);
        float2 c[L::SPL][VEC];
        make_angles<T, D, VEC>(a, pairs, t, lane, cs[warp], c);
        for (int base = lo; base < hi; base += U * L::RPW) {
            Slot<T, VEC> raw[U][L::SPL];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < L::SPL; ++j) {   // past the last row: that row once more, for the sums; it is not stored
                    const int r = min(base + u * L::RPW + sub, hi - 1);
                    raw[u][j] = load_slot<T, VEC, IL>(src + (size_t)r * D, sl + j * L::LPR, a.pairs);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = base + u * L::RPW + sub;
                float x[L::SPL][2 * VEC];
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < L::SPL; ++j) {
                    pairs_of<T, VEC, IL>(raw[u][j], x[j]);
#pragma unroll
                    for (int i = 0; i < 2 * VEC; ++i) sum = fmaf(x[j][i], x[j][i], sum);
                }
                if (a.norm) {
                    const float scale = rsqrtf(row_sum<L::LPR>(sum) * (1.f / D) + a.eps);
#pragma unroll
                    for (int j = 0; j < L::SPL; ++j)
#pragma unroll
                        for (int i = 0; i < 2 * VEC; ++i) x[j][i] *= scale * g[j][i];
                }
#pragma unroll
                for (int j = 0; j < L::SPL; ++j) {
                    if (sl + j * L::LPR < a.pairs / VEC)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float xa = x[j][i], xb = x[j][VEC + i];
                            x[j][i] = xa * c[j][i].x - xb * c[j][i].y;
                            x[j][VEC + i] = xa * c[j][i].y + xb * c[j][i].x;
                        }
                    if (r < hi) store_slot<T, VEC, IL>(dst + (size_t)r * D, sl + j * L::LPR, a.pairs, x[j]);
                }
            }
        }
    }
}

// The same split; a block keeps one weight's gradient.
template <typename T, int D, int VEC, bool IL>
__global__ void __launch_bounds__(32 * WARPS, VEC == 1 ? 1 : 2)
qk_rope_bwd_kernel(const __grid_constant__ QkRopeArgs a, int q_blocks, float* __restrict__ partial) {
    using L = RowLayout<D, VEC>;
    constexpr int U = VEC == 1 ? 1 : rows_in_flight<T, D, VEC>() / 2;
    __shared__ Pairs pairs;
    __shared__ __align__(16) float2 cs[WARPS][D / 2 + 2 * (D / 2 / VEC)];
    __shared__ float part[WARPS][D];
    make_pairs(a, pairs);
    const int tid = thread_index(), lane = tid & 31, sl = lane % L::LPR, sub = lane / L::LPR, warp = tid >> 5;
    const bool isq = (int)blockIdx.x < q_blocks;
    const int block = isq ? blockIdx.x : blockIdx.x - q_blocks, blocks = isq ? q_blocks : gridDim.x - q_blocks;
    const int n = isq ? a.Hq : a.Hk;
    float g[L::SPL][2 * VEC], dw[L::SPL][2 * VEC] = {};
    if (a.norm) load_weight<D, VEC, IL>(isq ? a.q_weight : a.k_weight, sl, a.pairs, g);
    for (long long t = (long long)block * WARPS + warp; t < a.tokens; t += (long long)blocks * WARPS) {
        const T* src = isq ? static_cast<const T*>(a.q) + t * a.q_stride : static_cast<const T*>(a.k) + t * a.k_stride;
        const T* dy = static_cast<const T*>(isq ? a.dq_out : a.dk_out) + t * n * D;
        T* dst = static_cast<T*>(isq ? a.dq : a.dk) + t * n * D;
        const long long next = (long long)blocks * WARPS;
        if (t + next < a.tokens) {
            rows_ahead(dy + next * n * D, n * D, lane);
            if (a.norm) rows_ahead(src + next * (isq ? a.q_stride : a.k_stride), n * D, lane);
        }
        float2 c[L::SPL][VEC];
        make_angles<T, D, VEC>(a, pairs, t, lane, cs[warp], c);
        for (int base = 0; base < n; base += U * L::RPW) {
            Slot<T, VEC> rx[U][L::SPL], rd[U][L::SPL];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int j = 0; j < L::SPL; ++j) {
                    const int r = min(base + u * L::RPW + sub, n - 1);
                    rd[u][j] = load_slot<T, VEC, IL>(dy + (size_t)r * D, sl + j * L::LPR, a.pairs);
                    if (a.norm) rx[u][j] = load_slot<T, VEC, IL>(src + (size_t)r * D, sl + j * L::LPR, a.pairs);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = base + u * L::RPW + sub;
                const bool on = r < n;
                float d[L::SPL][2 * VEC];
#pragma unroll
                for (int j = 0; j < L::SPL; ++j) {
                    pairs_of<T, VEC, IL>(rd[u][j], d[j]);
                    if (sl + j * L::LPR < a.pairs / VEC)
#pragma unroll
                        for (int i = 0; i < VEC; ++i) {
                            const float da = d[j][i], db = d[j][VEC + i];
                            d[j][i] = da * c[j][i].x + db * c[j][i].y;
                            d[j][VEC + i] = db * c[j][i].x - da * c[j][i].y;
                        }
                }
                if (a.norm) {
                    float x[L::SPL][2 * VEC];
                    float sum = 0.f, dot = 0.f;
#pragma unroll
                    for (int j = 0; j < L::SPL; ++j) {
                        pairs_of<T, VEC, IL>(rx[u][j], x[j]);
#pragma unroll
                        for (int i = 0; i < 2 * VEC; ++i) {
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
                            if (on) dw[j][i] = fmaf(d[j][i], m, dw[j][i]);
                            d[j][i] = (d[j][i] * g[j][i] - m * mean) * rs;
                        }
                }
                if (on)
#pragma unroll
                    for (int j = 0; j < L::SPL; ++j) store_slot<T, VEC, IL>(dst + (size_t)r * D, sl + j * L::LPR, a.pairs, d[j]);
            }
        }
    }
    if (!partial) return;
    // the block's share of the weight's gradient: the rows of a warp, then the warps in order
#pragma unroll
    for (int j = 0; j < L::SPL; ++j) {
#pragma unroll
        for (int i = 0; i < 2 * VEC; ++i)
#pragma unroll
            for (int m = L::LPR; m < 32; m <<= 1) dw[j][i] += __shfl_xor_sync(0xffffffffu, dw[j][i], m);
        int pa, pb;
        places<VEC, IL>(sl + j * L::LPR, a.pairs, &pa, &pb);
        if (lane < L::LPR)
#pragma unroll
            for (int i = 0; i < 2 * VEC; ++i)
                part[warp][i < VEC ? (IL ? pa + 2 * i : pa + i) : (IL ? pa + 2 * (i - VEC) + 1 : pb + i - VEC)] = dw[j][i];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < D; x += 32 * WARPS) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s += part[i][x];
        partial[(size_t)blockIdx.x * D + x] = s;
    }
}

// The weights' gradients: a block sums 32 channels of one of them over the blocks' shares, 32 runs of them in order.
__global__ void __launch_bounds__(1024) qk_rope_weights_kernel(const float* __restrict__ partial, int q_blocks, int blocks, int D,
                                                               float* __restrict__ dwq, float* __restrict__ dwk) {
    __shared__ float runs[32][33];
    float* out = blockIdx.y == 0 ? dwq : dwk;
    if (!out) return;
    const int c = threadIdx.x & 31, g = threadIdx.x >> 5, ch = blockIdx.x * 32 + c;
    const int from = blockIdx.y == 0 ? 0 : q_blocks, to = blockIdx.y == 0 ? q_blocks : blocks;
    float s = 0.f;
    if (ch < D)
#pragma unroll 4
        for (int i = from + g; i < to; i += 32) s += partial[(size_t)i * D + ch];
    runs[c][g] = s;
    __syncthreads();
    s = row_sum<32>(runs[g][c]);
    if (c == 0 && blockIdx.x * 32 + g < D) out[blockIdx.x * 32 + g] = s;
}

template <typename T, int D, int VEC, bool IL>
cudaError_t run(const QkRopeArgs& a, float* ws, cudaStream_t s) {
    const long long blocks = (a.tokens + WARPS - 1) / WARPS;
    // blocks that run at once (three an SM, backwards two), shared out by the work a token is: a warp's passes over its
    // heads, and about one and a half more for its angles
    const int most = a.dq ? QK_ROPE_BLOCKS : 148 * 3;
    const auto work = [](int heads) { return 2ll * ((heads + RowLayout<D, VEC>::RPW - 1) / RowLayout<D, VEC>::RPW) + 3; };
    int q_blocks = (int)(most * work(a.Hq) / (work(a.Hq) + work(a.Hk)));
    q_blocks = q_blocks < 1 ? 1 : q_blocks > most - 1 ? most - 1 : q_blocks;
    int k_blocks = most - q_blocks;
    q_blocks = (int)(blocks < q_blocks ? blocks : q_blocks);
    k_blocks = (int)(blocks < k_blocks ? blocks : k_blocks);
    if (!a.dq) {
        // few tokens: their heads over several warps, as long as there are SMs without work and rows to share (1 to 64 tokens
        // of 16 + 4 heads: 4.3 us in a replayed graph, 6.3 with a token's heads in one warp; from 256 tokens on the same)
        const int rows = ((a.Hq > a.Hk ? a.Hq : a.Hk) + RowLayout<D, VEC>::RPW - 1) / RowLayout<D, VEC>::RPW;
        const long long want = (148 + 2 * blocks - 1) / (2 * blocks);
        const int parts = (int)(want < rows ? want : rows);
        TraceScope trace(K_QK_ROPE, s);
        qk_rope_fwd_kernel<T, D, VEC, IL><<<dim3(q_blocks + k_blocks, parts), 32 * WARPS, 0, s>>>(a, q_blocks);
        return cudaGetLastError();
    }
    const bool weights = a.norm && (a.dq_weight || a.dk_weight);
    {
        TraceScope trace(K_QK_ROPE_BWD, s);
        qk_rope_bwd_kernel<T, D, VEC, IL><<<q_blocks + k_blocks, 32 * WARPS, 0, s>>>(a, q_blocks, weights ? ws : nullptr);
    }
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !weights) return e;
    TraceScope trace(K_QK_ROPE_BWD, s);
    qk_rope_weights_kernel<<<dim3((D + 31) / 32, 2), 1024, 0, s>>>(ws, q_blocks, q_blocks + k_blocks, D, a.dq_weight, a.dk_weight);
    return cudaGetLastError();
}
template <typename T, int D>
cudaError_t run_d(const QkRopeArgs& a, float* ws, cudaStream_t s) {
    // as many pairs at a time as 16 bytes hold where the pairs divide so, else four, else one. 4 x 4096 tokens of 16 + 4 heads
    // of 128, forward / backward in us: bf16 64 pairs (eight) 38 / 63, 60 pairs (four) 47 / 63, 61 pairs (one) 78 / 121;
    // fp32 60 pairs (four) 74 / 123, 61 pairs (one) 100 / 167.
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

cudaError_t qk_rope_error_word(unsigned int** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_rope_error);
}

}  // namespace gdn2

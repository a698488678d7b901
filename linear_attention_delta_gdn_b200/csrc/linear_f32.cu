// linear_f32.cu -- linear attention with a decay per head in 32-bit precision: forward and backward over whole
// sequences, in chunks of 64 tokens that run in parallel.
//
// Three launches (linear.cuh has the pass they compute):
//   1. chunk_states_kernel  per chunk, the state its tokens alone leave at its end, sum_j a^{C-1-j} k_j v_j^T (the
//                           backward also at its start, sum_i a^{i+1} q_i dout_i^T)
//   2. join_states_kernel   per head, the running state over the chunks: every chunk's start (end) state in place of
//                           its own contribution, and the final state
//   3. chunk_out_kernel     per chunk, the outputs: rows of (X Y^T * decay) Z + a^. X R with R the chunk's state
// The backward's dq, dk and dv are three such passes over two sets of states.
//
// The products run on tensor cores with every 32-bit operand split into two tf32 terms, x = big + small (11 + 11
// significant bits): big big + big small + small big leaves out terms below 2^-22, about what 32-bit rounding of a
// long sum costs, where plain tf32 operands would leave 2^-11. Sums are 32-bit.
//
// This is the path for checks of a model's numerics; its work is the products' (three mma.sync for one, and the splitting
// of each operand, 47% of the issue slots in chunk_out_kernel), its time that of the launches where there are few tokens:
// training on 2 x 1001 tokens, 4 heads of 64, takes 59 us in six launches, 2 x 13 in the outputs of one pass. 4 x 4096
// tokens of 16 heads of 128 take 1190 us forward and 2890 backward, where their bytes would take 82 and 164.
#include <cuda_runtime.h>

#include "chunk_common.cuh"
#include "internal.h"
#include "linear.cuh"

namespace gdn2 {
namespace {

using linear::Seqs;

__device__ unsigned int g_linear32_error;

constexpr int C32 = 64;     // tokens of a chunk
constexpr int NT32 = 256;   // threads of a block

// A 32-bit value as two tf32 terms. An infinity has no remainder.
__device__ __forceinline__ void split(float x, uint32_t* big, uint32_t* small) {
    *big = chunk::to_tf32(x);
    const float b = __uint_as_float(*big);
    *small = chunk::to_tf32(fabsf(b) < __int_as_float(0x7f800000) ? x - b : 0.f);
}

// How the 8 warps of a block share an M x N product: WM x WN warps, each MT x NT tiles of 16 x 8.
template <int M, int N>
struct WarpTiles {
    static constexpr int MALL = M / 16, NALL = N / 8;
    static constexpr int WM = MALL >= 8 ? 4 : MALL >= 2 ? (NALL >= 4 ? 2 : (MALL < 4 ? MALL : 4)) : 1;
    static constexpr int WN = (8 / WM) < NALL ? 8 / WM : NALL;
    static constexpr int MT = MALL / WM, NT = NALL / WN;
    static_assert(MT * WM == MALL && NT * WN == NALL, "tiles must divide");
};

// acc += A B for this warp's tiles; a(m, k) and b(k, n) give the operands' elements. Eight products a time are summed by
// the tensor core from zero and added to acc in 32 bits: its own accumulation cuts bits off instead of rounding, which
// over a long sum would add up.
template <int M, int N, int K, typename FA, typename FB>
__device__ __forceinline__ void warp_gemm(float (&acc)[WarpTiles<M, N>::MT][WarpTiles<M, N>::NT][4], FA a, FB b) {
    using W = WarpTiles<M, N>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (warp >= W::WM * W::WN) return;
    const int m0 = (warp / W::WN) * (16 * W::MT), n0 = (warp % W::WN) * (8 * W::NT);
#pragma unroll 2
    for (int k0 = 0; k0 < K; k0 += 8) {
        uint32_t ab[W::MT][4], as[W::MT][4];
#pragma unroll
        for (int i = 0; i < W::MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                split(a(m0 + 16 * i + g + 8 * (e & 1), k0 + t + 4 * (e >> 1)), &ab[i][e], &as[i][e]);
#pragma unroll
        for (int j = 0; j < W::NT; ++j) {
            uint32_t bb[2], bs[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) split(b(k0 + t + 4 * e, n0 + 8 * j + g), &bb[e], &bs[e]);
#pragma unroll
            for (int i = 0; i < W::MT; ++i) {
                float d[4] = {};
                chunk::mma_tf32_16x8x8(d, as[i][0], as[i][1], as[i][2], as[i][3], bb[0], bb[1]);
                chunk::mma_tf32_16x8x8(d, ab[i][0], ab[i][1], ab[i][2], ab[i][3], bs[0], bs[1]);
                chunk::mma_tf32_16x8x8(d, ab[i][0], ab[i][1], ab[i][2], ab[i][3], bb[0], bb[1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] += d[e];
            }
        }
    }
}

// Calls f(row, column, acc element) for the elements of this warp's tiles.
template <int M, int N, typename F>
__device__ __forceinline__ void each_element(float (&acc)[WarpTiles<M, N>::MT][WarpTiles<M, N>::NT][4], F f) {
    using W = WarpTiles<M, N>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (warp >= W::WM * W::WN) return;
    const int m0 = (warp / W::WN) * (16 * W::MT), n0 = (warp % W::WN) * (8 * W::NT);
#pragma unroll
    for (int i = 0; i < W::MT; ++i)
#pragma unroll
        for (int j = 0; j < W::NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) f(m0 + 16 * i + g + 8 * (e >> 1), n0 + 8 * j + 2 * t + (e & 1), acc[i][j][e]);
}

// One chunk's rows of a token tensor on their way into shared memory, zeros behind the chunk's last token (the rows
// there may be another sequence's).
template <int D, int LD>
__device__ __forceinline__ void load_rows(float* dst, const void* src, long long row0, int valid, int H, int h) {
    constexpr int PER = D / 4;
    for (int x = threadIdx.x; x < C32 * PER; x += NT32) {
        const int r = x / PER, p = x % PER;
        if (r < valid)
            tc::cp_async16_cg(dst + r * LD + 4 * p, static_cast<const float*>(src) + ((size_t)(row0 + r) * H + h) * D + 4 * p);
        else
            *reinterpret_cast<float4*>(dst + r * LD + 4 * p) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
}
// A matrix of R rows of D, the same way.
template <int R, int D, int LD>
__device__ __forceinline__ void load_state(float* dst, const float* src) {
    constexpr int PER = D / 4;
    for (int x = threadIdx.x; x < R * PER; x += NT32) tc::cp_async16_cg(dst + (x / PER) * LD + 4 * (x % PER), src + 4 * x);
}
// How a call's chunk states lie: a sequence has nc chunks at most, a head's states one behind the other ([N, H, NC]); or, by
// row, packed sequences' in the order of their tokens ([slot, H]), so that they take the room of the tokens and not of N
// sequences of the longest one. Sequence n's slots start at row0 / 64 + n: its ceil(len / 64) chunks end in front of
// (row0 + len) / 64 + n + 1, where the next one's start.
struct Chunks {
    int nc, by_row;
    long long total;   // states
};
__device__ __forceinline__ long long state_index(const Seqs& s, const Chunks& k, int n, int h, long long begin, int c) {
    return k.by_row ? (begin / C32 + n + c) * s.H + h : ((long long)n * s.H + h) * k.nc + c;
}
struct Unit {
    int n, h, c, len, valid;
    long long row0, state;   // first token row; index of the chunk's state
};
// Blocks are (sequence, head, chunk), chunk fastest. False for a chunk behind its sequence's end.
__device__ __forceinline__ bool unit_of(const Seqs& s, const Chunks& k, Unit* u) {
    const int x = blockIdx.x;
    u->c = x % k.nc;
    u->h = (x / k.nc) % s.H;
    u->n = x / k.nc / s.H;
    long long begin;
    u->len = linear::seq_span(s, u->n, &begin, &g_linear32_error);
    u->valid = min(C32, u->len - u->c * C32);
    u->row0 = begin + (long long)u->c * C32;
    u->state = state_index(s, k, u->n, u->h, begin, u->c);
    return u->valid > 0 && GDN2_IN(g_linear32_error, u->state >= 0 && u->state < k.total);
}

struct StateJob {
    const void *y, *z;
    float* states;       // [state index, Dk, Dv]
    const float* start;  // [N, H, Dk, Dv] or null
    float* end;          // or null
    int rev;
};
struct StateJobs {
    StateJob job[2];
};

template <int DK, int DV>
__global__ void __launch_bounds__(NT32) chunk_states_kernel(Seqs s, Chunks k, const float* __restrict__ log_decay, StateJobs jobs) {
    constexpr int LY = DK + 8, LZ = DV + 8;   // 8-column shift a row: the k-major fragment reads meet no bank twice
    extern __shared__ float sm[];
    float *Y = sm, *Z = sm + C32 * LY;
    const StateJob& job = jobs.job[blockIdx.y];
    Unit u;
    if (!unit_of(s, k, &u)) return;
    const float l2 = linear::log2_decay(log_decay, u.h);
    load_rows<DK, LY>(Y, job.y, u.row0, u.valid, s.H, u.h);
    load_rows<DV, LZ>(Z, job.z, u.row0, u.valid, s.H, u.h);
    __shared__ float f[C32];
    if (threadIdx.x < C32) {
        const int j = threadIdx.x;
        f[j] = j < u.valid ? linear::decay_pow(l2, job.rev ? j + 1 : u.valid - 1 - j) : 0.f;
    }
    tc::cp_async_wait_all();
    __syncthreads();
    float acc[WarpTiles<DK, DV>::MT][WarpTiles<DK, DV>::NT][4] = {};
    warp_gemm<DK, DV, C32>(acc, [&](int m, int k) { return Y[k * LY + m]; }, [&](int k, int n) { return Z[k * LZ + n] * f[k]; });
    float* out = job.states + (size_t)u.state * DK * DV;
    each_element<DK, DV>(acc, [&](int m, int n, float x) { out[m * DV + n] = x; });
}

// One thread per state element and head: the chunks in order, each contribution replaced by the state in front of it.
__global__ void __launch_bounds__(256) join_states_kernel(Seqs s, Chunks k, const float* __restrict__ log_decay, StateJobs jobs) {
    const StateJob& job = jobs.job[blockIdx.y];
    const int dd = s.Dk * s.Dv;
    const int per = dd / 256;
    const int head = blockIdx.x / per, e = (blockIdx.x % per) * 256 + threadIdx.x;
    const int n = head / s.H, h = head % s.H;
    long long begin;
    const int len = linear::seq_span(s, n, &begin, &g_linear32_error);
    const float l2 = linear::log2_decay(log_decay, h);
    int mine = linear::pieces(len, C32);
    if (mine && !GDN2_IN(g_linear32_error, mine <= k.nc && state_index(s, k, n, h, begin, mine - 1) < k.total)) mine = 0;
    float S = job.start ? job.start[(size_t)head * dd + e] : 0.f;
    float* st = job.states + (size_t)state_index(s, k, n, h, begin, 0) * dd + e;
    const size_t step = (size_t)dd * (k.by_row ? s.H : 1);   // from a chunk's state to the next one's
    const float whole = linear::decay_pow(l2, C32), last = linear::decay_pow(l2, len - (mine - 1) * C32);
    constexpr int AHEAD = 8;   // loads in flight a thread
    for (int c0 = 0; c0 < mine; c0 += AHEAD) {
        float x[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int c = job.rev ? mine - 1 - (c0 + i) : c0 + i;
            x[i] = c0 + i < mine ? st[c * step] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            if (c0 + i >= mine) break;
            const int c = job.rev ? mine - 1 - (c0 + i) : c0 + i;
            st[c * step] = S;
            S = fmaf(c == mine - 1 ? last : whole, S, x[i]);
        }
    }
    if (job.end) job.end[(size_t)head * dd + e] = S;
}

struct OutJob {
    const void *x, *y, *z;
    const float* states;
    void* out;
    int rev, transposed;   // transposed: the state is read as [DZ][DR]
};
struct OutJobs {
    OutJob job[3];
};

// Shared memory of a block: all operands at once, so that every load is under way from the start. P takes the place of Y.
template <int DR, int DZ>
struct OutTiles {
    static constexpr int LX = DR + 4, LZ = DZ + 8, LP = C32 + 4;   // shifts a row: fragment reads meet no bank twice
    static constexpr int Y = C32 * LX, Z = Y + C32 * (LX > LP ? LX : LP), S = Z + C32 * LZ;
    static constexpr int FLOATS = S + (DR * LZ > DZ * LX ? DR * LZ : DZ * LX);
};

template <int DR, int DZ>
__global__ void __launch_bounds__(NT32) chunk_out_kernel(Seqs s, Chunks k, const float* __restrict__ log_decay, OutJobs jobs) {
    using L = OutTiles<DR, DZ>;
    constexpr int LX = L::LX, LZ = L::LZ, LP = L::LP;
    extern __shared__ float sm[];
    float *X = sm, *Y = sm + L::Y, *Z = sm + L::Z, *S = sm + L::S, *P = Y;
    __shared__ float pw[C32 + 1];
    const OutJob& job = jobs.job[blockIdx.y];
    Unit u;
    if (!unit_of(s, k, &u)) return;
    const float l2 = linear::log2_decay(log_decay, u.h);
    const float* state = job.states + (size_t)u.state * DR * DZ;
    load_rows<DR, LX>(X, job.x, u.row0, u.valid, s.H, u.h);
    load_rows<DR, LX>(Y, job.y, u.row0, u.valid, s.H, u.h);
    tc::cp_async_commit();
    if (job.transposed)
        load_state<DZ, DR, LX>(S, state);
    else
        load_state<DR, DZ, LZ>(S, state);
    load_rows<DZ, LZ>(Z, job.z, u.row0, u.valid, s.H, u.h);
    tc::cp_async_commit();
    if (threadIdx.x <= C32) pw[threadIdx.x] = linear::decay_pow(l2, threadIdx.x);
    tc::cp_async_wait_but1();
    __syncthreads();
    float p[WarpTiles<C32, C32>::MT][WarpTiles<C32, C32>::NT][4] = {};
    warp_gemm<C32, C32, DR>(p, [&](int m, int k) { return X[m * LX + k]; }, [&](int k, int n) { return Y[n * LX + k]; });
    tc::cp_async_wait_all();
    __syncthreads();
    each_element<C32, C32>(p, [&](int m, int n, float x) {
        const int far = job.rev ? n - m : m - n;
        P[m * LP + n] = far >= 0 ? x * pw[far] : 0.f;
    });
    float acc[WarpTiles<C32, DZ>::MT][WarpTiles<C32, DZ>::NT][4] = {};
    if (job.transposed)
        warp_gemm<C32, DZ, DR>(acc, [&](int m, int k) { return X[m * LX + k]; }, [&](int k, int n) { return S[n * LX + k]; });
    else
        warp_gemm<C32, DZ, DR>(acc, [&](int m, int k) { return X[m * LX + k]; }, [&](int k, int n) { return S[k * LZ + n]; });
    each_element<C32, DZ>(acc, [&](int m, int, float& x) { x *= m < u.valid ? pw[job.rev ? u.valid - 1 - m : m + 1] : 0.f; });
    __syncthreads();
    warp_gemm<C32, DZ, C32>(acc, [&](int m, int k) { return P[m * LP + k]; }, [&](int k, int n) { return Z[k * LZ + n]; });
    float* out = static_cast<float*>(job.out);
    each_element<C32, DZ>(acc, [&](int m, int n, float x) {
        if (m < u.valid) out[((size_t)(u.row0 + m) * s.H + u.h) * DZ + n] = x;
    });
}

// The smaller of the two layouts: by row, sequences of much the same length would take more.
Chunks chunks_of(const Seqs& s, bool packed) {
    const int nc = linear::pieces(s.T, C32);
    const long long by_row = s.Ttot / C32 + s.N, by_sequence = (long long)s.N * nc;
    const bool rows = packed && by_row < by_sequence;
    return Chunks{nc, rows, s.H * (rows ? by_row : by_sequence)};
}

template <int DK, int DV>
cudaError_t states(const LinearArgs& a, const Chunks& k, const StateJobs& jobs, int n, cudaStream_t s) {
    const int smem = (int)sizeof(float) * C32 * (DK + 8 + DV + 8);
    cudaError_t e = cudaFuncSetAttribute(chunk_states_kernel<DK, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    TraceScope trace(K_LINEAR_STATES, s);
    chunk_states_kernel<DK, DV><<<dim3(a.seq.N * a.seq.H * k.nc, n), NT32, smem, s>>>(a.seq, k, a.log_decay, jobs);
    return cudaGetLastError();
}
template <int DR, int DZ>
cudaError_t outputs(const LinearArgs& a, const Chunks& k, const OutJobs& jobs, int n, cudaStream_t s) {
    const int smem = (int)sizeof(float) * OutTiles<DR, DZ>::FLOATS;
    cudaError_t e = cudaFuncSetAttribute(chunk_out_kernel<DR, DZ>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    TraceScope trace(K_LINEAR_OUT, s);
    chunk_out_kernel<DR, DZ><<<dim3(a.seq.N * a.seq.H * k.nc, n), NT32, smem, s>>>(a.seq, k, a.log_decay, jobs);
    return cudaGetLastError();
}

template <int DK, int DV>
cudaError_t run(const LinearArgs& a, bool bwd, cudaStream_t s) {
    const Chunks k = chunks_of(a.seq, a.seq.cu != nullptr);
    const size_t set = (size_t)k.total * DK * DV;
    float* w = static_cast<float*>(a.ws);
    StateJobs sj{};
    int n = 0;
    sj.job[n++] = StateJob{a.k, a.v, w, a.S0, bwd ? nullptr : a.ST, 0};
    if (bwd) sj.job[n++] = StateJob{a.q, a.dout, w + set, a.dST, a.dS0, 1};
    cudaError_t e = k.nc ? states<DK, DV>(a, k, sj, n, s) : cudaSuccess;
    if (e != cudaSuccess) return e;
    {
        TraceScope trace(K_LINEAR_JOIN, s);
        join_states_kernel<<<dim3(a.seq.N * a.seq.H * (DK * DV / 256), n), 256, 0, s>>>(a.seq, k, a.log_decay, sj);
        if ((e = cudaGetLastError()) != cudaSuccess || !k.nc) return e;
    }
    OutJobs oj{};
    if (!bwd) {
        oj.job[0] = OutJob{a.q, a.k, a.v, w, a.o, 0, 0};
        return outputs<DK, DV>(a, k, oj, 1, s);
    }
    oj.job[0] = OutJob{a.dout, a.v, a.k, w, a.dq, 0, 1};
    oj.job[1] = OutJob{a.v, a.dout, a.q, w + set, a.dk, 1, 1};
    const OutJob dv{a.k, a.q, a.dout, w + set, a.dv, 1, 0};
    if constexpr (DK == DV) {   // one kernel shape: one launch
        oj.job[2] = dv;
        return outputs<DK, DV>(a, k, oj, 3, s);
    }
    if ((e = outputs<DV, DK>(a, k, oj, 2, s)) != cudaSuccess) return e;
    oj.job[0] = dv;
    return outputs<DK, DV>(a, k, oj, 1, s);
}

template <int DK>
cudaError_t run_dv(const LinearArgs& a, bool bwd, cudaStream_t s) {
    switch (a.seq.Dv) {
    case 16: return run<DK, 16>(a, bwd, s);
    case 32: return run<DK, 32>(a, bwd, s);
    case 64: return run<DK, 64>(a, bwd, s);
    default: return run<DK, 128>(a, bwd, s);
    }
}
cudaError_t run_dk(const LinearArgs& a, bool bwd, cudaStream_t s) {
    switch (a.seq.Dk) {
    case 16: return run_dv<16>(a, bwd, s);
    case 32: return run_dv<32>(a, bwd, s);
    case 64: return run_dv<64>(a, bwd, s);
    default: return run_dv<128>(a, bwd, s);
    }
}

}  // namespace

size_t linear32_workspace(const Seqs& s, bool packed, bool backward) {
    return (size_t)chunks_of(s, packed).total * s.Dk * s.Dv * sizeof(float) * (backward ? 2 : 1);
}

cudaError_t linear32_launch(const LinearArgs& a, bool bwd, cudaStream_t s) {
    return run_dk(a, bwd, s);
}

cudaError_t linear32_error_word(unsigned int** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_linear32_error);
}

}  // namespace gdn2

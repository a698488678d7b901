// linear_chunk.cu -- linear attention with a decay per head on tcgen05 tensor cores: bf16, chunks of 128 tokens.
//
// A pass (linear.cuh) walks the chunks of a head with the state carried on chip. Per chunk of 128 rows, with
// P_ij = (x_i . y_j) a^|i-j| on the causal side and f, g the powers that bring rows and state to the chunk's border:
//     out = diag(f) X R + P Z,        R' = a^C R + Y^T diag(g) Z
// A block owns 64 columns of Z (and of out and R), so a head of 128 is two blocks and 64 heads fill the GPU; X and Y
// are then read by both, the second time from L2. Products per chunk and block (tcgen05, M = 128, 32-bit TMEM):
//     A = X Y^T (N 128)    D = Y^T Zh + Y^T Zl (N 64)    O1 = X R (N 64)    O2 = P Z (N 64, P read from TMEM)
// The state R lives in registers of one warpgroup in 32 bits. D does not depend on it, so the only thing one chunk
// hands the next is R' = a^C R + D and its bf16 copy for O1.
//
// Roundings. P and the copy of R round to bf16 (2^-8 each at most): they feed out, which is bf16 itself. The state is
// a 32-bit result, so g_j z_j goes into D as two bf16 terms, hi and the rest: 2^-18, where one term would leave 2^-9
// in a state that every later token reads. Sums are 32-bit.
//
// Warps: 0 loads (TMA), 1 issues the MMAs; warpgroup 1 turns A into P; warpgroup 2 makes Zh and Zl; warpgroup 3 keeps
// the state and writes the outputs. A block takes work items (sequence, head, column slice, segment, pass) in turn and
// the warps run ahead of one another across items.
//
// Few heads: a sequence's chunks are cut into segments of whole chunks, each an item of its own. A first launch leaves
// the state that each segment's tokens alone make (k and v are read twice then); a segment's start is the sum of those
// before it, each under its decay.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "internal.h"
#include "linear.cuh"
#include "tc.cuh"

namespace gdn2 {
namespace {

using linear::Seqs;
using namespace tc;

__device__ unsigned int g_linear_error;

constexpr int CT = 128;         // tokens of a chunk
constexpr int SL = 64;          // columns of a slice
constexpr int NT = 512;         // threads of a block
constexpr int MAX_PASS = 3;

struct Pass {
    CUtensorMap x, y, z, out;
    const float* start;      // state in front of the first (behind the last) token, [N, H, Dk, Dv], or null
    float* end;              // the state at the other end, or null
    float* seg;              // the segments' own states, [N, H, seg, slice][SL][DRP], or null
    void* out_ptr;           // the tensor behind out, for a sequence's last, partial chunk
    int start_transposed;    // start is [DZ][DR]
    int rev;
};
struct Params {
    Pass pass[MAX_PASS];
    Seqs seq;
    const float* log_decay;
    int npass, dr, dz, slices;
    int nseg, cps;           // segments of a sequence at most, chunks of a segment
    long long items;
};

// One work item and the chunk range it walks.
struct Item {
    const Pass* p;
    int pass, n, h, slice, seg;
    long long row0;          // the sequence's first token row
    int len, nc, c0, c1;     // the sequence's length and chunks; this item's chunks
    float l2;                // log2 of the decay
    __device__ __forceinline__ int chunk(int i) const { return p->rev ? c1 - 1 - i : c0 + i; }
    __device__ __forceinline__ int valid(int c) const { return min(CT, len - c * CT); }
    __device__ __forceinline__ int count() const { return c1 - c0; }
};
template <bool STATES>
__device__ __forceinline__ Item item_of(const Params& p, long long x) {
    Item t;
    t.slice = (int)(x % p.slices); x /= p.slices;
    t.pass = (int)(x % p.npass); x /= p.npass;
    t.h = (int)(x % p.seq.H); x /= p.seq.H;
    t.n = (int)(x % p.seq.N);
    t.seg = (int)(x / p.seq.N);
    t.p = &p.pass[t.pass];
    t.len = linear::seq_span(p.seq, t.n, &t.row0, &g_linear_error);
    t.nc = (t.len + CT - 1) / CT;
    t.c0 = min(t.nc, t.seg * p.cps);
    t.c1 = min(t.nc, t.c0 + p.cps);
    if (STATES) {   // nothing comes behind the last segment (in front of the first one, backwards)
        const int last = (t.nc + p.cps - 1) / p.cps - 1;
        if (t.p->rev ? t.seg == 0 : t.seg >= last) t.c1 = t.c0;
    }
    t.l2 = linear::log2_decay(p.log_decay, t.h);
    return t;
}

template <int DRP, bool STATES>
struct Cfg {
    static constexpr uint32_t XB = STATES ? 0 : CT * DRP * 2;      // bytes of a row-operand tile
    static constexpr uint32_t YB = CT * DRP * 2;
    static constexpr uint32_t ZB = CT * SL * 2;
    static constexpr int STAGES = (DRP == 128 && !STATES) ? 2 : 3;
    static constexpr uint32_t SB = STATES ? 0 : DRP * SL * 2;      // bf16 copy of the state
    static constexpr uint32_t OB = STATES ? 0 : CT * SL * 2;       // output staging
    static constexpr uint32_t OFF_Y = STAGES * XB, OFF_Z = OFF_Y + STAGES * YB, OFF_ZH = OFF_Z + STAGES * ZB,
                              OFF_ZL = OFF_ZH + ZB, OFF_S = OFF_ZL + ZB, OFF_O = OFF_S + SB, TOTAL = OFF_O + OB;
    static constexpr uint32_t SMEM = TOTAL + 1024;                 // tiles start on 1024 bytes
    // TMEM columns: A (then P in its first half) twice, D twice, O1, O2
    static constexpr uint32_t T_A = 0, T_D = 256, T_O1 = 384, T_O2 = 448;
};

struct Bars {
    uint64_t full_x[3], full_y[3], full_z[3], empty_x[3], empty_y[3], empty_z[3];
    uint64_t a_full[2], a_free[2], p_full, z_full, d_full[2], d_free[2], s_full, s_free, o_full, o_free, drain;
};

// Waits by a whole warp: every lane has the same answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, phase));
    if (!ok) atomicOr(&g_linear_error, linear::ERR_WAIT);
    return ok;
}

// ------------------------------------------------------------ warp 0: loads

template <int DRP, bool STATES>
__device__ void load_tiles(const Params& p, unsigned char* sm, Bars& b) {
    using K = Cfg<DRP, STATES>;
    uint32_t ny = 0, nx = 0, nz = 0;   // tiles asked for so far, over all items
    bool ok = true;
    for (long long it = blockIdx.x; ok && it < p.items; it += gridDim.x) {
        const Item t = item_of<STATES>(p, it);
        for (int i = 0; i < t.count(); ++i) {
            const uint32_t s = ny % K::STAGES, ph = ((ny / K::STAGES) & 1) ^ 1;
            const int row = (int)(t.row0 + (long long)t.chunk(i) * CT);
            if (!(ok = mbar_wait(&b.empty_y[s], ph))) break;
            mbar_arrive_expect_tx(&b.full_y[s], K::YB);
#pragma unroll
            for (int c = 0; c < DRP / 64; ++c)
                tma_load_3d(sm + K::OFF_Y + s * K::YB + c * CT * 128, &t.p->y, 64 * c, t.h, row, &b.full_y[s]);
            ++ny;
            if (!STATES) {
                if (!(ok = mbar_wait(&b.empty_x[s], ph))) break;
                mbar_arrive_expect_tx(&b.full_x[s], K::XB);
#pragma unroll
                for (int c = 0; c < DRP / 64; ++c)
                    tma_load_3d(sm + s * K::XB + c * CT * 128, &t.p->x, 64 * c, t.h, row, &b.full_x[s]);
                ++nx;
            }
            if (!(ok = mbar_wait(&b.empty_z[s], ph))) break;
            mbar_arrive_expect_tx(&b.full_z[s], K::ZB);
            tma_load_3d(sm + K::OFF_Z + s * K::ZB, &t.p->z, t.slice * SL, t.h, row, &b.full_z[s]);
            ++nz;
        }
    }
    if (ok) return;   // every tile was waited for by those who read it
    atomicOr(&g_linear_error, linear::ERR_WAIT);
    // let the copies in flight land before the block gives up its shared memory: each stage's last one
    auto land = [](uint64_t* full, uint32_t asked) {
        for (uint32_t k = 1; k <= (uint32_t)K::STAGES && k <= asked; ++k)
            mbar_wait(&full[(asked - k) % K::STAGES], ((asked - k) / K::STAGES) & 1);
    };
    land(b.full_y, ny);
    land(b.full_x, nx);
    land(b.full_z, nz);
}

// ------------------------------------------------------------ warp 1: products

template <int DRP, bool STATES>
__device__ void issue_products(const Params& p, unsigned char* sm, uint32_t tm, Bars& b) {
    using K = Cfg<DRP, STATES>;
    const uint32_t base = smem_u32(sm);
    const uint32_t idA = idesc_bf16(128, 128, false, false), idD = idesc_bf16(DRP, SL, true, true),
                   idO = idesc_bf16(128, SL, false, true);
    const int kr = p.dr / 16;   // K steps over the row operand's real channels
    uint32_t n = 0;
    bool ok = true;
    for (long long x = blockIdx.x; ok && x < p.items; x += gridDim.x) {
        const Item t = item_of<STATES>(p, x);
        for (int i = 0; i < t.count(); ++i, ++n) {
            const uint32_t s = n % K::STAGES, ph = (n / K::STAGES) & 1, d = n & 1, dph = (n >> 1) & 1, one = n & 1;
            const uint32_t xt = base + s * K::XB, yt = base + K::OFF_Y + s * K::YB, zt = base + K::OFF_Z + s * K::ZB;
            const bool ragged = t.valid(t.chunk(i)) < CT;
            if (!(ok = mbar_wait(&b.full_y[s], ph))) break;
            // behind a sequence's end the tiles hold another's rows: warpgroup 2 clears them first
            if (ragged && !(ok = mbar_wait(&b.z_full, one))) break;
            if (!STATES) {
                if (!(ok = mbar_wait(&b.full_x[s], ph) && mbar_wait(&b.a_free[d], dph ^ 1))) break;
                tc_fence_after();
                for (int kk = 0; kk < kr; ++kk)
                    mma_bf16(tm + K::T_A + d * CT, desc_k(xt, CT, 0, kk), desc_k(yt, CT, 0, kk), idA, kk > 0);
                mma_commit(&b.a_full[d]);
            }
            if (!(ok = mbar_wait(&b.z_full, one) && mbar_wait(&b.d_free[d], dph ^ 1))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < CT / 16; ++kk)
                mma_bf16(tm + K::T_D + d * SL, desc_mn(yt, CT, 0, kk), desc_mn(base + K::OFF_ZH, CT, 0, kk), idD, kk > 0);
#pragma unroll
            for (int kk = 0; kk < CT / 16; ++kk)
                mma_bf16(tm + K::T_D + d * SL, desc_mn(yt, CT, 0, kk), desc_mn(base + K::OFF_ZL, CT, 0, kk), idD, 1);
            mma_commit(&b.d_full[d]);
            mma_commit(&b.empty_y[s]);
            if (STATES) {
                mma_commit(&b.empty_z[s]);
                continue;
            }
            if (!(ok = mbar_wait(&b.s_full, one) && mbar_wait(&b.o_free, one ^ 1))) break;
            tc_fence_after();
            for (int kk = 0; kk < kr; ++kk)
                mma_bf16(tm + K::T_O1, desc_k(xt, CT, 0, kk), desc_mn(base + K::OFF_S, DRP, 0, kk), idO, kk > 0);
            mma_commit(&b.s_free);
            mma_commit(&b.empty_x[s]);
            if (!(ok = mbar_wait(&b.full_z[s], ph) && mbar_wait(&b.p_full, one))) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < CT / 16; ++kk)
                mma_bf16_ts(tm + K::T_O2, tm + K::T_A + d * CT + 8 * kk, desc_mn(zt, CT, 0, kk), idO, kk > 0);
            mma_commit(&b.o_full);
            mma_commit(&b.a_free[d]);
            mma_commit(&b.empty_z[s]);
        }
    }
    if (!ok) atomicOr(&g_linear_error, linear::ERR_WAIT);
    // what was issued ends before TMEM is given back
    mma_commit(&b.drain);
    mbar_wait(&b.drain, 0);
}

// ------------------------------------------------------------ warpgroup 1: A -> P

// Row i = 32 w + lane against column blocks of 32. Off the diagonal block a^|i-j| is a row part times a column part,
// both with exponents >= 0 (border of the column block next to the diagonal); on it the power comes from a table.
template <int DRP>
__device__ void weigh_pairs(const Params& p, uint32_t tm, Bars& b, float* tab) {
    using K = Cfg<DRP, false>;
    const int w = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    uint32_t n = 0;
    for (long long x = blockIdx.x; x < p.items; x += gridDim.x) {
        const Item t = item_of<false>(p, x);
        const bool rev = t.p->rev;
        __syncwarp();
        tab[lane] = linear::decay_pow(t.l2, lane);   // this warp's own table of a^0 .. a^31
        __syncwarp();
        for (int i = 0; i < t.count(); ++i, ++n) {
            if (!warp_wait(&b.a_full[n & 1], (n >> 1) & 1)) return;
            tc_fence_after();
            const uint32_t ta = tm + K::T_A + (n & 1) * CT + ((uint32_t)(32 * w) << 16);
#pragma unroll
            for (int jb = 0; jb < 4; ++jb) {
                float v[32], o[16];
                if (rev ? jb < w : jb > w) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = 0.f;
                } else {
                    tmem_ld32(ta + 32 * jb, v);
                    tmem_wait_ld(v);
                    if (jb == w) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const int far = rev ? j - lane : lane - j;
                            v[j] = far >= 0 ? v[j] * tab[far & 31] : 0.f;
                        }
                    } else {
                        const float row = linear::decay_pow(t.l2, rev ? 32 * (jb - w) - lane : 32 * (w - jb) + lane - 31);
#pragma unroll
                        for (int j4 = 0; j4 < 8; ++j4) {
                            // column parts: a^(31-j) forwards, a^j backwards
                            const float4 c = *reinterpret_cast<const float4*>(tab + (rev ? 4 * j4 : 28 - 4 * j4));
                            v[4 * j4 + 0] *= row * (rev ? c.x : c.w);
                            v[4 * j4 + 1] *= row * (rev ? c.y : c.z);
                            v[4 * j4 + 2] *= row * (rev ? c.z : c.y);
                            v[4 * j4 + 3] *= row * (rev ? c.w : c.x);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __uint_as_float(pack_bf16x2(v[2 * j], v[2 * j + 1]));
                }
                // columns 16 jb .. of P lie in A's columns up to 32 jb + 31, which this warp has read
                tmem_st16(ta + 16 * jb, o);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&b.p_full);
        }
    }
}

// ------------------------------------------------------------ warpgroup 2: g_j z_j in two terms

template <int DRP, bool STATES>
__device__ void split_values(const Params& p, unsigned char* sm, Bars& b) {
    using K = Cfg<DRP, STATES>;
    const int j = threadIdx.x & 127;
    uint32_t n = 0;
    for (long long x = blockIdx.x; x < p.items; x += gridDim.x) {
        const Item t = item_of<STATES>(p, x);
        for (int i = 0; i < t.count(); ++i, ++n) {
            const uint32_t s = n % K::STAGES, ph = (n / K::STAGES) & 1;
            const int valid = t.valid(t.chunk(i));
            unsigned char* Z = sm + K::OFF_Z + s * K::ZB;
            unsigned char *Zh = sm + K::OFF_ZH, *Zl = sm + K::OFF_ZL;
            if (!warp_wait(&b.full_z[s], ph)) return;
            if (valid < CT && !warp_wait(&b.full_y[s], ph)) return;
            // Zh and Zl are free once the last chunk's D is done
            if (n > 0 && !warp_wait(&b.d_full[(n - 1) & 1], ((n - 1) >> 1) & 1)) return;
            if (j < valid) {
                const float g = linear::decay_pow(t.l2, t.p->rev ? j + 1 : valid - 1 - j);
#pragma unroll
                for (int c = 0; c < SL / 8; ++c) {
                    float v[8], r[8];
                    ld_row8(Z, CT, j, c, v);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] *= g;
                        r[e] = v[e] - __bfloat162float(__float2bfloat16_rn(v[e]));
                    }
                    st_row8(Zh, CT, j, c, v);
                    st_row8(Zl, CT, j, c, r);
                }
            } else {
                const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int c = 0; c < SL / 8; ++c) {
                    const uint32_t at = tile_chunk_off(CT, j, c);
                    *reinterpret_cast<uint4*>(Zh + at) = zero;
                    *reinterpret_cast<uint4*>(Zl + at) = zero;
                    *reinterpret_cast<uint4*>(Z + at) = zero;
                }
                for (int c = 0; c < DRP / 8; ++c)
                    *reinterpret_cast<uint4*>(sm + K::OFF_Y + s * K::YB + tile_chunk_off(CT, j, c)) = zero;
            }
            fence_async_smem();
            mbar_arrive(&b.z_full);
        }
    }
}

// ------------------------------------------------------------ warpgroup 3: the state, the outputs

// Start state of an item: row r of the slice's columns.
template <int DRP, bool STATES>
__device__ __forceinline__ void start_state(const Params& p, const Item& t, int r, bool real, float (&S)[SL]) {
#pragma unroll
    for (int j = 0; j < SL; ++j) S[j] = 0.f;
    if (STATES || !real) return;
    const Pass& q = *t.p;
    const size_t head = (size_t)t.n * p.seq.H + t.h;
    const int seg_tokens = p.cps * CT, nseg = (t.nc + p.cps - 1) / p.cps;
    if (q.start && r < p.dr) {
        // tokens between the sequence's end that the state stands at and this segment
        const long long away = q.rev ? max(0ll, t.len - (t.seg + 1ll) * seg_tokens) : (long long)t.seg * seg_tokens;
        const float f = linear::decay_pow(t.l2, (int)away);
        const float* src = q.start + head * p.dr * p.dz;
        if (q.start_transposed) {
#pragma unroll
            for (int j = 0; j < SL; ++j)
                if (t.slice * SL + j < p.dz) S[j] = f * src[(size_t)(t.slice * SL + j) * p.dr + r];
        } else {
#pragma unroll
            for (int j = 0; j < SL; j += 4)
                if (t.slice * SL + j < p.dz) {
                    const float4 v = *reinterpret_cast<const float4*>(src + (size_t)r * p.dz + t.slice * SL + j);
                    S[j] = f * v.x; S[j + 1] = f * v.y; S[j + 2] = f * v.z; S[j + 3] = f * v.w;
                }
        }
    }
    const int from = q.rev ? t.seg + 1 : 0, to = q.rev ? nseg : t.seg;
    for (int o = from; o < to; ++o) {
        const float f = linear::decay_pow(t.l2, (q.rev ? o - t.seg - 1 : t.seg - 1 - o) * seg_tokens);
        const float* src = q.seg + ((head * p.nseg + o) * p.slices + t.slice) * (size_t)(SL * DRP) + r;
#pragma unroll
        for (int j = 0; j < SL; ++j) S[j] = fmaf(f, src[j * DRP], S[j]);
    }
}

template <int DRP, bool STATES>
__device__ void carry_and_write(const Params& p, unsigned char* sm, uint32_t tm, Bars& b) {
    using K = Cfg<DRP, STATES>;
    const int w = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, tid = threadIdx.x & 127;
    // accumulator rows: 128 in lanes 0..127; 64 in the first 16 lanes of each quarter
    const int r = DRP == 128 ? 32 * w + lane : 16 * w + (lane & 15);
    const bool real = DRP == 128 || lane < 16;
    const uint32_t quarter = (uint32_t)(32 * w) << 16;
    unsigned char *Sb = sm + K::OFF_S, *Ob = sm + K::OFF_O;
    uint32_t n = 0;
    float S[SL];
    auto copy_state = [&]() {   // the bf16 copy that the next O1 reads
        if (real)
#pragma unroll
            for (int c = 0; c < SL / 8; ++c) st_row8(Sb, DRP, r, c, S + 8 * c);
        fence_async_smem();
        mbar_arrive(&b.s_full);
    };
    bool ok = true;
    for (long long x = blockIdx.x; ok && x < p.items; x += gridDim.x) {
        const Item t = item_of<STATES>(p, x);
        const bool last_seg = t.p->rev ? t.seg == 0 : t.seg == max(0, (t.nc + p.cps - 1) / p.cps - 1);
        const bool writes_end = !STATES && t.p->end && last_seg;
        if (t.count() == 0 && !writes_end) continue;
        start_state<DRP, STATES>(p, t, r, real, S);
        if (!STATES && t.count()) {
            if (n > 0) ok = warp_wait(&b.s_free, (n - 1) & 1);
            if (ok) copy_state();
        }
        for (int i = 0; i < t.count(); ++i, ++n) {
            const int c = t.chunk(i), valid = t.valid(c);
            const uint32_t d = n & 1, dph = (n >> 1) & 1;
            ok = ok && warp_wait(&b.d_full[d], dph);
            if (ok) {
                tc_fence_after();
                const float aC = linear::decay_pow(t.l2, valid);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float D[32];
                    tmem_ld32(tm + K::T_D + d * SL + 32 * h + quarter, D);
                    tmem_wait_ld(D);
#pragma unroll
                    for (int j = 0; j < 32; ++j) S[32 * h + j] = fmaf(aC, S[32 * h + j], D[j]);
                }
                tc_fence_before();
                mbar_arrive(&b.d_free[d]);
                if (!STATES && i + 1 < t.count()) {
                    ok = warp_wait(&b.s_free, n & 1);
                    if (ok) copy_state();
                }
            }
            if (STATES) {
                if (!ok) break;
                continue;
            }
            ok = ok && warp_wait(&b.o_full, n & 1);
            const int row = (int)(t.row0 + (long long)c * CT);
            if (tid == 0) bulk_wait_read();   // the staging tile's last store has been read
            ok = !named_sync_or(1, 128, !ok);
            if (!ok) break;
            tc_fence_after();
            {
                const int orow = 32 * w + lane;
                const float f = linear::decay_pow(t.l2, t.p->rev ? max(0, valid - 1 - orow) : orow + 1);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float o1[16], o2[16];
                    tmem_ld16(tm + K::T_O1 + 16 * h + quarter, o1);
                    tmem_ld16(tm + K::T_O2 + 16 * h + quarter, o2);
                    tmem_wait_ld(o1, o2);
#pragma unroll
                    for (int j = 0; j < 16; ++j) o2[j] = fmaf(f, o1[j], o2[j]);
                    st_row8(Ob, CT, orow, 2 * h, o2);
                    st_row8(Ob, CT, orow, 2 * h + 1, o2 + 8);
                }
                tc_fence_before();
                mbar_arrive(&b.o_free);
            }
            fence_async_smem();
            named_sync(1, 128);
            if (valid == CT) {
                if (tid == 0) {
                    tma_store_3d(&t.p->out, t.slice * SL, t.h, row, Ob);
                    bulk_commit();
                }
            } else {   // the rows behind the end are not this sequence's: 16-byte pieces of the real rows
                __nv_bfloat16* out = static_cast<__nv_bfloat16*>(t.p->out_ptr);
                for (int e = tid; e < valid * (SL / 8); e += 128) {
                    const int rr = e / (SL / 8), cc = e % (SL / 8);
                    if (t.slice * SL + 8 * cc < p.dz)
                        *reinterpret_cast<uint4*>(out + ((size_t)(row + rr) * p.seq.H + t.h) * p.dz + t.slice * SL + 8 * cc) =
                            *reinterpret_cast<const uint4*>(Ob + tile_chunk_off(CT, rr, cc));
                }
            }
        }
        if (!ok || !real) continue;
        if (STATES) {
            float* dst = t.p->seg + ((((size_t)t.n * p.seq.H + t.h) * p.nseg + t.seg) * p.slices + t.slice) * (size_t)(SL * DRP) + r;
#pragma unroll
            for (int j = 0; j < SL; ++j) dst[j * DRP] = S[j];
        } else if (writes_end && r < p.dr) {
            float* dst = t.p->end + (((size_t)t.n * p.seq.H + t.h) * p.dr + r) * p.dz + t.slice * SL;
#pragma unroll
            for (int j = 0; j < SL; j += 4)
                if (t.slice * SL + j < p.dz) *reinterpret_cast<float4*>(dst + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        }
    }
    if (tid == 0) bulk_wait_all();
    __syncwarp();
}

template <int DRP, bool STATES>
__global__ void __launch_bounds__(NT, 1) linear_chunk_kernel(const __grid_constant__ Params p) {
    using K = Cfg<DRP, STATES>;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    __shared__ Bars b;
    __shared__ uint32_t tmem;
    __shared__ __align__(16) float tab[4][32];
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < 3; ++s) {
            mbar_init(&b.full_x[s], 1); mbar_init(&b.full_y[s], 1); mbar_init(&b.full_z[s], 1);
            mbar_init(&b.empty_x[s], 1); mbar_init(&b.empty_y[s], 1); mbar_init(&b.empty_z[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.d_full[i], 1); mbar_init(&b.d_free[i], 128);
            mbar_init(&b.a_full[i], 1); mbar_init(&b.a_free[i], 1);
        }
        mbar_init(&b.p_full, 128); mbar_init(&b.z_full, 128);
        mbar_init(&b.s_full, 128); mbar_init(&b.s_free, 1);
        mbar_init(&b.o_full, 1); mbar_init(&b.o_free, 128);
        mbar_init(&b.drain, 1);
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc(&tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem;
    if (warp == 0) {
        if (threadIdx.x == 0) load_tiles<DRP, STATES>(p, sm, b);
        __syncwarp();
    } else if (warp == 1) {
        if (threadIdx.x == 32) issue_products<DRP, STATES>(p, sm, tm, b);
        __syncwarp();
    } else if (warp >= 4 && warp < 8) {
        if constexpr (!STATES) weigh_pairs<DRP>(p, tm, b, tab[warp & 3]);
    } else if (warp >= 8 && warp < 12) split_values<DRP, STATES>(p, sm, b);
    else if (warp >= 12) carry_and_write<DRP, STATES>(p, sm, tm, b);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tm, 512);
}

CUresult encode(CUtensorMap* map, const void* ptr, const Seqs& s, int D) {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    if (!fn) return CUDA_ERROR_NOT_FOUND;
    // [rows, H, D] in boxes of 128 rows x 1 head x 64 channels; channels behind D and rows behind the tensor read as 0
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)s.H, (cuuint64_t)s.Ttot};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.H * D * 2};
    cuuint32_t box[3] = {64, 1, CT}, step[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// Blocks that run at once. Without a device (the workspace is sized on hosts too) a B200's.
int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
        (void)cudaGetLastError();
        n = 148;
    }
    return n;
}

struct Cut {
    int nseg, cps;
};
// How a sequence's chunks are cut. Time in chunks of one block: the fullest block's chunks, 2 more for each item's
// start and end, and for more than one segment the launch before (its chunks cost about 0.6 of a main one's, and the
// launch itself 3).
Cut choose_cut(const Seqs& s, int heads) {
    const int nc = (s.T + CT - 1) / CT, nsm = sm_count();
    Cut best{1, std::max(nc, 1)};
    double best_time = 1e30;
    for (int r = 1; r <= 64 && r <= std::max(nc, 1); ++r) {
        const int cps = std::max(1, (nc + r - 1) / r), nseg = std::max(1, (nc + cps - 1) / cps);
        const double waves = (double)(((long long)heads * nseg + nsm - 1) / nsm);
        const double t = waves * (cps + 2) + (nseg > 1 ? waves * (0.6 * cps + 2) + 3 : 0.0);
        if (t < best_time) {
            best_time = t;
            best = Cut{nseg, cps};
        }
    }
    return best;
}

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
int padded(int d) { return d > 64 ? 128 : 64; }
int slices_of(int dz) { return (dz + SL - 1) / SL; }
size_t seg_bytes(const Seqs& s, const Cut& c, int dr, int dz) {
    return c.nseg > 1 ? align256((size_t)s.N * s.H * c.nseg * slices_of(dz) * SL * padded(dr) * sizeof(float)) : 0;
}
size_t state_bytes(const Seqs& s) { return align256((size_t)s.N * s.H * s.Dk * s.Dv * sizeof(float)); }

// The passes of one launch: the same row and value sizes.
struct Group {
    int npass, dr, dz;
    Pass pass[MAX_PASS];
};

template <int DRP, bool STATES>
cudaError_t launch(const Params& p, cudaStream_t s) {
    using K = Cfg<DRP, STATES>;
    cudaError_t e = cudaFuncSetAttribute(linear_chunk_kernel<DRP, STATES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)K::SMEM);
    if (e != cudaSuccess) return e;
    const long long grid = std::min<long long>(p.items, sm_count());
    TraceScope trace(STATES ? K_LINEAR_SEGMENT : K_LINEAR_CHUNK, s);
    linear_chunk_kernel<DRP, STATES><<<(unsigned)grid, NT, K::SMEM, s>>>(p);
    return cudaGetLastError();
}

cudaError_t run_group(const LinearArgs& a, const Group& g, const Cut& cut, cudaStream_t s) {
    Params p{};
    for (int i = 0; i < g.npass; ++i) p.pass[i] = g.pass[i];
    p.seq = a.seq;
    p.log_decay = a.log_decay;
    p.npass = g.npass;
    p.dr = g.dr;
    p.dz = g.dz;
    p.slices = slices_of(g.dz);
    p.nseg = cut.nseg;
    p.cps = cut.cps;
    p.items = (long long)cut.nseg * a.seq.N * a.seq.H * g.npass * p.slices;
    cudaError_t e = cudaSuccess;
    if (cut.nseg > 1) e = padded(g.dr) == 128 ? launch<128, true>(p, s) : launch<64, true>(p, s);
    if (e != cudaSuccess) return e;
    return padded(g.dr) == 128 ? launch<128, false>(p, s) : launch<64, false>(p, s);
}

// Passes of the forward (1) or the backward (3), as (row, value) sizes.
int heads_of(const Seqs& s, bool bwd) {
    const int k = slices_of(s.Dk), v = slices_of(s.Dv);
    return s.N * s.H * (bwd ? 2 * k + v : v);
}

}  // namespace

size_t linear_chunk_workspace(const Seqs& s, bool bwd) {
    if (s.T == 0) return 0;
    const Cut c = choose_cut(s, heads_of(s, bwd));
    const size_t keep = c.nseg > 1 ? state_bytes(s) : 0;   // a start state that the call's end state overwrites
    if (!bwd) return keep + seg_bytes(s, c, s.Dk, s.Dv);
    return keep + 2 * seg_bytes(s, c, s.Dv, s.Dk) + seg_bytes(s, c, s.Dk, s.Dv);
}

cudaError_t linear_chunk_launch(const LinearArgs& a, bool bwd, cudaStream_t s) {
    const Seqs& q = a.seq;
    if (q.T == 0) {   // no tokens: the state is handed on
        float* end = bwd ? a.dS0 : a.ST;
        const float* start = bwd ? a.dST : a.S0;
        const size_t bytes = (size_t)q.N * q.H * q.Dk * q.Dv * sizeof(float);
        if (!end || end == start) return cudaSuccess;
        return start ? cudaMemcpyAsync(end, start, bytes, cudaMemcpyDeviceToDevice, s) : cudaMemsetAsync(end, 0, bytes, s);
    }
    const Cut cut = choose_cut(q, heads_of(q, bwd));
    unsigned char* w = static_cast<unsigned char*>(a.ws);
    const float *S0 = a.S0, *dST = a.dST;
    if (cut.nseg > 1) {
        // every segment reads the start state, the last one writes the end state: in place needs a copy
        const float*& start = bwd ? dST : S0;
        if (start && start == (bwd ? a.dS0 : a.ST)) {
            cudaError_t e = cudaMemcpyAsync(w, start, (size_t)q.N * q.H * q.Dk * q.Dv * sizeof(float), cudaMemcpyDeviceToDevice, s);
            if (e != cudaSuccess) return e;
            start = reinterpret_cast<const float*>(w);
        }
        w += state_bytes(q);
    }
    auto seg = [&](int dr, int dz) {
        float* at = cut.nseg > 1 ? reinterpret_cast<float*>(w) : nullptr;
        w += seg_bytes(q, cut, dr, dz);
        return at;
    };
    bool good = true;
    auto pass = [&](const void* x, int dr, const void* y, const void* z, int dz, void* out, const float* start, float* end,
                    bool transposed, bool rev) {
        Pass p{};
        good = good && encode(&p.x, x, q, dr) == CUDA_SUCCESS && encode(&p.y, y, q, dr) == CUDA_SUCCESS &&
               encode(&p.z, z, q, dz) == CUDA_SUCCESS && encode(&p.out, out, q, dz) == CUDA_SUCCESS;
        p.start = start;
        p.end = end;
        p.seg = seg(dr, dz);
        p.out_ptr = out;
        p.start_transposed = transposed;
        p.rev = rev;
        return p;
    };
    const int Dk = q.Dk, Dv = q.Dv;
    if (!bwd) {
        Group g{1, Dk, Dv, {}};
        g.pass[0] = pass(a.q, Dk, a.k, a.v, Dv, a.o, S0, a.ST, false, false);
        return good ? run_group(a, g, cut, s) : cudaErrorInvalidValue;
    }
    const Pass dq = pass(a.dout, Dv, a.v, a.k, Dk, a.dq, S0, nullptr, true, false);
    const Pass dk = pass(a.v, Dv, a.dout, a.q, Dk, a.dk, dST, nullptr, true, true);
    const Pass dv = pass(a.k, Dk, a.q, a.dout, Dv, a.dv, dST, a.dS0, false, true);
    if (!good) return cudaErrorInvalidValue;
    // an end state over its start state is only safe once every pass that reads the start has run: dv's comes last
    Group both{2, Dv, Dk, {dq, dk}}, one{1, Dk, Dv, {dv}};
    if (Dk == Dv && (!a.dS0 || a.dS0 != dST)) {
        both.npass = 3;
        both.pass[2] = dv;
        return run_group(a, both, cut, s);
    }
    cudaError_t e = run_group(a, both, cut, s);
    return e != cudaSuccess ? e : run_group(a, one, cut, s);
}

cudaError_t linear_chunk_take_errors(unsigned int* bits) {
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_linear_error, sizeof(unsigned int));
    if (e != cudaSuccess) return e;
    const unsigned int zero = 0;
    return cudaMemcpyToSymbol(g_linear_error, &zero, sizeof(unsigned int));
}

}  // namespace gdn2

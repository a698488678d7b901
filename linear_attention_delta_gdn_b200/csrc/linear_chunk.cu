// linear_chunk.cu -- linear attention with a decay per head on tcgen05 tensor cores: bf16, chunks of 128 tokens.
//
// A pass (linear.cuh) walks the chunks of a head with the state carried on chip. Per chunk of 128 rows, with
// P_ij = (x_i . y_j) a^|i-j| on the causal side and f, g the powers that bring rows and state to the chunk's border:
//     out = diag(f) X R + P Z,        R' = a^C R + Y^T diag(g) Z
// A block owns 64 columns of Z (and of out and R), so a head of 128 is two blocks and 64 heads fill the GPU; X and Y
// are then read by both, the second time from L2. Products per chunk and block (tcgen05, M = 128, 32-bit TMEM):
//     A = X Y^T (N 128)    D = Y^T [Zh | Zl] (N 128)    O1 = X R (N 64)    O2 = P Z (N 64, P read from TMEM)
// The state R lives in registers of one warpgroup in 32 bits. D does not depend on it, so the only thing one chunk
// hands the next is R' = a^C R + D and its bf16 copy for O1.
//
// What bounds it: a chunk takes a block 1.7 to 1.9 us (3400 to 3700 cycles), for rows of 64 as for 128 and for one block as for 128 of
// them: the round trips between the roles. Its products are 1670 cycles of the tensor pipe alone (64 a K step at
// N 128, 48 at N 64 from shared memory, 32 from TMEM); the pairs' warpgroup works 2800 (P 1300 and outputs 1300), the
// values' 2200, the state's 1200; a chunk's tiles take 2400 from request to arrival, and X, held from its A to its O1 a
// chunk later, has two stages. Measured: 72 us for 4 x 4096 tokens, 16 heads of 128 (273 MB, 58% of the copy rate; 30% of
// the tensor pipe's cycles, 128 blocks), 279 us with the backward, 380 us for 65536 tokens of 16 heads from a stored
// state (two launches). The backward's launch alone takes 208 us: 384 items on 148 blocks, 41% of the tensor pipe's cycles,
// 1.03 GB from L2 and 369 MB from memory for 268 MB of inputs.
// Tried and not faster: Zh and Zl made before D is waited for (registers), Zh and Zl in two buffers with the outputs stored
// from registers (76 us), three buffers of Z through TMA with rolled loops (74 us), X in three stages (79 us), P shared
// between two warpgroups (90 us), A ahead of D (78 us), the product loops unrolled (73 us).
//
// Roundings. P and the copy of R round to bf16 (2^-8 each at most): they feed out, which is bf16 itself. The state is
// a 32-bit result, so g_j z_j goes into D as two bf16 terms, hi and the rest: 2^-18, where one term would leave 2^-9
// in a state that every later token reads. Sums are 32-bit.
//
// Warps: 0 loads (TMA), 1 issues the MMAs; warpgroup 1 turns A into P and writes the outputs; warpgroup 2 makes Zh and Zl;
// warpgroup 3 keeps the state. A block takes work items (sequence, head, column slice, segment, pass) in turn and the
// warps run ahead of one another across items.
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

using linear::Cut;
using linear::Seqs;
using namespace tc;

__device__ unsigned int g_linear_error;

constexpr int CT = linear::CHUNK;   // tokens of a chunk
constexpr int SL = 64;          // columns of a slice
constexpr int NT = 512;         // threads of a block
constexpr int MAX_PASS = 3;

struct Pass {
    CUtensorMap x, y, z, out;
    const void* z_ptr;
    const float* start;      // state in front of the first (behind the last) token, [N, H, Dk, Dv], or null
    float* end;              // the state at the other end, or null
    float* seg;              // the segments' own states, [slot, H, slice][SL][DRP], or null
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
    long long slots;         // of segments' states
    int items;
    int skipped;             // tests: a role that does nothing, so that the others' waits run out (0: none)
    uint32_t wait_ns;        // how long a wait lasts before it gives up
};
enum Role { LOADS = 1, PRODUCTS, PAIRS, VALUES, STATE };

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
// Once an item and by every role: a function, for the instruction cache's sake.
template <bool STATES>
__device__ __noinline__ void find_item(const Params& p, uint32_t x, Item* t) {
    const uint32_t slices = p.slices, npass = p.npass, H = p.seq.H, N = p.seq.N;
    t->slice = x % slices;
    x /= slices;
    t->pass = x % npass;
    x /= npass;
    t->h = x % H;
    x /= H;
    t->n = x % N;
    t->seg = x / N;
    t->p = &p.pass[t->pass];
    t->len = linear::seq_span(p.seq, t->n, &t->row0, &g_linear_error);
    t->nc = linear::pieces(t->len, CT);
    t->c0 = (int)min((long long)t->nc, (long long)t->seg * p.cps);
    t->c1 = min(t->nc, t->c0 + p.cps);
    if (STATES) {   // nothing comes behind the last segment (in front of the first one, backwards)
        const int last = linear::pieces(t->nc, p.cps) - 1;
        if (t->p->rev ? t->seg == 0 : t->seg >= last) t->c1 = t->c0;
    }
    t->l2 = linear::log2_decay(p.log_decay, t->h);
    if (!GDN2_IN(g_linear_error, t->seg < p.nseg && t->c0 >= 0 && t->c0 <= t->c1 && t->c1 <= t->nc)) t->c1 = t->c0;
}
// Where a segment's own state lies (null if the debug build finds that it lies outside: nothing is read or written then). Sequence n's segments take the slots from row0 / S + n on, S the tokens of a segment:
// ceil(len / S) of them never reach (row0 + len) / S + n + 1, where the next sequence's begin.
template <int DRP>
__device__ __forceinline__ float* segment_state(const Params& p, const Item& t, int seg) {
    const long long slot = t.row0 / ((long long)p.cps * CT) + t.n + seg;
    if (!GDN2_IN(g_linear_error, slot >= 0 && slot < p.slots && seg >= 0 && seg < p.nseg)) return nullptr;
    return t.p->seg + ((slot * p.seq.H + t.h) * p.slices + t.slice) * (long long)(SL * DRP);
}
// The block's first item is found once, before the roles start (its loads and the first reads of the parameters take as
// long as a chunk).
__device__ __forceinline__ Item& first_item() {
    __shared__ Item first;
    return first;
}
template <bool STATES>
__device__ __forceinline__ Item item_of(const Params& p, int x) {
    if (x == (int)blockIdx.x) return first_item();
    Item t;
    find_item<STATES>(p, (uint32_t)x, &t);
    return t;
}

template <int DRP, bool STATES>
struct Cfg {
    static constexpr uint32_t XB = STATES ? 0 : CT * DRP * 2;      // bytes of a row-operand tile
    static constexpr uint32_t YB = CT * DRP * 2;
    static constexpr uint32_t ZB = CT * SL * 2;
    static constexpr int STAGES = DRP == 64 ? 4 : STATES ? 3 : 2;  // of X and Y
    static constexpr int BUF = STATES ? 2 : 1;                     // of Zh, Zl and D: states alone leave room for two
    static constexpr int ZRAW = STATES ? 0 : 2;                    // Z as it is, for P Z
    static constexpr uint32_t SB = STATES ? 0 : DRP * SL * 2;      // bf16 copy of the state
    static constexpr uint32_t OB = STATES ? 0 : CT * SL * 2;       // output staging
    static constexpr uint32_t OFF_Y = STAGES * XB, OFF_Z = OFF_Y + STAGES * YB, OFF_ZH = OFF_Z + ZRAW * ZB,
                              OFF_S = OFF_ZH + BUF * 2 * ZB, OFF_O = OFF_S + SB, TOTAL = OFF_O + OB;
    static constexpr uint32_t SMEM = TOTAL + 1024;                 // tiles start on 1024 bytes
    // TMEM columns: A twice (then P in its first half), D (its Zh and its Zl part), O1, O2
    static constexpr uint32_t T_A = 0, T_D = 256, T_O1 = 384, T_O2 = 448;
};

// What the warps tell one another. A commit behind each product costs the tensor pipe time, so there is one for each: D
// done gives back its stage's Y and with it Zh and Zl, O1 done its X and the copy of the state, O2 done Z and P.
struct Bars {
    uint64_t full[4], d_done[4], o1_done[4];                // by stage
    uint64_t a_full[2], p_full[2], o2_done[2];              // by A's buffer
    uint64_t z_full[2], d_free[2];                          // by D's buffer
    uint64_t s_full, o_free, drain;
};

// The chunk loops of five kinds of warps share one instruction cache, and a loop that runs through it straight costs
// more in fetches than in work: the loops below are kept short (rolled over column blocks), and what a wait does when
// its barrier is not there yet is one function for all of them. It reads the timer every 16 tries (a try sleeps a while).
constexpr uint32_t TRY_NS = 20000;   // how long a try may sleep
__device__ __forceinline__ bool try_wait(uint32_t addr, uint32_t phase) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(phase), "r"(TRY_NS)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ uint32_t& wait_limit() {
    __shared__ uint32_t ns;
    return ns;
}
__device__ __noinline__ bool wait_on(uint32_t addr, uint32_t phase) {
    uint64_t t0 = 0;
    for (uint32_t tries = 1;; ++tries) {
        if (try_wait(addr, phase)) return true;
        if ((tries & 15) == 0) {
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > wait_limit()) return false;
        }
    }
}
// One thread.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t phase) {
    const uint32_t addr = smem_u32(bar);
    return try_wait(addr, phase) || wait_on(addr, phase);
}
// Two barriers whose tries are on their way together.
__device__ __forceinline__ bool wait2(uint64_t* bar0, uint32_t phase0, uint64_t* bar1, uint32_t phase1) {
    const uint32_t a0 = smem_u32(bar0), a1 = smem_u32(bar1);
    const bool r0 = try_wait(a0, phase0), r1 = try_wait(a1, phase1);
    return (r0 || wait_on(a0, phase0)) && (r1 || wait_on(a1, phase1));
}
// A whole warp: one lane asks (a dozen warps asking with every lane get in each other's way), all have its answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t phase) {
    bool ok = true;
    if ((threadIdx.x & 31) == 0) {
        ok = wait(bar, phase);
        if (!ok) atomicOr(&g_linear_error, ERR_WAIT);
    }
    return __shfl_sync(0xffffffffu, ok, 0);
}

// ------------------------------------------------------------ warp 0: loads

template <int DRP, bool STATES>
__device__ void load_tiles(const Params& p, unsigned char* sm, Bars& b) {
    using K = Cfg<DRP, STATES>;
    uint32_t ny = 0;   // stages asked for so far, over all items
    bool ok = true;
    // Two stages of X and Y cover the time of a read from L2, not that of one from memory: what comes AHEAD chunks later
    // is brought into L2 meanwhile, X and Y by one of a head's slices each. With two stages a chunk's own loads are late
    // already and go first (4 x 4096 tokens, 16 heads of 128, from memory: 72.9 against 74.4 us, 78.2 without prefetches);
    // with four the prefetches do (training on six packed sequences, 12 heads of 64: 149 against 160 us).
    constexpr int AHEAD = 3;
    constexpr bool LOADS_FIRST = K::STAGES == 2;
    auto into_l2 = [&](const Item& t, int i) {
        const int row = (int)(t.row0 + (long long)t.chunk(i) * CT);
#pragma unroll 1
        for (int c = 0; c < DRP / 64; ++c) {
            if (!STATES && t.slice == 0) tma_prefetch_3d(&t.p->x, 64 * c, t.h, row);
            if (t.slice == p.slices - 1) tma_prefetch_3d(&t.p->y, 64 * c, t.h, row);
        }
        tma_prefetch_3d(&t.p->z, t.slice * SL, t.h, row);
    };
    for (int it = blockIdx.x; ok && it < p.items; it += gridDim.x) {
        const Item t = item_of<STATES>(p, it);
        for (int i = 1; i < AHEAD && i < t.count(); ++i) into_l2(t, i);
        for (int i = 0; i < t.count(); ++i) {
            const uint32_t s = ny % K::STAGES, ph = ((ny / K::STAGES) & 1) ^ 1;
            if (!LOADS_FIRST && i + AHEAD < t.count()) into_l2(t, i + AHEAD);
            const int row = (int)(t.row0 + (long long)t.chunk(i) * CT);
            if (!(ok = wait(&b.d_done[s], ph))) break;
            mbar_arrive_expect_tx(&b.full[s], K::YB);
#pragma unroll
            for (int c = 0; c < DRP / 64; ++c)
                tma_load_3d(sm + K::OFF_Y + s * K::YB + c * CT * 128, &t.p->y, 64 * c, t.h, row, &b.full[s]);
            ++ny;
            if (!STATES) {   // X and Y come back at different times, and are waited for together
                if (!(ok = wait(&b.o1_done[s], ph))) {
                    mbar_arrive(&b.full[s]);   // no X comes any more: the barrier then closes with the stage's Y
                    break;
                }
                mbar_arrive_expect_tx(&b.full[s], K::XB);
#pragma unroll
                for (int c = 0; c < DRP / 64; ++c)
                    tma_load_3d(sm + s * K::XB + c * CT * 128, &t.p->x, 64 * c, t.h, row, &b.full[s]);
            }
            if (LOADS_FIRST && i + AHEAD < t.count()) into_l2(t, i + AHEAD);
        }
    }
    if (!ok) atomicOr(&g_linear_error, ERR_WAIT);
    // The copies in flight land before the block gives up its shared memory: each stage's last ones. Those who read them
    // may have given up; else they are there.
    for (uint32_t k = 1; k <= (uint32_t)K::STAGES && k <= ny; ++k)
        wait(&b.full[(ny - k) % K::STAGES], ((ny - k) / K::STAGES) & 1);
}

// ------------------------------------------------------------ warp 1: products

template <int DRP, bool STATES>
__device__ void issue_products(const Params& p, unsigned char* sm, uint32_t tm, Bars& b) {
    using K = Cfg<DRP, STATES>;
    // Descriptors of the tiles' first K step: a stage or a K step adds its byte offset / 16 to the address field.
    // Making them anew for every product costs more time than the product takes.
    const uint32_t base = smem_u32(sm);
    const uint64_t x_k = desc_k(base, CT, 0, 0), y_k = desc_k(base + K::OFF_Y, CT, 0, 0),
                   y_mn = desc_mn(base + K::OFF_Y, CT, 0, 0), z_mn = desc_mn(base + K::OFF_Z, CT, 0, 0),
                   zh_mn = desc_mn(base + K::OFF_ZH, CT, 0, 0), s_mn = desc_mn(base + K::OFF_S, DRP, 0, 0);
    const uint32_t idA = idesc_bf16(128, 128, false, false), idD = idesc_bf16(DRP, 2 * SL, true, true),
                   idO = idesc_bf16(128, SL, false, true);
    constexpr uint64_t MN = (16 * 128) >> 4;   // 16 rows of an MN-major tile
    // K-major: 32 bytes a step within a panel of 64 columns, then the next panel
    auto k_step = [](int kk) { return (uint64_t)(((kk >> 2) * CT * 128 + (kk & 3) * 32) >> 4); };
    // Two cursors over the same chunks. A of the next chunk is issued before O1 and O2 of this one, so that turning it
    // into P has the time of four products.
    struct Cursor {
        int x, i, count;
        bool ragged_end;   // the item's chunk range ends in a partial chunk
        bool rev;
        uint32_t n;
    };
    auto settle = [&](Cursor& c) {   // to the cursor's chunk, into the next items if need be; false behind the last
        while (c.i >= c.count) {
            c.x += gridDim.x;
            if (c.x >= p.items) return false;
            const Item t = item_of<STATES>(p, c.x);
            c.i = 0;
            c.count = t.count();
            c.rev = t.p->rev;
            c.ragged_end = c.count > 0 && t.valid(t.c1 - 1) < CT;
        }
        return true;
    };
    bool ok = true;
    auto issue_pairs = [&](Cursor& c) {   // A of the cursor's chunk; moves on
        const uint32_t n = c.n, s = n % K::STAGES, ph = (n / K::STAGES) & 1, d = n & 1, dph = (n >> 1) & 1;
        const bool ragged = c.ragged_end && c.i == (c.rev ? 0 : c.count - 1);
        // behind a sequence's end the tiles hold another's rows: warpgroup 2 clears them first
        ok = wait2(&b.full[s], ph, &b.o2_done[d], dph ^ 1) && (!ragged || wait(&b.z_full[n % K::BUF], (n / K::BUF) & 1));
        if (!ok) return;
        tc_fence_after();
        const uint64_t xk = x_k + s * (K::XB >> 4), yk = y_k + s * (K::YB >> 4);
#pragma unroll 1
        for (int kk = 0; kk < DRP / 16; ++kk)
            mma_bf16(tm + K::T_A + d * CT, xk + k_step(kk), yk + k_step(kk), idA, kk > 0);
        mma_commit(&b.a_full[d]);
        ++c.i;
        ++c.n;
    };
    Cursor cur{(int)blockIdx.x - (int)gridDim.x, 0, 0, false, false, 0}, ahead = cur;   // in front of the first item
    if (!STATES && settle(ahead)) issue_pairs(ahead);
    while (ok && settle(cur)) {
        const uint32_t n = cur.n, s = n % K::STAGES, ph = (n / K::STAGES) & 1, d = n & 1, one = n & 1;
        const uint64_t xk = x_k + s * (K::XB >> 4), ymn = y_mn + s * (K::YB >> 4), zmn = z_mn + d * (K::ZB >> 4);
        ++cur.i;
        ++cur.n;
        if (STATES && !(ok = wait(&b.full[s], ph))) break;   // else A has waited for it
        const uint32_t zb = n % K::BUF, zph = (n / K::BUF) & 1;
        if (!(ok = wait2(&b.z_full[zb], zph, &b.d_free[zb], zph ^ 1))) break;
        tc_fence_after();
#pragma unroll 1
        for (int kk = 0; kk < CT / 16; ++kk)   // Zh and Zl are the two panels of one operand of 128 columns: Y is read once
            mma_bf16(tm + K::T_D + zb * 2 * SL, ymn + MN * kk, zh_mn + zb * (2 * K::ZB >> 4) + MN * kk, idD, kk > 0);
        mma_commit(&b.d_done[s]);
        if (STATES) continue;
        if (settle(ahead)) issue_pairs(ahead);
        if (!(ok = ok && wait2(&b.s_full, one, &b.o_free, one ^ 1))) break;
        tc_fence_after();
#pragma unroll 1
        for (int kk = 0; kk < DRP / 16; ++kk)
            mma_bf16(tm + K::T_O1, xk + k_step(kk), s_mn + MN * kk, idO, kk > 0);
        mma_commit(&b.o1_done[s]);
        if (!(ok = wait(&b.p_full[d], (n >> 1) & 1))) break;
        tc_fence_after();
#pragma unroll 1
        for (int kk = 0; kk < CT / 16; ++kk)
            mma_bf16_ts(tm + K::T_O2, tm + K::T_A + d * CT + 8 * kk, zmn + MN * kk, idO, kk > 0);
        mma_commit(&b.o2_done[d]);
    }
    if (!ok) atomicOr(&g_linear_error, ERR_WAIT);
    // what was issued ends before TMEM is given back
    mma_commit(&b.drain);
    wait(&b.drain, 0);
}

// ------------------------------------------------------------ warpgroup 1: A -> P, the outputs

// Mild decays keep a part of the pair weights for the outputs (weigh_pairs).
constexpr float MILD = -2.f;   // log2 of the decay
constexpr int MIDDLE = 16;     // of a warp's 32 rows: the power of the decay that row and column part differ by at most
// A chunk's outputs, 32 rows a warp: o = f O1 + e O2 with f the power between the state's border and the row, e the row
// part of the pair weights.
struct Out {
    const Pass* p;
    int row, valid, h, slice;
    float l2;
};
template <int DRP>
__device__ __forceinline__ bool write_outputs(const Params& p, const Out& q, uint32_t n, unsigned char* sm, uint32_t tm, Bars& b) {
    using K = Cfg<DRP, false>;
    const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3, orow = 32 * w + lane;
    const bool rev = q.p->rev;
    unsigned char* Ob = sm + K::OFF_O + w * (K::OB / 4);   // this warp's 32 rows
    const float f = linear::decay_pow(q.l2, rev ? max(0, q.valid - 1 - orow) : orow + 1);
    const float e = q.l2 >= MILD ? exp2f(q.l2 * (float)((rev ? 31 - lane : lane) - MIDDLE)) : 1.f;
    const uint32_t quarter = (uint32_t)(32 * w) << 16;
    if (lane == 0) bulk_wait_read();   // the last store has read the staging rows
    if (!warp_wait(&b.o2_done[n & 1], (n >> 1) & 1)) return false;
    tc_fence_after();
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
        float o1[32], o2[32];
        tmem_ld32(tm + K::T_O1 + 32 * k + quarter, o1);
        tmem_ld32(tm + K::T_O2 + 32 * k + quarter, o2);
        tmem_wait_ld(o1, o2);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float2 v = fma2(make_float2(f, f), make_float2(o1[j], o1[j + 1]), mul2(make_float2(e, e), make_float2(o2[j], o2[j + 1])));
            o2[j] = v.x;
            o2[j + 1] = v.y;
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) st_row8(Ob, 32, lane, 4 * k + c, o2 + 8 * c);
    }
    tc_fence_before();
    mbar_arrive(&b.o_free);
    if (q.valid == CT) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(&q.p->out, q.slice * SL, q.h, q.row + 32 * w, Ob);
            bulk_commit();
        }
    } else {   // the rows behind the end are not this sequence's: 16-byte pieces of the real ones
        __syncwarp();
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(q.p->out_ptr);
#pragma unroll 1
        for (int x = lane; x < 32 * (SL / 8); x += 32) {
            const int rr = x / (SL / 8), cc = x % (SL / 8);
            if (32 * w + rr < q.valid && q.slice * SL + 8 * cc < p.dz)
                *reinterpret_cast<uint4*>(out + ((size_t)(q.row + 32 * w + rr) * p.seq.H + q.h) * p.dz + q.slice * SL + 8 * cc) =
                    *reinterpret_cast<const uint4*>(Ob + tile_chunk_off(32, rr, cc));
        }
        __syncwarp();
    }
    return true;
}

// Row i = 32 w + lane against column blocks of 32, those on the causal side.
//
// Mild decays (a >= 1/4, MILD): a^|i-j| = a^(row part) a^(column part), the row part (lane - 16, or 15 - lane backwards)
// left to the outputs, the column part 32 |w - jb| -+ j + const between -15 and 112: one value a column for all lanes,
// read four at a time. pw[pos] holds it by position. P and its sum with Z are then up to 2^30 times (the last columns of a
// diagonal block) or 2^-32 (its first) what the outputs take of them, 32 bits of range that 2^127 has to spare; with the
// row part starting at 0 it was 2^62, and outputs of 2^84 became infinite. Stronger decays would grow further: their
// weights are read by distance, pw[128 + i - j], 0 off the causal side. With the row and column parts 4 x 4096 tokens of
// 16 heads of 128 take 73 us (a = 0.9) to 79 (a = 0.252), by distance 89 (a = 0.249).
template <int DRP>
__device__ void weigh_pairs(const Params& p, unsigned char* sm, uint32_t tm, Bars& b, float* pw) {
    using K = Cfg<DRP, false>;
    const int w = (threadIdx.x >> 5) & 3, tid = threadIdx.x & 127, lane = threadIdx.x & 31;
    uint32_t n = 0;
    bool ok = true;
    Out out{};
    for (int x = blockIdx.x; x < p.items; x += gridDim.x) {
        const Item t = item_of<false>(p, x);
        if (t.count() == 0) continue;
        const bool rev = t.p->rev, mild = t.l2 >= MILD;
        if (named_sync_or(2, 128, !ok)) break;       // the last item's weights have been read
        if (mild) {
            pw[rev ? 127 - tid : tid] = exp2f(t.l2 * (float)(96 + MIDDLE - tid));
        } else {
            pw[128 + (rev ? -tid : tid)] = linear::decay_pow(t.l2, tid);
            if (tid) pw[128 + (rev ? tid : -tid)] = 0.f;
        }
        named_sync(2, 128);
        const int from = rev ? w : 0, to = rev ? 3 : w;
        for (int i = 0; ok && i < t.count(); ++i, ++n) {
            if (!(ok = warp_wait(&b.a_full[n & 1], (n >> 1) & 1))) break;
            tc_fence_after();
            const uint32_t ta = tm + K::T_A + (n & 1) * CT + ((uint32_t)(32 * w) << 16);
            // columns 16 jb .. of P lie in A's columns below 32 jb + 32, which this warp has read or does not need
#pragma unroll 1
            for (int jb = 0; jb < 4; ++jb) {
                float o[16];
                if (jb < from || jb > to) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = 0.f;
                } else {
                    float u[32];
                    tmem_ld32(ta + 32 * jb, u);
                    if (mild) {
                        const float4* q = reinterpret_cast<const float4*>(pw + 32 * (rev ? jb - w : 3 - w + jb));
                        tmem_wait_ld(u);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float4 c = q[j];
                            const float2 lo = mul2(make_float2(u[4 * j], u[4 * j + 1]), make_float2(c.x, c.y));
                            const float2 hi = mul2(make_float2(u[4 * j + 2], u[4 * j + 3]), make_float2(c.z, c.w));
                            o[2 * j] = __uint_as_float(pack_bf16x2(lo.x, lo.y));
                            o[2 * j + 1] = __uint_as_float(pack_bf16x2(hi.x, hi.y));
                        }
                        if (jb == w) {   // the bits of the pairs on the causal side: j <= lane, backwards j >= lane
                            const uint32_t keep = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                const uint32_t m = ((keep >> (2 * j)) & 1u ? 0xffffu : 0u) | ((keep >> (2 * j + 1)) & 1u ? 0xffff0000u : 0u);
                                o[j] = __uint_as_float(__float_as_uint(o[j]) & m);
                            }
                        }
                    } else {
                        const float* q = pw + 128 + tid - 32 * jb;
                        tmem_wait_ld(u);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            o[j] = __uint_as_float(pack_bf16x2(u[2 * j] * q[-2 * j], u[2 * j + 1] * q[-2 * j - 1]));
                    }
                }
                tmem_st16(ta + 16 * jb, o);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(&b.p_full[n & 1]);
            // the chunk before: its O2 ended while this one's P was made
            if (n > 0 && !(ok = write_outputs<DRP>(p, out, n - 1, sm, tm, b))) break;
            const int c = t.chunk(i);
            out = Out{t.p, (int)(t.row0 + (long long)c * CT), t.valid(c), t.h, t.slice, t.l2};
        }
    }
    if (ok && n > 0) write_outputs<DRP>(p, out, n - 1, sm, tm, b);
    if (lane == 0) bulk_wait_all();
    __syncwarp();
}

// ------------------------------------------------------------ warpgroup 2: g_j z_j in two terms

// z (gh + gl) as hi + lo, two values at a time in bf16 arithmetic: hi is the rounded product, and its remainder
// z gh - hi fits bf16 but for its last bit (8 x 8-bit products). The weight, its remainder and lo's rounding leave
// 2^-18 each, as the split of a 32-bit product would, in half the instructions.
__device__ __forceinline__ void two_terms(uint32_t z2, __nv_bfloat162 gh, __nv_bfloat162 gl, uint32_t* hi2, uint32_t* lo2) {
    const __nv_bfloat162 z = *reinterpret_cast<__nv_bfloat162*>(&z2);
    const __nv_bfloat162 hi = __hfma2(z, gh, __hmul2(z, gl));
    const __nv_bfloat162 lo = __hfma2(z, gl, __hfma2(z, gh, __hneg2(hi)));
    *hi2 = *reinterpret_cast<const uint32_t*>(&hi);
    *lo2 = *reinterpret_cast<const uint32_t*>(&lo);
}

// Z does not come through TMA: its rows go from global memory to registers a chunk ahead (eight lanes a row), and from
// there to shared memory as they are and as the two terms. Nothing then waits for a stage to be given back. Where only
// states are made, two warpgroups take the chunks, and the two buffers, in turn (`share`).
template <int DRP, bool STATES>
__device__ void split_values(const Params& p, unsigned char* sm, Bars& b, uint32_t share) {
    using K = Cfg<DRP, STATES>;
    const int tid = threadIdx.x & 127, lane = threadIdx.x & 31, w = (threadIdx.x >> 5) & 3;
    const int r0 = 32 * w + (lane >> 3), c = lane & 7;   // rows r0 + 4 k, 16-byte piece c
    uint32_t n = 0xffffffffu;                            // chunks so far, over items
    Item t;
    int x = blockIdx.x, i = -1;
    if (x < p.items) t = item_of<STATES>(p, x);
    auto next = [&]() {   // to this warpgroup's next chunk, over items; false behind the last
        do {
            ++n;
            ++i;
            while (x < p.items && i >= t.count()) {
                x += gridDim.x;
                i = 0;
                if (x < p.items) t = item_of<STATES>(p, x);
            }
        } while (STATES && x < p.items && (n & 1) != share);
        return x < p.items;
    };
    uint4 ahead[8];
    auto load = [&]() {
        const int valid = t.valid(t.chunk(i)), col = t.slice * SL + 8 * c;
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(t.p->z_ptr) + ((t.row0 + (long long)t.chunk(i) * CT + r0) * p.seq.H + t.h) * p.dz + col);
        const size_t step = (size_t)4 * p.seq.H * p.dz / 8;
#pragma unroll
        for (int k = 0; k < 8; ++k) ahead[k] = r0 + 4 * k < valid && col < p.dz ? __ldg(src + k * step) : make_uint4(0, 0, 0, 0);
    };
    bool more = next();
    if (more) load();
    __nv_bfloat162 gh[8], gl[8];   // the rows' weights
    int have = -1, have_x = -1;
    while (more) {
        const uint32_t m = n, zb = m % K::BUF, back = m - K::BUF;
        const int valid = t.valid(t.chunk(i));
        const float l2 = t.l2;
        const bool rev = t.p->rev;
        if (valid != have || x != have_x) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int r = r0 + 4 * k;
                const float g = linear::decay_pow(l2, rev ? r + 1 : max(0, valid - 1 - r));
                gh[k] = __float2bfloat162_rn(g);
                gl[k] = __float2bfloat162_rn(g - __low2float(gh[k]));
            }
            have = valid;
            have_x = x;
        }
        uint4 z[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) z[k] = ahead[k];
        more = next();
        if (more) load();
        // Zh and Zl are free once the D that read them is done, this copy of Z once the chunk before that has its O2
        if (m >= (uint32_t)K::BUF && !warp_wait(&b.d_done[back % K::STAGES], (back / K::STAGES) & 1)) return;
        if (!STATES && !warp_wait(&b.o2_done[m & 1], ((m >> 1) & 1) ^ 1)) return;
        unsigned char* Z = sm + K::OFF_Z + (m & 1) * K::ZB;
        unsigned char *Zh = sm + K::OFF_ZH + zb * 2 * K::ZB, *Zl = Zh + K::ZB;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint4 hi, lo;
            two_terms(z[k].x, gh[k], gl[k], &hi.x, &lo.x);
            two_terms(z[k].y, gh[k], gl[k], &hi.y, &lo.y);
            two_terms(z[k].z, gh[k], gl[k], &hi.z, &lo.z);
            two_terms(z[k].w, gh[k], gl[k], &hi.w, &lo.w);
            const uint32_t at = tile_chunk_off(CT, r0 + 4 * k, c);
            *reinterpret_cast<uint4*>(Zh + at) = hi;
            *reinterpret_cast<uint4*>(Zl + at) = lo;
            if (!STATES) *reinterpret_cast<uint4*>(Z + at) = z[k];
        }
        if (valid < CT) {   // rows of Y behind the sequence's end: they are another's, and would meet the zeros of Z
            const uint32_t s = m % K::STAGES;
            if (!warp_wait(&b.full[s], (m / K::STAGES) & 1)) return;
            if (tid >= valid)
#pragma unroll 1
                for (int q = 0; q < DRP / 8; ++q)
                    *reinterpret_cast<uint4*>(sm + K::OFF_Y + s * K::YB + tile_chunk_off(CT, tid, q)) = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
        mbar_arrive(&b.z_full[zb]);
    }
}

// ------------------------------------------------------------ warpgroup 3: the state

// Start state of an item: row r of the slice's columns.
template <int DRP, bool STATES>
__device__ __forceinline__ void start_state(const Params& p, const Item& t, int r, bool real, float (&S)[SL]) {
#pragma unroll
    for (int j = 0; j < SL; ++j) S[j] = 0.f;
    if (STATES || !real) return;
    const Pass& q = *t.p;
    const size_t head = (size_t)t.n * p.seq.H + t.h;
    const long long seg_tokens = (long long)p.cps * CT;
    const int nseg = linear::pieces(t.nc, p.cps);
    // the start state under its decay, then the segments' states between it and here, each under its own
    const int from = q.rev ? t.seg + 1 : 0, to = q.rev ? nseg : t.seg;
#pragma unroll 1
    for (int o = from - 1; o < max(from, to); ++o) {
        const bool first = o < from;
        if (first && (!q.start || r >= p.dr)) continue;
        // tokens between where that state stands and this segment
        const long long away = !first ? (long long)(q.rev ? o - t.seg - 1 : t.seg - 1 - o) * seg_tokens
                               : q.rev ? max(0ll, t.len - (t.seg + 1) * seg_tokens) : t.seg * seg_tokens;
        const float f = linear::decay_pow(t.l2, (int)away);
        if (first && !q.start_transposed) {
            const float* src = q.start + (head * p.dr + r) * p.dz + t.slice * SL;
#pragma unroll
            for (int j = 0; j < SL; j += 4)
                if (t.slice * SL + j < p.dz) {
                    const float4 v = *reinterpret_cast<const float4*>(src + j);
                    S[j] = f * v.x; S[j + 1] = f * v.y; S[j + 2] = f * v.z; S[j + 3] = f * v.w;
                }
        } else {   // columns contiguous over the rows
            const float* src = first ? q.start + (head * p.dz + t.slice * SL) * p.dr : segment_state<DRP>(p, t, o);
            if (!src) continue;
            src += r;
            const int step = first ? p.dr : DRP, cols = first ? p.dz - t.slice * SL : SL;
#pragma unroll
            for (int j = 0; j < SL; ++j)
                if (j < cols) S[j] = fmaf(f, src[j * step], S[j]);
        }
    }
}

template <int DRP, bool STATES>
__device__ void carry_state(const Params& p, unsigned char* sm, uint32_t tm, Bars& b) {
    using K = Cfg<DRP, STATES>;
    const int w = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    // accumulator rows: 128 in lanes 0..127; 64 in the first 16 lanes of each quarter
    const int r = DRP == 128 ? 32 * w + lane : 16 * w + (lane & 15);
    const bool real = DRP == 128 || lane < 16;
    const uint32_t quarter = (uint32_t)(32 * w) << 16;
    unsigned char* Sb = sm + K::OFF_S;
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
    for (int x = blockIdx.x; ok && x < p.items; x += gridDim.x) {
        const Item t = item_of<STATES>(p, x);
        const bool last_seg = t.p->rev ? t.seg == 0 : t.seg == max(0, linear::pieces(t.nc, p.cps) - 1);
        const bool writes_end = !STATES && t.p->end && last_seg;
        if (t.count() == 0 && !writes_end) continue;
        start_state<DRP, STATES>(p, t, r, real, S);
        if (!STATES && t.count()) {
            if (n > 0) ok = warp_wait(&b.o1_done[(n - 1) % K::STAGES], ((n - 1) / K::STAGES) & 1);
            if (ok) copy_state();
        }
        for (int i = 0; i < t.count(); ++i, ++n) {
            const int c = t.chunk(i), valid = t.valid(c);
            const uint32_t zb = n % K::BUF;
            ok = ok && warp_wait(&b.d_done[n % K::STAGES], (n / K::STAGES) & 1);
            if (ok) {
                tc_fence_after();
                const float aC = linear::decay_pow(t.l2, valid);
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    float hi[16], lo[16];
                    tmem_ld16(tm + K::T_D + zb * 2 * SL + 16 * h + quarter, hi);
                    tmem_ld16(tm + K::T_D + zb * 2 * SL + SL + 16 * h + quarter, lo);
                    tmem_wait_ld(hi, lo);
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {   // a^C S, then the small part, then the large one
                        const float2 v = fma2(make_float2(aC, aC), make_float2(S[16 * h + j], S[16 * h + j + 1]),
                                              make_float2(lo[j], lo[j + 1]));
                        S[16 * h + j] = v.x + hi[j];
                        S[16 * h + j + 1] = v.y + hi[j + 1];
                    }
                }
                tc_fence_before();
                mbar_arrive(&b.d_free[zb]);
            }
            if (!STATES && ok && i + 1 < t.count()) {
                ok = warp_wait(&b.o1_done[n % K::STAGES], (n / K::STAGES) & 1);
                if (ok) copy_state();
            }
            if (!ok) break;
        }
        if (!ok || !real) continue;
        if (STATES) {
            if (float* dst = segment_state<DRP>(p, t, t.seg)) {
#pragma unroll
                for (int j = 0; j < SL; ++j) dst[j * DRP + r] = S[j];
            }
        } else if (writes_end && r < p.dr) {
            float* dst = t.p->end + (((size_t)t.n * p.seq.H + t.h) * p.dr + r) * p.dz + t.slice * SL;
#pragma unroll
            for (int j = 0; j < SL; j += 4)
                if (t.slice * SL + j < p.dz) *reinterpret_cast<float4*>(dst + j) = make_float4(S[j], S[j + 1], S[j + 2], S[j + 3]);
        }
    }
}

template <int DRP, bool STATES>
__global__ void __launch_bounds__(NT, 1) linear_chunk_kernel(const __grid_constant__ Params p) {
    using K = Cfg<DRP, STATES>;
    extern __shared__ unsigned char raw[];
    unsigned char* sm = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    __shared__ Bars b;
    __shared__ uint32_t tmem;
    __shared__ __align__(16) float pw[256];
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < K::STAGES; ++i) {
            mbar_init(&b.full[i], STATES ? 1 : 2);
            mbar_init(&b.d_done[i], 1);
            mbar_init(&b.o1_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&b.a_full[i], 1);
            mbar_init(&b.p_full[i], 128);
            mbar_init(&b.o2_done[i], 1);
            mbar_init(&b.z_full[i], 128);
            mbar_init(&b.d_free[i], 128);
        }
        mbar_init(&b.s_full, 128);
        mbar_init(&b.o_free, 128);
        mbar_init(&b.drain, 1);
        fence_mbar_init();
        wait_limit() = p.wait_ns;
    }
    if (warp == 2) {
        tmem_alloc(&tmem, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 96) {
        find_item<STATES>(p, blockIdx.x, &first_item());
        if (!STATES) tma_prefetch_desc(&first_item().p->x);
        tma_prefetch_desc(&first_item().p->y);
        if (!STATES) tma_prefetch_desc(&first_item().p->out);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem;
    const int skipped = p.skipped;
    if (warp == 0) {
        if (skipped != LOADS && elect_one()) load_tiles<DRP, STATES>(p, sm, b);
        __syncwarp();
    } else if (warp == 1) {
        if (skipped != PRODUCTS && elect_one()) issue_products<DRP, STATES>(p, sm, tm, b);
        __syncwarp();
    } else if (!STATES && warp >= 4 && warp < 8) {
        if constexpr (!STATES)
            if (skipped != PAIRS) weigh_pairs<DRP>(p, sm, tm, b, pw);
    } else if (warp >= 4 && warp < 12) {
        if (skipped != VALUES) split_values<DRP, STATES>(p, sm, b, warp >= 8);
    } else if (warp >= 12) {
        if (skipped != STATE) carry_state<DRP, STATES>(p, sm, tm, b);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tm, 512);
}

CUresult encode(CUtensorMap* map, const void* ptr, const Seqs& s, int D, int rows) {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        cudaDriverEntryPointQueryResult q;
        void* f = nullptr;
        const cudaError_t e = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    if (!fn) return CUDA_ERROR_NOT_FOUND;
    // [rows, H, D] in boxes of some rows x 1 head x 64 channels; channels behind D and rows behind the tensor read as 0
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)s.H, (cuuint64_t)s.Ttot};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.H * D * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, step[3] = {1, 1, 1};
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

long long most_items(long long heads) { return linear::most_items(heads, sm_count()); }
bool may_cut(const Seqs& s, long long heads) { return linear::may_cut(s.T, heads, sm_count()); }
Cut choose_cut(const Seqs& s, long long heads) { return linear::choose_cut(s.N, s.T, s.Ttot, s.cu != nullptr, heads, sm_count()); }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
int padded(int d) { return d > 64 ? 128 : 64; }
int slices_of(int dz) { return (dz + SL - 1) / SL; }
size_t seg_bytes(const Seqs& s, const Cut& c, int dr, int dz) {
    return align256((size_t)c.slots * s.H * slices_of(dz) * SL * padded(dr) * sizeof(float));
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
    // Items of one length are taken in turn by one block an SM. A cut packed call's are not, and many are empty: there each
    // has a block of its own, and the hardware hands out the next one to the SM that gets free.
    const int grid = p.seq.cu && p.nseg > 1 ? p.items : std::min(p.items, sm_count());
    TraceScope trace(STATES ? K_LINEAR_SEGMENT : K_LINEAR_CHUNK, s);
    linear_chunk_kernel<DRP, STATES><<<grid, NT, K::SMEM, s>>>(p);
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
    p.slots = cut.slots;
    const long long items = (long long)cut.nseg * a.seq.N * a.seq.H * g.npass * p.slices;
    if (items > 2000000000ll) return cudaErrorInvalidConfiguration;
    p.items = (int)items;
    p.skipped = test_skip_linear_role();
    p.wait_ns = p.skipped ? 5000000u : 2000000000u;
    cudaError_t e = cudaSuccess;
    if (cut.nseg > 1) e = padded(g.dr) == 128 ? launch<128, true>(p, s) : launch<64, true>(p, s);
    if (e != cudaSuccess) return e;
    return padded(g.dr) == 128 ? launch<128, false>(p, s) : launch<64, false>(p, s);
}

// Passes of the forward (1) or the backward (3), as (row, value) sizes.
long long heads_of(const Seqs& s, bool bwd) {
    const int k = slices_of(s.Dk), v = slices_of(s.Dv);
    return (long long)s.N * s.H * (bwd ? 2 * k + v : v);
}

}  // namespace

size_t linear_chunk_workspace(const Seqs& s, bool bwd) {
    const long long heads = heads_of(s, bwd);
    if (!may_cut(s, heads)) return 0;
    // a start state that the call's end state overwrites, then the segments' states (each region 256-byte aligned)
    return state_bytes(s) + (size_t)most_items(heads) * SL * padded(std::max(s.Dk, s.Dv)) * sizeof(float) + 3 * 256;
}

cudaError_t linear_chunk_launch(const LinearArgs& a, bool bwd, cudaStream_t s) {
    const Seqs& q = a.seq;
    if (q.T == 0) return linear32_launch(a, bwd, s);   // no tokens: states alone are handed on (and cu_seqlens checked)
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
        good = good && encode(&p.x, x, q, dr, CT) == CUDA_SUCCESS && encode(&p.y, y, q, dr, CT) == CUDA_SUCCESS &&
               encode(&p.z, z, q, dz, CT) == CUDA_SUCCESS && encode(&p.out, out, q, dz, 32) == CUDA_SUCCESS;
        p.start = start;
        p.end = end;
        p.seg = seg(dr, dz);
        p.z_ptr = z;
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

cudaError_t linear_chunk_error_word(unsigned int** word) {
    return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_linear_error);
}

}  // namespace gdn2

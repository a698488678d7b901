// linear_api.cu -- C entry points of linear attention with a decay per head (whole sequences, packed sequences, the
// single-token step) and of the query/key norm with rotation: argument checks, workspace sizes, dispatch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <nvtx3/nvToolsExt.h>

#include "gdn2.h"
#include "internal.h"
#include "linear.cuh"
#include "qk_rope.cuh"

using namespace gdn2;

namespace {

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

gdn2_status fail(gdn2_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
gdn2_status fail(gdn2_status s, const char* fmt, ...) {
    char msg[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    set_last_error(msg);
    return s;
}
gdn2_status cuda_status(cudaError_t e, const char* where) {
    return e == cudaSuccess ? GDN2_OK : fail(GDN2_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}
bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

gdn2_status check_dims(const linear::Seqs& s, gdn2_dtype dt) {
    if (dt != GDN2_F32 && dt != GDN2_BF16) return fail(GDN2_ERR_INVALID, "dtype %d is not GDN2_F32 or GDN2_BF16", (int)dt);
    if (s.N < 1 || s.H < 1) return fail(GDN2_ERR_INVALID, "%d sequences and H=%d must be >= 1", s.N, s.H);
    if (s.T < 0 || s.Ttot < 0) return fail(GDN2_ERR_INVALID, "T=%d and %lld rows must be >= 0", s.T, s.Ttot);
    if (!dim_ok(s.Dk) || !dim_ok(s.Dv))
        return fail(GDN2_ERR_UNSUPPORTED, "Dk=%d, Dv=%d: each must be 16, 32, 64 or 128", s.Dk, s.Dv);
    // blocks are counted in ints, token rows of a packed call in int32 (cu_seqlens)
    const double heads = (double)s.N * s.H, chunks = heads * (((double)s.T + 63) / 64);
    if (heads * (s.Dk * s.Dv / 256) > 2147483647.0 || chunks > 2147483647.0 || (double)s.Ttot > 2147483647.0)
        return fail(GDN2_ERR_INVALID, "problem too large");
    return GDN2_OK;
}

#define REQUIRE_PTR(p)                                                                          \
    do {                                                                                        \
        if (!(p)) return fail(GDN2_ERR_INVALID, "%s must not be NULL", #p);                     \
        if (!aligned((p), 16)) return fail(GDN2_ERR_INVALID, "%s must be 16-byte aligned", #p); \
    } while (0)
#define OPTIONAL_PTR(p)                                                                                \
    do {                                                                                               \
        if ((p) && !aligned((p), 16)) return fail(GDN2_ERR_INVALID, "%s must be 16-byte aligned", #p); \
    } while (0)
#define REQUIRE_WORD_PTR(p)                                                                    \
    do {                                                                                       \
        if (!(p)) return fail(GDN2_ERR_INVALID, "%s must not be NULL", #p);                    \
        if (!aligned((p), 4)) return fail(GDN2_ERR_INVALID, "%s must be 4-byte aligned", #p);  \
    } while (0)

size_t workspace(const linear::Seqs& s, gdn2_dtype dt, bool bwd, bool packed) {
    return align256(dt == GDN2_BF16 ? linear_chunk_workspace(s, bwd) : linear32_workspace(s, packed, bwd));
}
// No sequence of a packed call is longer than its tensor, however loose the bound: plans, grids and workspace go by that.
void tighten(linear::Seqs& s) {
    if (s.Ttot >= 0 && s.T > s.Ttot) s.T = (int)s.Ttot;
}

gdn2_status run(linear::Seqs seq, const void* q, const void* k, const void* v, const float* log_decay, const float* S0,
                const void* dout, const float* dST, void* o, float* ST, void* dq, void* dk, void* dv, float* dS0, bool bwd,
                gdn2_dtype dt, void* ws, size_t ws_bytes, void* stream, const char* fn) {
    NvtxRange nvtx(fn);
    if (seq.cu) tighten(seq);
    gdn2_status st = check_dims(seq, dt);
    if (st != GDN2_OK) return st;
    REQUIRE_WORD_PTR(log_decay);
    OPTIONAL_PTR(S0);
    OPTIONAL_PTR(ST);
    OPTIONAL_PTR(dST);
    OPTIONAL_PTR(dS0);
    if (seq.T > 0 && seq.Ttot > 0) {
        REQUIRE_PTR(q); REQUIRE_PTR(k); REQUIRE_PTR(v);
        if (bwd) {
            REQUIRE_PTR(dout); REQUIRE_PTR(dq); REQUIRE_PTR(dk); REQUIRE_PTR(dv);
        } else {
            REQUIRE_PTR(o);
        }
        const size_t need = workspace(seq, dt, bwd, seq.cu != nullptr);
        if (need && (!ws || ws_bytes < need))
            return fail(GDN2_ERR_WORKSPACE, "%s needs %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
        if (need && !aligned(ws, 256)) return fail(GDN2_ERR_INVALID, "ws must be 256-byte aligned");
    }
    LinearArgs a{};
    a.seq = seq;
    if (seq.Ttot == 0) a.seq.T = 0;   // no rows: every sequence is empty
    a.dt = dt;
    a.q = q; a.k = k; a.v = v; a.dout = bwd ? dout : nullptr;
    a.log_decay = log_decay; a.S0 = S0; a.dST = dST;
    a.o = o; a.ST = ST; a.dq = dq; a.dk = dk; a.dv = dv; a.dS0 = dS0;
    a.ws = ws;
    cudaStream_t str = static_cast<cudaStream_t>(stream);
    return cuda_status(dt == GDN2_BF16 ? linear_chunk_launch(a, bwd, str) : linear32_launch(a, bwd, str), fn);
}

linear::Seqs dense(int B, int T, int H, int Dk, int Dv) {
    return linear::Seqs{nullptr, B, T, (long long)B * T, H, Dk, Dv};
}

}  // namespace

extern "C" {

size_t gdn2_linear_workspace_size(gdn2_op op, int N, int T, int H, int Dk, int Dv, gdn2_dtype dt) {
    if (op != GDN2_OP_FWD && op != GDN2_OP_BWD) return 0;
    const linear::Seqs s{nullptr, N, T, 0, H, Dk, Dv};
    if (check_dims(s, dt) != GDN2_OK) return 0;
    return workspace(s, dt, op == GDN2_OP_BWD, false);
}

size_t gdn2_linear_varlen_workspace_size(gdn2_op op, int N, int Tmax, long long Ttot, int H, int Dk, int Dv, gdn2_dtype dt) {
    if (op != GDN2_OP_FWD && op != GDN2_OP_BWD) return 0;
    linear::Seqs s{nullptr, N, Tmax, Ttot, H, Dk, Dv};
    tighten(s);
    if (check_dims(s, dt) != GDN2_OK) return 0;
    return workspace(s, dt, op == GDN2_OP_BWD, true);
}

gdn2_status gdn2_linear_fwd(const void* q, const void* k, const void* v, const float* log_decay, const float* S0, void* o,
                            float* ST, int B, int T, int H, int Dk, int Dv, gdn2_dtype dt, void* ws, size_t ws_bytes,
                            void* stream) {
    return run(dense(B, T, H, Dk, Dv), q, k, v, log_decay, S0, nullptr, nullptr, o, ST, nullptr, nullptr, nullptr, nullptr,
               false, dt, ws, ws_bytes, stream, "gdn2_linear_fwd");
}

gdn2_status gdn2_linear_bwd(const void* q, const void* k, const void* v, const float* log_decay, const float* S0,
                            const void* dout, const float* dST, void* dq, void* dk, void* dv, float* dS0, int B, int T, int H,
                            int Dk, int Dv, gdn2_dtype dt, void* ws, size_t ws_bytes, void* stream) {
    return run(dense(B, T, H, Dk, Dv), q, k, v, log_decay, S0, dout, dST, nullptr, nullptr, dq, dk, dv, dS0, true, dt, ws,
               ws_bytes, stream, "gdn2_linear_bwd");
}

gdn2_status gdn2_linear_varlen_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                                   const int* cu_seqlens, int N, int Tmax, long long Ttot, const float* S0, void* o, float* ST,
                                   int H, int Dk, int Dv, gdn2_dtype dt, void* ws, size_t ws_bytes, void* stream) {
    REQUIRE_WORD_PTR(cu_seqlens);
    return run(linear::Seqs{cu_seqlens, N, Tmax, Ttot, H, Dk, Dv}, q, k, v, log_decay, S0, nullptr, nullptr, o, ST, nullptr,
               nullptr, nullptr, nullptr, false, dt, ws, ws_bytes, stream, "gdn2_linear_varlen_fwd");
}

gdn2_status gdn2_linear_varlen_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                                   const int* cu_seqlens, int N, int Tmax, long long Ttot, const float* S0, const void* dout,
                                   const float* dST, void* dq, void* dk, void* dv, float* dS0, int H, int Dk, int Dv,
                                   gdn2_dtype dt, void* ws, size_t ws_bytes, void* stream) {
    REQUIRE_WORD_PTR(cu_seqlens);
    return run(linear::Seqs{cu_seqlens, N, Tmax, Ttot, H, Dk, Dv}, q, k, v, log_decay, S0, dout, dST, nullptr, nullptr, dq, dk,
               dv, dS0, true, dt, ws, ws_bytes, stream, "gdn2_linear_varlen_bwd");
}

gdn2_status gdn2_linear_decode_step(const void* q, const void* k, const void* v, const float* log_decay, float* S,
                                    const int* slots, int num_slots, void* o, int B, int H, int Dk, int Dv, gdn2_dtype dt,
                                    void* stream) {
    NvtxRange nvtx("gdn2_linear_decode_step");
    gdn2_status st = check_dims(dense(B, 1, H, Dk, Dv), dt);
    if (st != GDN2_OK) return st;
    REQUIRE_PTR(q); REQUIRE_PTR(k); REQUIRE_PTR(v); REQUIRE_PTR(S); REQUIRE_PTR(o);
    REQUIRE_WORD_PTR(log_decay);
    if (slots && !aligned(slots, 4)) return fail(GDN2_ERR_INVALID, "slots must be 4-byte aligned");
    if (num_slots < 1 || (!slots && num_slots < B))
        return fail(GDN2_ERR_INVALID, "%d states: need one at least, and without slots one for each of the %d rows", num_slots, B);
    LinearStepArgs a{dt, q, k, v, log_decay, S, slots, num_slots, o, B, H, Dk, Dv};
    return cuda_status(linear_step_launch(a, static_cast<cudaStream_t>(stream)), "gdn2_linear_decode_step");
}

size_t gdn2_qk_norm_rope_workspace_size(int D) { return dim_ok(D) ? (size_t)QK_ROPE_BLOCKS * D * sizeof(float) : 0; }

static gdn2_status rope(QkRopeArgs a, int pos_bytes, int B, int T, bool bwd, void* ws, size_t ws_bytes, void* stream,
                        const char* fn) {
    NvtxRange nvtx(fn);
    if (a.dt != GDN2_F32 && a.dt != GDN2_BF16) return fail(GDN2_ERR_INVALID, "dtype %d is not GDN2_F32 or GDN2_BF16", (int)a.dt);
    if (B < 1 || T < 0 || a.Hq < 1 || a.Hk < 1)
        return fail(GDN2_ERR_INVALID, "B=%d, Hq=%d and Hk=%d must be >= 1, T=%d >= 0", B, a.Hq, a.Hk, T);
    if (!dim_ok(a.D)) return fail(GDN2_ERR_UNSUPPORTED, "D=%d must be 16, 32, 64 or 128", a.D);
    if (a.pairs < 1 || a.pairs > a.D / 2) return fail(GDN2_ERR_INVALID, "%d pairs: must be 1 to D / 2 = %d", a.pairs, a.D / 2);
    if (pos_bytes != 4 && pos_bytes != 8) return fail(GDN2_ERR_INVALID, "positions of %d bytes: must be 4 or 8", pos_bytes);
    if (a.num_axes < 1) return fail(GDN2_ERR_INVALID, "%d axes: must be >= 1", a.num_axes);
    if (a.norm && !(a.eps > 0.f && isfinite(a.eps))) return fail(GDN2_ERR_INVALID, "eps must be positive and finite");
    const int es = a.dt == GDN2_BF16 ? 2 : 4;
    const long long strides[2] = {a.q_stride, a.k_stride};
    const int widths[2] = {a.Hq, a.Hk};
    for (int i = 0; i < 2; ++i)
        if (strides[i] < (long long)widths[i] * a.D || (strides[i] * es) % 16)
            return fail(GDN2_ERR_INVALID, "%s_stride=%lld: tokens must not overlap and must start on 16 bytes", i ? "k" : "q", strides[i]);
    if ((double)B * T * (a.Hq + a.Hk) > 2147483647.0 * 4) return fail(GDN2_ERR_INVALID, "problem too large");
    a.tokens = (long long)B * T;
    a.pos64 = pos_bytes == 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (bwd && a.norm) {
        if (a.dq_weight && !aligned(a.dq_weight, 16)) return fail(GDN2_ERR_INVALID, "dq_weight must be 16-byte aligned");
        if (a.dk_weight && !aligned(a.dk_weight, 16)) return fail(GDN2_ERR_INVALID, "dk_weight must be 16-byte aligned");
    }
    if (a.tokens == 0) {   // no rows: the weight gradients are empty sums
        for (float* w : {a.dq_weight, a.dk_weight})
            if (bwd && a.norm && w) {
                cudaError_t e = cudaMemsetAsync(w, 0, a.D * sizeof(float), s);
                if (e != cudaSuccess) return cuda_status(e, fn);
            }
        return GDN2_OK;
    }
    const void *q = a.q, *k = a.k, *inv_freq = a.inv_freq, *positions = a.positions;
    REQUIRE_PTR(q); REQUIRE_PTR(k);
    REQUIRE_WORD_PTR(inv_freq); REQUIRE_WORD_PTR(positions);
    if (pos_bytes == 8 && !aligned(positions, 8)) return fail(GDN2_ERR_INVALID, "positions must be 8-byte aligned");
    if (a.axes && !aligned(a.axes, 4)) return fail(GDN2_ERR_INVALID, "axes must be 4-byte aligned");
    const float *q_weight = a.q_weight, *k_weight = a.k_weight;
    OPTIONAL_PTR(q_weight); OPTIONAL_PTR(k_weight);
    if (!bwd) {
        void *q_out = a.q_out, *k_out = a.k_out;
        REQUIRE_PTR(q_out); REQUIRE_PTR(k_out);
    } else {
        const void *dq_out = a.dq_out, *dk_out = a.dk_out;
        void *dq = a.dq, *dk = a.dk;
        REQUIRE_PTR(dq_out); REQUIRE_PTR(dk_out); REQUIRE_PTR(dq); REQUIRE_PTR(dk);
        const size_t need = a.norm && (a.dq_weight || a.dk_weight) ? gdn2_qk_norm_rope_workspace_size(a.D) : 0;
        if (need && (!ws || ws_bytes < need))
            return fail(GDN2_ERR_WORKSPACE, "%s needs %zu workspace bytes, got %zu", fn, need, ws ? ws_bytes : (size_t)0);
        if (need && !aligned(ws, 256)) return fail(GDN2_ERR_INVALID, "ws must be 256-byte aligned");
    }
    return cuda_status(qk_rope_launch(a, static_cast<float*>(ws), s), fn);
}

gdn2_status gdn2_qk_norm_rope_fwd(const void* q, const void* k, long long q_stride, long long k_stride, const void* positions,
                                  int pos_bytes, int num_axes, const float* inv_freq, const int* axes, int pairs, int interleaved,
                                  int norm, float eps, const float* q_weight, const float* k_weight, void* q_out, void* k_out,
                                  int B, int T, int Hq, int Hk, int D, gdn2_dtype dt, void* stream) {
    QkRopeArgs a{};
    a.dt = dt;
    a.Hq = Hq; a.Hk = Hk; a.D = D;
    a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride;
    a.positions = positions; a.num_axes = num_axes; a.inv_freq = inv_freq; a.axes = axes;
    a.pairs = pairs; a.interleaved = interleaved; a.norm = norm; a.eps = eps;
    a.q_weight = q_weight; a.k_weight = k_weight;
    a.q_out = q_out; a.k_out = k_out;
    return rope(a, pos_bytes, B, T, false, nullptr, 0, stream, "gdn2_qk_norm_rope_fwd");
}

gdn2_status gdn2_qk_norm_rope_bwd(const void* q, const void* k, long long q_stride, long long k_stride, const void* dq_out,
                                  const void* dk_out, const void* positions, int pos_bytes, int num_axes, const float* inv_freq,
                                  const int* axes, int pairs, int interleaved, int norm, float eps, const float* q_weight,
                                  const float* k_weight, void* dq, void* dk, float* dq_weight, float* dk_weight, int B, int T,
                                  int Hq, int Hk, int D, gdn2_dtype dt, void* ws, size_t ws_bytes, void* stream) {
    QkRopeArgs a{};
    a.dt = dt;
    a.Hq = Hq; a.Hk = Hk; a.D = D;
    a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride;
    a.positions = positions; a.num_axes = num_axes; a.inv_freq = inv_freq; a.axes = axes;
    a.pairs = pairs; a.interleaved = interleaved; a.norm = norm; a.eps = eps;
    a.q_weight = q_weight; a.k_weight = k_weight;
    a.dq_out = dq_out; a.dk_out = dk_out; a.dq = dq; a.dk = dk; a.dq_weight = dq_weight; a.dk_weight = dk_weight;
    return rope(a, pos_bytes, B, T, true, ws, ws_bytes, stream, "gdn2_qk_norm_rope_bwd");
}

}  // extern "C"

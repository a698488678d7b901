// device_records.h -- what the kernels' error words say, as one status and one text. Plain C++, so that it can be checked
// where there is no GPU.
#pragma once

#include <stdarg.h>
#include <stddef.h>
#include <stdio.h>

#include "gdn2.h"

namespace gdn2 {

constexpr unsigned int GDN2_DBG_BIT = 1u << 30;   // an index check of the debug build failed

// Bits of a packed call's record (varlen.cu, the linear kernels).
constexpr unsigned int ERR_LONG = 1u;      // a sequence longer than Tmax (cut)
constexpr unsigned int ERR_OUTSIDE = 2u;   // a sequence outside [0, Ttot) or of negative length (dropped)
// Further bits of the linear kernels'.
constexpr unsigned int ERR_SLOT = 4u;      // a decode slot outside the pool or named twice (skipped)
constexpr unsigned int ERR_WAIT = 8u;      // a bounded wait gave up

// The error words since the previous reading.
struct DeviceRecords {
    unsigned int fwd, bwd;        // chunk_fwd_kernel, chunk_bwd_kernel: bits of waits, GDN2_DBG_BIT
    unsigned int varlen;          // packed-sequence copies
    unsigned int linear;          // linear attention, both precisions: bits of packed calls and waits, GDN2_DBG_BIT
    unsigned int step, rope;
};

// The gravest record gives the status, a wait that gave up (outputs are garbage) before a failed index check (accesses
// were skipped) before arguments found wrong on the device; the text has them all in that order, for reading clears them.
inline gdn2_status describe_records(const DeviceRecords& r, char* text, size_t cap) {
    gdn2_status status = GDN2_OK;
    size_t at = 0;
    if (cap) text[0] = 0;
    auto add = [&](gdn2_status s, const char* fmt, auto... args) {
        if (status == GDN2_OK) status = s;
        const char* sep = at ? "; " : "";
        for (int part = 0; part < 2 && at + 1 < cap; ++part) {
            const int n = part == 0 ? snprintf(text + at, cap - at, "%s", sep) : snprintf(text + at, cap - at, fmt, args...);
            at += n < 0 ? 0 : (size_t)n;
        }
    };
    const unsigned int waits_fwd = r.fwd & ~GDN2_DBG_BIT, waits_bwd = r.bwd & ~GDN2_DBG_BIT;
    if (waits_fwd | waits_bwd)
        add(GDN2_ERR_TIMEOUT,
            "device wait gave up: chunk_fwd_kernel bits 0x%x, chunk_bwd_kernel bits 0x%x "
            "(1 MMA completion, 2 tile loads, 4 forward ready flag / gradient unit, 8 backward ready flag, "
            "16 launched with a block size the kernel is not built for)",
            waits_fwd, waits_bwd);
    if (r.linear & ERR_WAIT) add(GDN2_ERR_TIMEOUT, "%s", "device wait gave up: linear_chunk_kernel");
    if ((r.fwd | r.bwd) & GDN2_DBG_BIT)
        add(GDN2_ERR_INVALID,
            "index check failed (debug build; the accesses it guarded were skipped): chunk_fwd_kernel bits "
            "0x%x, chunk_bwd_kernel bits 0x%x",
            r.fwd, r.bwd);
    if (r.linear & GDN2_DBG_BIT)
        add(GDN2_ERR_INVALID, "index check failed (debug build; the accesses it guarded were skipped): linear attention bits 0x%x", r.linear);
    const unsigned int packed = (r.varlen | r.linear) & (ERR_LONG | ERR_OUTSIDE);
    if (packed)
        add(GDN2_ERR_INVALID, "cu_seqlens: %s%s", (packed & ERR_LONG) ? "a sequence was longer than Tmax (cut) " : "",
            (packed & ERR_OUTSIDE) ? "a sequence lay outside [0, Ttot) or had a negative length (dropped)" : "");
    if (r.step & ERR_SLOT)
        add(GDN2_ERR_INVALID, "%s", "slots: a row's slot lay outside the pool, or an earlier row had named it (row skipped)");
    if (r.rope) add(GDN2_ERR_INVALID, "%s", "axes: a pair's axis lay outside [0, num_axes) (pair not turned)");
    return status;
}

}  // namespace gdn2

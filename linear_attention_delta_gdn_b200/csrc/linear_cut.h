// linear_cut.h -- how linear attention on tensor cores cuts a sequence's chunks into segments. Plain C++, so that the
// plan can be checked where there is no GPU.
#pragma once

#include <algorithm>

#ifdef __CUDACC__
#define GDN2_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define GDN2_HOST_DEVICE inline
#endif

namespace gdn2 {
namespace linear {

constexpr int CHUNK = 128;   // tokens of a chunk

// Pieces of `size` that n >= 0 make, the last one perhaps partial; n may be 2^31 - 1.
GDN2_HOST_DEVICE int pieces(int n, int size) { return (int)(((unsigned int)n + (unsigned int)size - 1u) / (unsigned int)size); }

// Segments of cps chunks, nseg of them a sequence at most, `slots` states for them all (and head and slice).
struct Cut {
    int nseg, cps;
    long long slots;
};
// Items of a call that is cut at all, at most: its workspace is sized by them (a packed call's lengths are not known
// then). `heads` counts the blocks of 64 columns over all sequences, `nsm` the blocks that run at once.
inline long long most_items(long long heads, int nsm) { return 2 * heads + 4 * nsm; }
inline bool may_cut(int T, long long heads, int nsm) { return T > CHUNK && heads < 4 * nsm; }

// Time in chunks of one block (1.7 to 1.9 us): the fullest block's chunks and 4 more for each of its items' start and end, in
// more than one segment also 1.5 for each segment that an item's start is summed from, and the launch before, whose chunks
// cost half as much (a sequence's last segment has none there), with 3 for the launch itself. Sequences of one length go in
// waves. Of packed ones only the sum of their lengths is known here: the fullest block is taken to have the mean and half
// an item more, and an item without chunks costs 1. One sequence of 65536 tokens, 16 heads of 128: 951 us uncut, 675 / 465 /
// 381 us in 2 / 3 / 4 segments (one wave), 403 us in 9 (two waves), 564 us in 5 (two waves, the second nearly empty). Eight
// packed sequences of 12557 tokens in all, 8 heads of 64 x 128: 91 us uncut, 85 us in 2 or 3 segments, 105 us in 6.
inline Cut choose_cut(int N, int T, long long Ttot, bool packed, long long heads, int nsm) {
    const int nc = pieces(T, CHUNK);
    Cut best{1, std::max(nc, 1), 0};
    if (!may_cut(T, heads, nsm)) return best;
    const double total = (Ttot / (double)CHUNK + 0.5 * N) * ((double)heads / N);   // packed chunks, over all heads
    double best_time = 1e30;
    for (int r = 1; r <= 64 && r <= nc; ++r) {
        const int cps = pieces(nc, r), nseg = pieces(nc, cps);
        const long long slots = Ttot / ((long long)cps * CHUNK) + N + 1;
        if (nseg > 1 && slots * (heads / N) > most_items(heads, nsm)) break;
        // a launch's time from the cost of a chunk and of an item, its segments a sequence, and of packed sequences its
        // chunks and its items with chunks
        auto time = [&](double chunk, double item, int segs, double chunks, double items) {
            const double one = chunk * cps + item;
            if (!packed) return (double)((heads * segs + nsm - 1) / nsm) * one;
            return std::max(one, (chunk * chunks + 4 * items + std::max(0.0, (double)heads * nseg - items)) / nsm + 0.5 * one);
        };
        const double items = 0.5 * heads + total / cps;
        double t = time(1.0, 4 + 1.5 * (nseg - 1), nseg, total, items);
        if (nseg > 1) t += time(0.5, 4, nseg - 1, std::max(0.0, total - 0.5 * heads * cps), std::max(0.0, items - heads)) + 3;
        if (t < best_time) {
            best_time = t;
            best = Cut{nseg, cps, nseg > 1 ? slots : 0};
        }
    }
    return best;
}

}  // namespace linear
}  // namespace gdn2

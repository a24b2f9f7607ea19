// How the work items of a ragged batch are numbered.
#pragma once

#include "pdq_kernels.h"

namespace pdq {

// Items (a page that new tokens touch; a tile of rows) are numbered without a
// prefix sum.  A sequence of n rows has up to floor(n mul / per) + extra of them;
// those of sequence s begin at floor(cu_q[s] mul / per) + extra s, and floor(a + b)
// >= floor(a) + floor(b) leaves room enough before those of sequence s + 1.
// Without cu_q a sequence has one row and ceil(mul / per) items.
__device__ __forceinline__ int items_of_a_row(int mul, int per) { return mul == 1 ? 1 : (mul + per - 1) / per; }

__device__ __forceinline__ int64_t item_start(const KvBatch& b, int s, int mul, int per, int extra) {
    if (!b.cu_q) return (int64_t)s * items_of_a_row(mul, per);
    return (int64_t)min(max(b.cu_q[s], 0), b.tokens) * mul / per + (int64_t)extra * s;
}

// Item w is the k-th of sequence s, the last one that begins at or before it: 64
// candidates a step, one step for up to 64 sequences.  The whole wavefront calls it
// with the same w.  False: w is no sequence's.  Those are the items before the first
// sequence's (cu_q[0] rows before it belong to none), and with offsets that descend
// any that the search does not place; k is negative there.  Whether sequence s has a
// k-th item is for the caller to see: room is left behind its last.
__device__ __forceinline__ bool item_of(const KvBatch& b, int64_t w, int mul, int per, int extra, int& s, int64_t& k) {
    if (!b.cu_q) {
        s = (int)(w / items_of_a_row(mul, per));
    } else {
        const int lane = threadIdx.x & 63;
        int lo = 0, n = b.batch;
        while (n > 1) {
            const int step = (n + 63) / 64;
            const bool in = lane * step < n && item_start(b, lo + lane * step, mul, per, extra) <= w;
            const int c = max(__popcll(__ballot(in)), 1) - 1;
            lo += c * step;
            n = min(step, n - c * step);
        }
        s = __builtin_amdgcn_readfirstlane(lo);
    }
    k = w - item_start(b, s, mul, per, extra);
    return k >= 0;
}

}  // namespace pdq

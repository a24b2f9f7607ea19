// What the kernels of the INT8 key/value cache share: the cache's layout, where
// a sequence's new tokens lie, which rows a work item is.
#pragma once

#include "kv_items.h"
#include "pdq_device.h"

namespace pdq {

// A value at an address that is the same in every lane, of memory that the kernel
// does not write: through the scalar cache, so that waiting for it does not wait
// for the vector loads in flight.
template <typename T>
__device__ __forceinline__ T uniform_load(const T* p) {
    const uint64_t u = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)u), hi = __builtin_amdgcn_readfirstlane((int)(u >> 32));
    return *reinterpret_cast<const __attribute__((address_space(4))) T*>((uint64_t)hi << 32 | lo);
}

template <bool Uniform, typename T>
__device__ __forceinline__ T load_as(const T* p) {
    if constexpr (Uniform) return uniform_load(p);
    else return *p;
}

// One sequence of the batch as the kernels see it.  What the device arrays hold
// cannot be checked on the host: new rows are clamped to [0, tokens), so that
// no value of cu_q reaches outside q, k, v.
struct KvSeq {
    int q0, n;  // first new row, new rows
    int len;    // tokens after the call, as given
    int p0;     // position of the first new row: len - n (may be negative)
};

template <bool Uniform = false>  // s is the same in every lane
__device__ __forceinline__ KvSeq kv_seq(const KvBatch& b, int s) {
    KvSeq r;
    if (b.cu_q) {
        r.q0 = min(max(load_as<Uniform>(b.cu_q + s), 0), b.tokens);
        r.n = min(max(load_as<Uniform>(b.cu_q + s + 1), r.q0), b.tokens) - r.q0;
    } else {
        r.q0 = s;
        r.n = 1;
    }
    // lengths outside [0, 2^30] count as the nearer of the two: positions and their differences stay in int32
    r.len = min(max(load_as<Uniform>(b.seq_len + s), 0), 1 << 30);
    r.p0 = r.len - r.n;
    return r;
}

// The sequence of row t, the same in the whole wavefront: the last one that
// begins at or before it, 64 candidates a step.
__device__ __forceinline__ int row_seq(const KvBatch& b, int t) {
    if (!b.cu_q) return t;
    const int lane = threadIdx.x & 63;
    int lo = 0, n = b.batch;
    while (n > 1) {
        const int step = (n + 63) / 64;
        const bool in = lane * step < n && b.cu_q[lo + lane * step] <= t;
        const int k = max(__popcll(__ballot(in)), 1) - 1;
        lo += k * step;
        n = min(step, n - k * step);
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

}  // namespace pdq

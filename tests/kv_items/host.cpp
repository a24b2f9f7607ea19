// The numbering of the key/value kernels' work items (csrc/kv_items.h) on the host.
//
// The functions are those that the kernels call.  A wavefront's 64 lanes run them one
// after the other: a lane that reaches a ballot whose outcome is not known yet leaves
// its vote and stops; when all have voted the lanes run again with that outcome.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <vector>

using std::max;
using std::min;

namespace {

struct Vote {};
struct {
    unsigned x;
} lane_id;
std::vector<uint64_t> known;
size_t asked;
uint64_t votes;

uint64_t ballot(bool in) {
    if (asked < known.size()) return known[asked++];
    votes |= (uint64_t)in << lane_id.x;
    throw Vote();
}

template <typename F>
void wavefront(F f) {
    known.clear();
    for (bool done = false; !done;) {
        votes = 0;
        done = true;
        for (lane_id.x = 0; lane_id.x < 64; ++lane_id.x) {
            asked = 0;
            try {
                f();
            } catch (Vote) {
                done = false;
            }
        }
        if (!done) known.push_back(votes);
    }
}

}  // namespace

#undef __device__
#undef __forceinline__
#define __device__
#define __forceinline__ inline
#define threadIdx lane_id
#define __ballot ballot
#define __popcll __builtin_popcountll
#define __builtin_amdgcn_readfirstlane(v) (v)
#include "kv_items.h"

// Items 0 .. count - 1: their sequences, their numbers there and whether they are a sequence's.
extern "C" void items(const int32_t* cu_q, int batch, int tokens, int mul, int per, int extra, int64_t count, int32_t* s,
                      int64_t* k, uint8_t* there) {
    pdq::KvBatch b{};
    b.cu_q = cu_q;
    b.batch = batch;
    b.tokens = tokens;
    for (int64_t w = 0; w < count; ++w)
        wavefront([&] {
            int sw = 0;
            there[w] = pdq::item_of(b, w, mul, per, extra, sw, k[w]);
            s[w] = sw;
        });
}

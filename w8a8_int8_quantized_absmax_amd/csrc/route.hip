// Routing to experts (gfx950): scores of the router's logits, groups, the largest k,
// their weights; and the rows (token and slot) sorted by expert.
//
// Latency and not bytes.  A token is taken by 16 lanes (64 where there are more than 256
// experts), its logits in their registers, and the largest is found k times over: maxima
// within 16 lanes are four lane permutations, no LDS.  What decides a choice is binary64: a
// score next to another's would else be ordered by its last rounding; scores that decide
// nothing are formed for the chosen experts alone.
// Counting is by workgroup (LDS atomics on whole numbers, whose order changes nothing), the
// places by sums over the workgroups before, so that the order is the tokens' own: two
// launches, one where a workgroup takes all tokens.

#include <algorithm>

#include "fp8_device.h"

namespace pdq {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64, kMost = 512;  // experts

// Whole numbers in the order of the doubles; NaN 1 (below every number), 0 is kept for "not to be chosen".
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return 1;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | (uint64_t(1) << 63);
}

// The same of binary32 values.
__device__ __forceinline__ uint32_t order_key(float v) {
    if (v != v) return 1;
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u >> 31 ? ~u : u | 0x80000000u;
}

template <int kCtrl>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {
    return (uint64_t)dpp_u32<kCtrl>((uint32_t)(v >> 32)) << 32 | dpp_u32<kCtrl>((uint32_t)v);
}

// f over the L lanes of a token, the same in each of them.
template <int L, typename F>
__device__ __forceinline__ uint64_t reduce_u64(uint64_t v, F f) {
    v = f(v, dpp_u64<0xB1>(v));   // quad_perm [1, 0, 3, 2]
    v = f(v, dpp_u64<0x4E>(v));   // quad_perm [2, 3, 0, 1]
    v = f(v, dpp_u64<0x141>(v));  // row_half_mirror
    v = f(v, dpp_u64<0x140>(v));  // row_mirror
    if constexpr (L == 64) {
        v = f(v, (uint64_t)__shfl_xor((unsigned long long)v, 16));
        v = f(v, (uint64_t)__shfl_xor((unsigned long long)v, 32));
    }
    return v;
}

template <int L>
__device__ __forceinline__ double sum_of(double v) {
    return __longlong_as_double((long long)reduce_u64<L>((uint64_t)__double_as_longlong(v), [](uint64_t a, uint64_t b) {
        return (uint64_t)__double_as_longlong(__longlong_as_double((long long)a) + __longlong_as_double((long long)b));
    }));
}

template <int L>
__device__ __forceinline__ uint64_t max_of(uint64_t v) {
    return reduce_u64<L>(v, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
}

template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
    v = row16_max(v);
    if constexpr (L == 64) {
        v = max(v, (uint32_t)__shfl_xor((int)v, 16));
        v = max(v, (uint32_t)__shfl_xor((int)v, 32));
    }
    return v;
}

template <int L>
__device__ __forceinline__ uint32_t min_of(uint32_t v) {
    v = min(v, dpp_u32<0xB1>(v));
    v = min(v, dpp_u32<0x4E>(v));
    v = min(v, dpp_u32<0x141>(v));
    v = min(v, dpp_u32<0x140>(v));
    if constexpr (L == 64) {
        v = min(v, (uint32_t)__shfl_xor((int)v, 16));
        v = min(v, (uint32_t)__shfl_xor((int)v, 32));
    }
    return v;
}

// Whether a lane of the token says so.
template <int L>
__device__ __forceinline__ bool any_of(bool v) {
    const uint64_t all = __ballot(v);
    return L == 64 ? all != 0 : (all >> (threadIdx.x & 48) & 0xffff) != 0;
}

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t row, int e) {
    const int64_t at = row + e;
    if (a.dt == kF32) return static_cast<const float*>(a.logits)[at];
    const uint32_t v = static_cast<const uint16_t*>(a.logits)[at];
    return a.dt == kBF16 ? bf16_to_f32(v) : f16_to_f32(v);
}

// exp(x - top); infinite logits share a softmax's weight.
__device__ __forceinline__ double shifted_exp(float x, float top) {
    return x == top ? 1.0 : exp((double)x - (double)top);
}

__device__ __forceinline__ double sigmoid(float x) { return 1.0 / (1.0 + exp(-(double)x)); }

struct SortSpace {
    int total[kMost], next[kMost], wave_next[kWaves][kMost], sums[kWaves];
    unsigned long long lanes[kWaves][kMost];
};

// The rows of the workgroup's tokens [t0, t1) to their places, by the whole workgroup: an expert's
// begin behind those of the experts before it, a workgroup's behind those of the workgroups
// before it.  hist: the blocks' counts, rows of `pitch`.
__device__ void sort_rows(const RouteArgs& a, const int* hist, int pitch, int blocks, int block, int t0, int t1,
                          SortSpace& s) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    s.total[tid] = 0;  // kThreads == kMost
    s.next[tid] = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        s.wave_next[w][tid] = 0;
        s.lanes[w][tid] = 0;
    }
    __syncthreads();
    // counts: four experts a lane, the blocks dealt to the slices of lanes
    const int quads = pitch / 4, slices = kThreads / quads, slice = tid / quads;
    if (slice < slices) {
        v4i total = v4i{}, before = v4i{};
        const v4i* h = reinterpret_cast<const v4i*>(hist) + tid % quads;
        for (int b = slice; b < blocks; b += slices) {
            const v4i n = h[(int64_t)b * quads];
            total += n;
            if (b < block) before += n;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = tid % quads * 4 + i;
            if (total[i]) atomicAdd(&s.total[e], total[i]);
            if (before[i]) atomicAdd(&s.next[e], before[i]);
        }
    }
    // the workgroup's own, by wavefront
    const int64_t f0 = (int64_t)t0 * a.k, f1 = (int64_t)t1 * a.k;
    const int64_t each = (f1 - f0 + 64 * kWaves - 1) / (64 * kWaves) * 64;  // rows of a wavefront
    const int64_t w0 = min(f0 + wave * each, f1), w1 = min(w0 + each, f1);
    for (int64_t f = w0 + lane; f < w1; f += 64) {
        const int id = a.ids[f];
        if (id >= 0) atomicAdd(&s.wave_next[wave][id], 1);
    }
    __syncthreads();
    const int mine = s.total[tid];
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(sum, d);
        if (lane >= d) sum += o;
    }
    if (lane == 63) s.sums[wave] = sum;
    __syncthreads();
    int base = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        if (w < wave) base += s.sums[w];
        all += s.sums[w];
    }
    const int first = base + sum - mine;
    if (tid < a.experts) {
        if (block == 0) {
            a.offsets[tid] = first;
            if (tid == a.experts - 1) a.offsets[a.experts] = all;
        }
        int at = first + s.next[tid];
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const int n = s.wave_next[w][tid];
            s.wave_next[w][tid] = at;
            at += n;
        }
    }
    __syncthreads();
    const int64_t rows = (int64_t)a.tokens * a.k;
    for (int64_t i = all + (int64_t)block * kThreads + tid; i < rows; i += (int64_t)blocks * kThreads) a.rows[i] = -1;
    for (int64_t f = w0; f < w1; f += 64) {  // in order, 64 rows at a time
        const int id = f + lane < w1 ? a.ids[f + lane] : -1;
        if (id >= 0) atomicOr(&s.lanes[wave][id], 1ull << lane);
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();
        unsigned long long same = 0;
        int at = 0;
        if (id >= 0) {
            same = s.lanes[wave][id];
            at = s.wave_next[wave][id];
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();
        if (id >= 0) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            a.rows[at + rank] = (int)(f + lane);
            if (rank == 0) {  // the first of its expert's
                s.wave_next[wave][id] = at + __popcll(same);
                s.lanes[wave][id] = 0;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();
    }
}

// L lanes a token, VPL experts a lane (lane + L j).  kAlone: the workgroup takes all tokens, and sorts
// them too.  Key: uint32_t where the logits order the experts, uint64_t where the biased scores do.
template <typename Key, int L, int VPL, bool kAlone>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a, int per, int pitch) {
    constexpr int kTeams = kThreads / L, kSlots = L == 16 ? 2 : 1;  // at most 32 choices
    __shared__ __attribute__((aligned(16))) int hist[kMost];
    // the groups' scores; and, afterwards, what sorting needs
    union Space {
        double scores[kTeams][L * VPL];
        SortSpace sort;
        __device__ Space() {}
    };
    __shared__ Space space;
    const int lane = threadIdx.x & 63, r = lane & (L - 1), team = threadIdx.x / L;
    hist[threadIdx.x] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * per, t1 = min(t0 + per, a.tokens);
    const int size = a.experts / a.groups;
    const bool every = sizeof(Key) == 8 || a.groups > 1;  // the scores of every expert take part in the choice
    for (int t = t0 + team; t < t1; t += kTeams) {
        const int64_t row = t * a.ldl;
        float x[VPL];
        bool nan = false;
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = r + L * j;
            x[j] = e < a.experts ? logit(a, row, e) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            nan |= x[j] != x[j];
            top = fmaxf(top, x[j]);
        }
        nan = any_of<L>(nan);
        top = fmaxf(top, dpp_f32<0xB1>(top));
        top = fmaxf(top, dpp_f32<0x4E>(top));
        top = fmaxf(top, dpp_f32<0x141>(top));
        top = fmaxf(top, dpp_f32<0x140>(top));
        if constexpr (L == 64) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
        }
        Key key[VPL];
        double sum = 1.0;
        if (every || (!a.sigmoid && !a.renormalize)) {
            double p[VPL];
            if (a.sigmoid) {
#pragma unroll
                for (int j = 0; j < VPL; ++j) p[j] = sigmoid(x[j]);
            } else {
                sum = 0.0;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    p[j] = x[j] == -INFINITY ? 0.0 : shifted_exp(x[j], top);
                    sum += p[j];
                }
                sum = sum_of<L>(sum);
                if (every) {
#pragma unroll
                    for (int j = 0; j < VPL; ++j) p[j] = p[j] / sum;
                }
            }
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int e = r + L * j;
                double c = p[j];
                if constexpr (sizeof(Key) == 8) {
                    if (e < a.experts) c += (double)a.bias[e];
                    key[j] = x[j] == -INFINITY || c == -INFINITY ? 0 : order_key(c);
                } else {
                    key[j] = x[j] == -INFINITY ? 0 : order_key(x[j]);
                }
                if (a.groups > 1) space.scores[team][e] = key[j] < 2 ? -INFINITY : c;
            }
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = x[j] == -INFINITY ? 0 : order_key(x[j]);
        }
        if (a.groups > 1) {  // lane i's groups: i, i + L, ..; at most 64
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
            __builtin_amdgcn_wave_barrier();
            uint64_t best[64 / L];
            int rank[64 / L];
#pragma unroll
            for (int q = 0; q < 64 / L; ++q) {
                const int g = r + L * q;
                best[q] = 0;
                rank[q] = 0;
                if (g < a.groups) {
                    double first = -INFINITY, second = -INFINITY;
                    const double* v = space.scores[team] + g * size;
#pragma unroll 4
                    for (int i = 0; i < size; ++i) {
                        second = fmax(second, fmin(first, v[i]));
                        first = fmax(first, v[i]);
                    }
                    if (first > -INFINITY) best[q] = order_key(a.group_score == 2 && second > -INFINITY ? first + second : first);
                }
            }
            // (their places in LDS taken over by the groups' keys)
            unsigned long long* const keys = reinterpret_cast<unsigned long long*>(space.scores[team]);
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int q = 0; q < 64 / L; ++q)
                if (r + L * q < a.groups) keys[r + L * q] = best[q];
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
            __builtin_amdgcn_wave_barrier();
#pragma unroll 4
            for (int h = 0; h < a.groups; ++h) {
                const uint64_t o = keys[h];
#pragma unroll
                for (int q = 0; q < 64 / L; ++q) rank[q] += o > best[q] || (o == best[q] && h < r + L * q);
            }
            uint64_t kept = 0;
#pragma unroll
            for (int q = 0; q < 64 / L; ++q) {
                const uint64_t b = __ballot(r + L * q < a.groups && rank[q] < a.top_groups);
                kept |= (L == 64 ? b : b >> (lane & 48) & 0xffff) << (L * q & 63);
            }
            __builtin_amdgcn_wave_barrier();
            const float per_size = 1.0f / (float)size;  // (exact enough: quotients of whole numbers up to 512)
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const int g = (int)(((float)(r + L * j) + 0.5f) * per_size);
                if (!(kept >> min(g, 63) & 1)) key[j] = 0;
            }
        }
        int id[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) id[q] = -1;
        for (int s = 0; s < a.k; ++s) {
            Key best = key[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j) best = max(key[j], best);
            best = max_of<L>(best);
            if (best == 0) break;  // (the same in a token's lanes)
            uint32_t at = 0xffffffffu;
#pragma unroll
            for (int j = VPL - 1; j >= 0; --j)
                if (key[j] == best) at = r + L * j;
            at = min_of<L>(at);  // the lowest of equals
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (at == (uint32_t)(r + L * j)) key[j] = 0;
#pragma unroll
            for (int q = 0; q < kSlots; ++q)
                if (s == r + L * q) id[q] = (int)at;
        }
        double p[kSlots], total = 0.0;
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            p[q] = 0.0;
            if (id[q] >= 0) {
                const float v = logit(a, row, id[q]);
                p[q] = a.sigmoid ? sigmoid(v) : shifted_exp(v, top);
            }
            total += p[q];
        }
        if (a.renormalize) total = sum_of<L>(total);
        else total = a.sigmoid ? 1.0 : sum;
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
            if (r + L * q >= a.k) continue;
            const int64_t flat = (int64_t)t * a.k + r + L * q;
            a.ids[flat] = id[q];
            // (a sum of 0: every score 0)
            const double w = total == 0.0 ? 0.0 : p[q] / total * (double)a.scale;
            a.weights[flat] = id[q] < 0 ? 0.0f : nan ? __builtin_nanf("") : (float)w;
            if (id[q] >= 0) atomicAdd(&hist[id[q]], 1);
        }
    }
    __syncthreads();
    if constexpr (kAlone) {
        sort_rows(a, hist, pitch, 1, 0, t0, t1, space.sort);
    } else {
        if ((int)threadIdx.x < pitch) a.hist[(int64_t)blockIdx.x * pitch + threadIdx.x] = hist[threadIdx.x];
    }
}

__global__ __launch_bounds__(kThreads) void k_route_sort(RouteArgs a, int per, int pitch) {
    __shared__ SortSpace space;
    const int t0 = blockIdx.x * per;
    sort_rows(a, a.hist, pitch, a.tokens ? gridDim.x : 0, blockIdx.x, min(t0, a.tokens), min(t0 + per, a.tokens), space);
}

// Tokens of a workgroup: 32 (16 lanes each), or as many as leave at most 256 workgroups, each of which
// reads every other's counts (with 512 of half the size: 8192 x 256 40.7 us against 30.2, 16384 x 64
// 18.6 / 15.8).  Up to 64 tokens one workgroup does it all: at 64 that takes 9.4 us where two launches
// take 8.3, but the host 2.7 us less.
int route_tokens(int64_t tokens) { return tokens <= 64 ? 64 : (int)std::max<int64_t>(32, (tokens + 255) / 256); }

int hist_pitch(int experts) { return (experts + 3) / 4 * 4; }

template <int L, int VPL>
void launch_scores(const RouteArgs& a, int per, uint32_t blocks, hipStream_t st) {
    const int pitch = hist_pitch(a.experts);
    const dim3 grid(blocks), block(kThreads);
    if (blocks == 1) {
        if (a.bias) hipLaunchKernelGGL((k_route<uint64_t, L, VPL, true>), grid, block, 0, st, a, per, pitch);
        else hipLaunchKernelGGL((k_route<uint32_t, L, VPL, true>), grid, block, 0, st, a, per, pitch);
    } else {
        if (a.bias) hipLaunchKernelGGL((k_route<uint64_t, L, VPL, false>), grid, block, 0, st, a, per, pitch);
        else hipLaunchKernelGGL((k_route<uint32_t, L, VPL, false>), grid, block, 0, st, a, per, pitch);
    }
}

}  // namespace

size_t route_space(int64_t tokens, int64_t experts) {
    const int64_t per = route_tokens(tokens);
    return (size_t)((tokens + per - 1) / per) * hist_pitch((int)experts) * 4;
}

void launch_route(const RouteArgs& a, hipStream_t st) {
    const int per = route_tokens(a.tokens);
    const uint32_t blocks = (uint32_t)((a.tokens + per - 1) / per);
    if (blocks > 0) {
        if (a.experts <= 32) launch_scores<16, 2>(a, per, blocks, st);
        else if (a.experts <= 64) launch_scores<16, 4>(a, per, blocks, st);
        else if (a.experts <= 128) launch_scores<16, 8>(a, per, blocks, st);
        else if (a.experts <= 192) launch_scores<16, 12>(a, per, blocks, st);
        else if (a.experts <= 256) launch_scores<16, 16>(a, per, blocks, st);
        else launch_scores<64, 8>(a, per, blocks, st);
        if (blocks == 1) return;
    }
    hipLaunchKernelGGL(k_route_sort, dim3(std::max(1u, blocks)), dim3(kThreads), 0, st, a, per, hist_pitch(a.experts));
}

}  // namespace pdq

// Routing to experts (gfx950): scores of the router's logits, groups, the largest k,
// their weights; and the rows (token and slot) sorted by expert.
//
// Latency and not bytes: a wavefront a token, the scores in its registers, and the
// largest found k times over.  What decides a choice is binary64: a score next to
// another's would else be ordered by its last rounding.  Counting is by workgroup
// (LDS atomics on whole numbers, whose order changes nothing), the places by sums
// over the workgroups before, so that the order is the tokens' own.

#include <algorithm>

#include "fp8_device.h"

namespace pdq {

namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;

// Whole numbers in the order of the doubles; NaN 1 (below every number), 0 is kept for "not to be chosen".
__device__ __forceinline__ uint64_t order_key(double v) {
    if (v != v) return 1;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u >> 63 ? ~u : u | (uint64_t(1) << 63);
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const uint64_t o = __shfl_xor((unsigned long long)v, d);
        v = o > v ? o : v;
    }
    return v;
}

template <int DT>
__device__ __forceinline__ float logit(const void* row, int e) {
    if constexpr (DT == kF32) return static_cast<const float*>(row)[e];
    else if constexpr (DT == kBF16) return bf16_to_f32(static_cast<const uint16_t*>(row)[e]);
    else return f16_to_f32(static_cast<const uint16_t*>(row)[e]);
}

// VPL: experts a lane (lane + 64 j).
template <int DT, int VPL>
__global__ __launch_bounds__(kThreads) void k_route(RouteArgs a, int per) {
    __shared__ int hist[64 * VPL];
    __shared__ double cs[kWaves][64 * VPL];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int e = threadIdx.x; e < a.experts; e += kThreads) hist[e] = 0;
    __syncthreads();
    const int t0 = blockIdx.x * per, t1 = min(t0 + per, a.tokens);
    const int size = a.experts / a.groups;
    for (int t = t0 + wave; t < t1; t += kWaves) {
        const char* row = static_cast<const char*>(a.logits) + t * a.ldl * Elem<DT>::bytes;
        double x[VPL], p[VPL];
        uint64_t key[VPL];
        bool nan = false;
        double top = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = lane + 64 * j;
            x[j] = e < a.experts ? (double)logit<DT>(row, e) : -INFINITY;
            nan |= x[j] != x[j];
            top = x[j] > top ? x[j] : top;
        }
        nan = __any(nan);
        if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) p[j] = 1.0 / (1.0 + exp(-x[j]));
        } else {
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) {
                const double o = __shfl_xor(top, d);
                top = o > top ? o : top;
            }
            double sum = 0.0;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                p[j] = x[j] == top ? 1.0 : exp(x[j] - top);  // infinite logits share the weight
                if (x[j] == -INFINITY) p[j] = 0.0;
                sum += p[j];
            }
#pragma unroll
            for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
#pragma unroll
            for (int j = 0; j < VPL; ++j) p[j] = p[j] / sum;
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const int e = lane + 64 * j;
            const double c = a.bias && e < a.experts ? p[j] + (double)a.bias[e] : x[j];
            key[j] = x[j] == -INFINITY || c == -INFINITY ? 0 : order_key(c);
            if (a.groups > 1) cs[wave][e] = key[j] < 2 ? -INFINITY : a.bias ? c : p[j];
        }
        if (a.groups > 1) {
            __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
            __builtin_amdgcn_wave_barrier();
            uint64_t mine = 0;
            if (lane < a.groups) {
                double first = -INFINITY, second = -INFINITY;
                for (int i = 0; i < size; ++i) {
                    const double v = cs[wave][lane * size + i];
                    if (v > first) {
                        second = first;
                        first = v;
                    } else if (v > second) {
                        second = v;
                    }
                }
                if (first > -INFINITY)
                    mine = order_key(a.group_score == 2 && second > -INFINITY ? first + second : first);
            }
            int rank = 0;
            for (int h = 0; h < a.groups; ++h) {
                const uint64_t o = __shfl((unsigned long long)mine, h);
                rank += o > mine || (o == mine && h < lane);
            }
            const uint64_t kept = __ballot(lane < a.groups && rank < a.top_groups);
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (!(kept >> min((lane + 64 * j) / size, 63) & 1)) key[j] = 0;
        }
        int id = -1;     // lane s: slot s
        double w = 0.0, sum = 0.0;
        for (int s = 0; s < a.k; ++s) {
            uint64_t best = key[0];
#pragma unroll
            for (int j = 1; j < VPL; ++j) best = key[j] > best ? key[j] : best;
            best = wave_max_u64(best);
            if (best == 0) break;
            int at = -1;
            double pv = 0.0;
#pragma unroll
            for (int j = 0; j < VPL; ++j) {
                const uint64_t eq = __ballot(key[j] == best);
                if (at < 0 && eq) {
                    const int l = __builtin_ctzll(eq);
                    at = 64 * j + l;
                    pv = __shfl(p[j], l);
                    if (lane == l) key[j] = 0;
                }
            }
            sum += pv;
            if (lane == s) {
                id = at;
                w = pv;
            }
        }
        if (lane < a.k) {
            if (a.renormalize) w = sum > 0.0 ? w / sum : sum == 0.0 ? 0.0 : sum;
            const int64_t flat = (int64_t)t * a.k + lane;
            a.ids[flat] = id;
            a.weights[flat] = id < 0 ? 0.0f : nan ? __builtin_nanf("") : (float)(w * (double)a.scale);
            if (id >= 0) atomicAdd(&hist[id], 1);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.experts; e += kThreads) a.hist[(int64_t)blockIdx.x * a.experts + e] = hist[e];
}

// The rows of the workgroup's tokens to their places: an expert's begin behind those
// of the experts before it, a workgroup's behind those of the workgroups before it.
__global__ __launch_bounds__(kThreads) void k_route_sort(RouteArgs a, int per) {
    __shared__ int next[1024], wsum[kWaves], all;
    __shared__ unsigned long long lanes[1024];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int before_all = 0;
    for (int e0 = 0; e0 < a.experts; e0 += kThreads) {
        const int e = e0 + threadIdx.x;
        int total = 0, before = 0;
        if (e < a.experts)
            for (int b = 0; a.tokens > 0 && b < (int)gridDim.x; ++b) {
                const int n = a.hist[(int64_t)b * a.experts + e];
                total += n;
                before += b < (int)blockIdx.x ? n : 0;
            }
        int sum = total;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 63) wsum[wave] = sum;
        __syncthreads();
        int base = before_all;
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) base += wsum[w];
            before_all += wsum[w];
        }
        if (e < a.experts) {
            next[e] = base + sum - total + before;
            lanes[e] = 0;
            if (blockIdx.x == 0) {
                a.offsets[e] = base + sum - total;
                if (e == a.experts - 1) a.offsets[a.experts] = base + sum;
            }
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) all = before_all;
    __syncthreads();
    const int64_t total = (int64_t)a.tokens * a.k;
    for (int64_t i = all + blockIdx.x * (int64_t)kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads)
        a.rows[i] = -1;
    if (wave != 0) return;
    const int64_t f0 = (int64_t)blockIdx.x * per * a.k, f1 = min(f0 + (int64_t)per * a.k, total);
    for (int64_t f = f0; f < f1; f += 64) {  // in order, 64 rows at a time
        const int id = f + lane < f1 ? a.ids[f + lane] : -1;
        if (id >= 0) atomicOr(&lanes[id], 1ull << lane);
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();
        unsigned long long same = 0;
        int base = 0;
        if (id >= 0) {
            same = lanes[id];
            base = next[id];
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();
        if (id >= 0) {
            const int rank = __popcll(same & ((1ull << lane) - 1));
            a.rows[base + rank] = (int)(f + lane);
            if (rank == 0) {  // the first of its expert's
                next[id] = base + __popcll(same);
                lanes[id] = 0;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
        __builtin_amdgcn_wave_barrier();
    }
}

// Tokens of a workgroup: 32, more where that would be more than 256 workgroups (each of
// which reads every other's counts).
int route_tokens(int64_t tokens) { return (int)std::max<int64_t>(32, (tokens + 255) / 256); }

template <int DT>
void launch_scores(const RouteArgs& a, int per, uint32_t blocks, hipStream_t st) {
    const dim3 grid(blocks), block(kThreads);
    if (a.experts <= 64) hipLaunchKernelGGL((k_route<DT, 1>), grid, block, 0, st, a, per);
    else if (a.experts <= 128) hipLaunchKernelGGL((k_route<DT, 2>), grid, block, 0, st, a, per);
    else if (a.experts <= 256) hipLaunchKernelGGL((k_route<DT, 4>), grid, block, 0, st, a, per);
    else hipLaunchKernelGGL((k_route<DT, 8>), grid, block, 0, st, a, per);
}

}  // namespace

int route_blocks(int64_t tokens) {
    const int per = route_tokens(tokens);
    return (int)((tokens + per - 1) / per);
}

void launch_route(const RouteArgs& a, int dt, hipStream_t st) {
    const int per = route_tokens(a.tokens);
    const uint32_t blocks = (uint32_t)std::max(1, route_blocks(a.tokens));
    if (a.tokens == 0) {  // no row: offsets alone
    } else if (dt == kF32) launch_scores<kF32>(a, per, blocks, st);
    else if (dt == kBF16) launch_scores<kBF16>(a, per, blocks, st);
    else launch_scores<kF16>(a, per, blocks, st);
    hipLaunchKernelGGL(k_route_sort, dim3(blocks), dim3(kThreads), 0, st, a, per);
}

}  // namespace pdq

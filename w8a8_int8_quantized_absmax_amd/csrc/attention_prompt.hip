// Attention over the paged INT8 key/value cache, many rows for each sequence
// (prompts, chunks of prompts): bound by the matrix products and the softmax
// between them.  include/pdq.h (pdq_kv_attention) states the arithmetic,
// attention_device.h how it is taken.
#include <algorithm>
#include <type_traits>

#include "attention_device.h"

namespace pdq {

namespace {

constexpr float kMost = 0x1p14f;  // a sum of eight weights beyond which M moves

constexpr int kKeys = 64;  // keys of a step

// Waves of a workgroup, 32 rows each.  Eight share the conversion of a step's
// codes between them and fill a compute unit (two to a SIMD, 256 registers); with
// 256 channels a wave needs more registers than that, and with 64 there is room
// for three smaller workgroups.
constexpr int waves(int D) { return D == 128 ? 8 : 4; }
constexpr int per_simd(int D) { return D == 256 ? 1 : D == 128 ? 2 : 3; }
constexpr int tile_rows(int D) { return 32 * waves(D); }

// LDS of one step's operands, in 16-byte pieces of 8 binary16 values.
// K: piece (c, t) = channels 8 c .. 8 c + 7 of token t.  V: piece (2 u + h, d) =
// channel NT m + t (NT = D / 32, d = 32 t + m) of the tokens 4 h .. 4 h + 3 and 8 + 4 h ..
// 8 + 4 h + 3 of the u-th 16 tokens, the order in which a lane of half h holds its
// weights.  A lane of a product reads the piece of its own row, a whole half wave
// 512 contiguous bytes; the paddings let the conversion's writes fall into
// different banks too.
template <int D>
struct KeyStage {
    static constexpr int kPitch = kKeys * 16 + (D == 64 ? 32 : 16);
    uint8_t at[D / 8 * kPitch];
};
template <int D>
struct ValueStage {
    static constexpr int kSkew = D == 128 ? 128 : 0;  // behind every second t
    static constexpr int kPitch = D * 16 + (D / 64 - 1) * kSkew + 16;
    uint8_t at[kKeys / 8 * kPitch];
    float4 scale[kKeys / 16];  // of each 16 tokens: S_k, log2 S_v, 1 / S_v, 0 or 1: a page is there
    static __device__ __forceinline__ int piece(int t, int m) { return t * 512 + (t >> 1) * kSkew + m * 16; }
};

// The sum over a wavefront, in all lanes.
__device__ __forceinline__ int lanes_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, false);   // quad_perm [1, 0, 3, 2]
    v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, false);   // quad_perm [2, 3, 0, 1]
    v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, false);  // row_half_mirror
    v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, false);  // row_mirror
    return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
           __builtin_amdgcn_readlane(v, 48);
}

// The row tile of rank `rank` when all sequences' tiles are taken by their number
// from the last to the first (the later a tile, the more keys it sees), at equal
// numbers by sequence; false: there are fewer.  One lane a sequence: with c(k) the
// tiles numbered k or more, the tile's number is the k with c(k + 1) <= rank <
// c(k).  Workgroups start in the order of their numbers, round the compute units:
// prompts of uneven lengths then share them evenly (9 prompts of 347 to 1531
// rows, 12 heads of 64: the busiest unit has 48 steps of 64 keys, 69 sequence by
// sequence, of 35 on average; 53 us, 72).  Used up to five times the workgroups that fit,
// with / without it, us: 3.2 times (40 prompts, 64 channels) 64 / 73, 3.3 (7 prompts, 128 channels) 96 / 103, 3.7 (8, 256
// channels) 150 / 171; beyond, 7.1 (64 channels) 179 / 186, 7.4 (128) 210 / 213, 13 (128) 358 / 357, 16 (256) 474 / 484, 25
// (128) 637 / 633: there the many tiles even out by themselves.
__device__ __forceinline__ bool heaviest_first(const AttentionArgs& a, int rows, int group, int rank, int& s, int64_t& tile) {
    const int lane = threadIdx.x & 63;
    const int mine = lane < a.b.batch ? (int)(((int64_t)kv_seq(a.b, lane).n * group + rows - 1) / rows) : 0;
    int lo = 0, hi = lanes_sum(mine), above = 0;  // c(lo) > rank >= c(hi) = above
    if (hi <= rank) return false;
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        const int c = lanes_sum(max(mine - mid, 0));
        if (c > rank) {
            lo = mid;
        } else {
            hi = mid;
            above = c;
        }
    }
    const uint64_t level = __ballot(mine > lo);
    const int before = __popcll(level & (((uint64_t)1 << lane) - 1));
    const uint64_t at = __ballot(mine > lo && before == rank - above);
    s = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)at) - 1);
    tile = lo;
    return true;
}

// One workgroup takes tile_rows(D) rows (token, query head of the group) of one
// key/value head over a part of their keys.  Scores are computed transposed, keys
// x rows, in 32x32x16 products, so that a row's scores lie in one lane (and the one
// 32 lanes on) and its weights are the operand of the value product as they stand;
// the output is accumulated transposed too.  Codes are loaded a step ahead,
// converted once for all waves and staged in one of two LDS buffers, one barrier
// a step.  CAP, BIAS: softcap, slopes are given.
//
// One prompt of 8192 tokens, 32 heads over 8 of 128 channels: 560 to 600 us, 0.92
// to 0.98 PFLOP/s of the pairs that are seen (a library product of 8192^3 reaches 1.24
// here).  No unit is full: of the cycles the matrix units are busy for 42%, the
// vector units for 46% (a weight costs a multiply-add, an exponential of two issue
// slots, an addition and half a conversion; a code of K or V two and a half), LDS
// for 40%.  They overlap badly: beside a wave that issues matrix instructions back to
// back, another wave's binary32 additions and multiply-adds hardly advance (57 in
// 33000 cycles; exponentials and packed binary16 do, where the first leaves it a few
// cycles between), so the two waves of a SIMD add their matrix and vector time.  Tried and slower, each
// on a form of 580 to 607 us: the two waves of a SIMD held half a step apart by a second barrier (620 us),
// 64 rows a wave (790), 32 keys a step with three waves a SIMD (609), four-wave workgroups, two a compute unit (590).
template <int DT, int D, bool CAP, bool BIAS>
__global__ __launch_bounds__(64 * waves(D), per_simd(D)) void k_attention_prompt(AttentionArgs a, int64_t items, int splits) {
    constexpr int KU = kKeys / 32, NU = kKeys / 16, NW = waves(D), kRows = tile_rows(D), NC = D / 16, NT = D / 32;
    // operands on their way from LDS while one is multiplied, where registers allow (8192 tokens: 577 to 587 us without, 563 with)
    constexpr int kAhead = D == 128 ? 8 : 0;
    constexpr int KB = kKeys * D / (64 * NW), VD = kKeys * D / (512 * NW);  // bytes of K, channels of V that a thread brings
    __shared__ KeyStage<D> ks[2];
    __shared__ ValueStage<D> vs[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 31, h = lane >> 5;
    const int group = a.hq / a.c.heads;
    const int hk = blockIdx.x % a.c.heads;
    int s;
    int64_t tile;
    if (a.b.cu_q && a.b.batch > 1 && a.b.batch <= 64 && gridDim.x <= 5 * 256 * (4 * per_simd(D) / NW)) {
        if (!heaviest_first(a, kRows, group, (int)(blockIdx.x / a.c.heads), s, tile)) return;
    } else {
        const int64_t item = items - 1 - blockIdx.x / a.c.heads;  // a prompt's last rows see most: before its others
        if (!item_of(a.b, item, group, kRows, 1, s, tile)) return;
    }
    const AttnSeq sq = attn_seq<true>(a, s);
    const int64_t rows = (int64_t)sq.q.n * group, r0 = tile * kRows;
    if (r0 >= rows) return;

    // the keys that the tile's rows see, in steps, and this workgroup's part of them
    int lo0, hi0, lo1, hi1;
    row_keys(a, sq, sq.q.p0 + (int)(r0 / group), lo0, hi0);
    row_keys(a, sq, sq.q.p0 + (int)(min(r0 + kRows, rows) - 1) / group, lo1, hi1);
    const int first = lo0 & ~(kKeys - 1);
    const int steps = hi1 < first ? 0 : (hi1 - first) / kKeys + 1;
    const int part = (steps + splits - 1) / splits;
    const int begin = __builtin_amdgcn_readfirstlane(first + min((int)blockIdx.y * part, steps) * kKeys);
    const int end = __builtin_amdgcn_readfirstlane(min(first + min(((int)blockIdx.y + 1) * part, steps) * kKeys, hi1 + 1));

    // this lane's row
    const int64_t r = r0 + wave * 32 + i;
    const bool valid = r < rows;
    const int tok = (int)(r / group), head = hk * group + (int)(r - (int64_t)tok * group);
    const int pos = sq.q.p0 + tok;
    int lo = 1, hi = 0, lo_max = 0, hi_min = INT32_MAX, lo_min = INT32_MAX, hi_max = -1;
    v8h qf[NC];
    float f, slope = 0.0f, l = 0.0f;
    float M = 0.0f, limit = -1.0f;  // limit: the sum of weights that moves M; any, before the first visible key
    {
        Raw8<DT> raw[NC];
        const uint16_t* row = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(sq.q.q0 + tok) * a.ldq + (int64_t)head * D;
        float top = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            raw[c] = valid ? load_raw8<DT>(row, 2 * c + h) : zero_raw8<DT>();
            if constexpr (DT == kBF16) {
                float x[8];
                widen8<DT>(raw[c], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(x[j]));
            }
        }
        int e = 14;
        if constexpr (DT == kBF16) {
            top = fmaxf(top, __shfl_xor(top, 32));
            e = row_exponent(top);
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if constexpr (DT == kBF16) {
                float x[8];
                widen8<DT>(raw[c], x);
#pragma unroll
                for (int j = 0; j < 8; ++j) qf[c][j] = (_Float16)ldexpf(x[j], 14 - e);
            } else {
                qf[c] = __builtin_bit_cast(v8h, raw[c].w[0]);
            }
        }
        f = ldexpf(CAP ? 2.0f * kLog2e / a.softcap * a.scale : kLog2e * a.scale, e - 14);
        if (valid) {
            row_keys(a, sq, pos, lo, hi);
            lo_max = lo_min = lo;
            hi_min = hi_max = hi;
            if constexpr (BIAS) slope = a.slopes[head] * kLog2e;
        }
#pragma unroll
        for (int m = 16; m >= 1; m >>= 1) {
            lo_max = max(lo_max, __shfl_xor(lo_max, m));
            lo_min = min(lo_min, __shfl_xor(lo_min, m));
            hi_min = min(hi_min, __shfl_xor(hi_min, m));
            hi_max = max(hi_max, __shfl_xor(hi_max, m));
        }
        lo_max = __builtin_amdgcn_readfirstlane(lo_max);
        lo_min = __builtin_amdgcn_readfirstlane(lo_min);
        hi_min = __builtin_amdgcn_readfirstlane(hi_min);
        hi_max = __builtin_amdgcn_readfirstlane(hi_max);
    }
    const float cap2 = a.softcap * kLog2e;
    v16f o[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[t][k] = 0.0f;

    // staging: a wave brings 64 / NW tokens of K, and 8 / NW pieces' rows of V, of one 16 tokens of a step
    const int32_t* table = a.b.page_table + (int64_t)s * a.b.ldt;
    const int shift = __builtin_ctz(a.c.page);
    const int mine = wave * NU / NW;  // the 16 tokens of a step that this wave brings
    constexpr int KL = D / KB, VL = D / VD;  // lanes of a token of K, of a row of V
    const int kt = wave * (kKeys / NW) + lane / KL, kj = lane % KL;       // token of the step, part of its channels
    const int vp = wave * (kKeys / 8 / NW) + lane / VL, vd = lane % VL * VD;  // 2 u + h, first channel
    uint4 rk[KB / 16];
    uint2 rv[2][VD / 2];
    float2 rs;
    bool rs_there;
    // Page numbers and scales come by vector loads, issued before the codes that they are used with or after: scalar
    // loads would have to arrive before the next barrier, which waits for the counter that LDS and they share.
    auto page_at = [&](int t0) -> int { return table[min(t0 + 16 * mine, end - 1) >> shift]; };
    // Where a step's 16 tokens of this wave lie in the pool: the same for K and V.  Without a page of the pool page 0
    // is loaded and not seen (with no pool at all no sequence has keys).
    const uint32_t page_bytes = (uint32_t)(a.c.heads * a.c.page * D), head_bytes = (uint32_t)(hk * a.c.page * D);
    const uint32_t k_lane = (kt & 15) * D + kj * KB, v_lane = (vp & 1) * (4 * D) + vd * 4;
    auto load = [&](int t0, int id) {
        const uint32_t p = (uint32_t)__builtin_amdgcn_readfirstlane(id);
        rs_there = p < (uint32_t)a.c.pages && t0 + 16 * mine < end;
        const uint32_t page = rs_there ? p : 0u, slot = (t0 + 16 * mine) & (a.c.page - 1);
        const uint64_t at = (uint64_t)page * page_bytes + (head_bytes + slot * D);
        const uint64_t s = (uint64_t)page * (uint32_t)a.c.heads + (uint32_t)hk;
        rs = make_float2(a.c.k_scale[s], a.c.v_scale[s]);
#pragma unroll
        for (int w = 0; w < KB / 16; ++w) rk[w] = *reinterpret_cast<const uint4*>(a.c.k + at + (k_lane + 16 * w));
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int w = 0; w < VD / 2; ++w)
                rv[q][w] = *reinterpret_cast<const uint2*>(a.c.v + at + (v_lane + q * 8 * D + 8 * w));
    };
    auto put_k = [&](KeyStage<D>& st) {
        uint8_t* p = st.at + kj * (KB / 8) * KeyStage<D>::kPitch + kt * 16;
#pragma unroll
        for (int w = 0; w < KB / 16; ++w) {
            *reinterpret_cast<v8h*>(p + (2 * w) * KeyStage<D>::kPitch) = join(codes4(rk[w].x), codes4(rk[w].y));
            *reinterpret_cast<v8h*>(p + (2 * w + 1) * KeyStage<D>::kPitch) = join(codes4(rk[w].z), codes4(rk[w].w));
        }
    };
    auto put_v = [&](ValueStage<D>& st) {
        uint8_t* p = st.at + vp * ValueStage<D>::kPitch;
#pragma unroll
        for (int w = 0; w < VD / 2; ++w) {
            const int t = (vd + 2 * w) % NT, m = (vd + 2 * w) / NT;
            *reinterpret_cast<v8h*>(p + ValueStage<D>::piece(t, m)) = join(codes4(rv[0][w].x), codes4(rv[1][w].x));
            *reinterpret_cast<v8h*>(p + ValueStage<D>::piece(t + 1, m)) = join(codes4(rv[0][w].y), codes4(rv[1][w].y));
        }
        if (lane == 0) {
            // a scale that is not finite reaches the weights of the keys that are seen; hidden ones add 0 times 0 to l
            const float inv = __builtin_amdgcn_rcpf(rs.y);
            st.scale[mine] = make_float4(rs.x, __log2f(rs.y), fabsf(inv) < INFINITY ? inv : 0.0f, rs_there ? 1.0f : 0.0f);
        }
    };

    struct Scores {
        v16f z[KU];
    };
    auto products = [&](const KeyStage<D>& st, Scores& x) {
#pragma unroll
        for (int u = 0; u < KU; ++u)
#pragma unroll
            for (int k = 0; k < 16; ++k) x.z[u][k] = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int u = 0; u < KU; ++u) {
                const v8h kf = *reinterpret_cast<const v8h*>(st.at + (2 * c + h) * KeyStage<D>::kPitch + (32 * u + i) * 16);
                x.z[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[c], x.z[u], 0, 0, 0);
            }
        if constexpr (kAhead > 0) {
            __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);
#pragma unroll
            for (int j = 0; j < KU * NC; ++j) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (j < KU * NC - kAhead) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
        }
    };
    // the weights of 16 tokens (u) from their exponents: as an operand, and their sum
    auto weights = [&](const Scores& x, int u, v8h& pf) {
        float p[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) p[k] = exp2_(x.z[u >> 1][8 * (u & 1) + k]);
        pf = __builtin_bit_cast(v8h, make_uint4(f32x2_to_16<kF16>(p[0], p[1]), f32x2_to_16<kF16>(p[2], p[3]),
                                                f32x2_to_16<kF16>(p[4], p[5]), f32x2_to_16<kF16>(p[6], p[7])));
        return ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    };
    auto step = [&](int t0, const KeyStage<D>& kst, const ValueStage<D>& vst) {
        float4 sc[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) sc[u] = vst.scale[u];
        Scores x;
        products(kst, x);
        bool pages = true;
#pragma unroll
        for (int u = 0; u < NU; ++u) pages &= sc[u].w != 0.0f;
        auto exponents = [&](auto masked) {
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const float fs = f * sc[u].x;
                float base = sc[u].y - M;
                // the bias: slope (t0 + 4 h - pos), and the rest of the key's distance times slope
                if constexpr (BIAS) base = __builtin_fmaf(slope, (float)(t0 + 4 * h - pos), base);
                // the cap: cap (1 - 2 / (2^(2 x log2 e) + 1)), the constant part with the base
                if constexpr (CAP) base += cap2;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float e = x.z[u >> 1][8 * (u & 1) + k];
                    const int off = 16 * u + 8 * (k >> 2) + (k & 3);
                    const float add = BIAS ? __builtin_fmaf(slope, (float)off, base) : base;
                    if constexpr (CAP)
                        e = __builtin_fmaf(-2.0f * cap2, __builtin_amdgcn_rcpf(exp2_(e * fs) + 1.0f), add);
                    else
                        e = __builtin_fmaf(e, fs, add);
                    if constexpr (masked.value) {
                        const int key = t0 + 4 * h + off;
                        e = key >= lo && key <= hi && sc[u].w != 0.0f ? e : -INFINITY;
                    }
                    x.z[u >> 1][8 * (u & 1) + k] = e;
                }
            }
        };
        if (t0 < lo_max || t0 + kKeys - 1 > hi_min || !pages)
            exponents(std::true_type{});
        else
            exponents(std::false_type{});
        v8h pf[NU], vf[NU][NT];
        auto values = [&](int u) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
                vf[u][t] = *reinterpret_cast<const v8h*>(vst.at + (2 * u + h) * ValueStage<D>::kPitch + ValueStage<D>::piece(t, i));
        };
#pragma unroll
        for (int u = 0; u < kAhead / NT; ++u) values(u);
        float sum[NU];
#pragma unroll
        for (int u = 0; u < NU; ++u) sum[u] = weights(x, u, pf[u]);
        float most = sum[0];
#pragma unroll
        for (int u = 1; u < NU; ++u) most = fmaxf(most, sum[u]);
        if (__any(most > limit)) {
            // a weight is near binary16's end, or this is a row's first step: M moves
            float top = -INFINITY;
#pragma unroll
            for (int u = 0; u < KU; ++u)
#pragma unroll
                for (int k = 0; k < 16; ++k) top = fmaxf(top, x.z[u][k]);
            top = fmaxf(top, __shfl_xor(top, 32));
            const bool over = fmaxf(most, __shfl_xor(most, 32)) > limit && top > -INFINITY;
            const float by = over ? ceilf(top) - kLift : 0.0f;
            const float keep = !over ? 1.0f : limit < 0.0f ? 0.0f : exp2_(-by);
            if (over) limit = kMost;
            M += by;
            l *= keep;
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] *= keep;
#pragma unroll
            for (int u = 0; u < KU; ++u)
#pragma unroll
                for (int k = 0; k < 16; ++k) x.z[u][k] -= by;
#pragma unroll
            for (int u = 0; u < NU; ++u) sum[u] = weights(x, u, pf[u]);
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            l = __builtin_fmaf(sum[u], sc[u].z, l);
        }
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            if (u >= kAhead / NT) values(u);
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf[u][t], pf[u], o[t], 0, 0, 0);
        }
        if constexpr (kAhead > 0) {
#pragma unroll
            for (int j = 0; j < NU * NT; ++j) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
                if (j < NU * NT - kAhead) __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
            }
        }
    };

    if (begin < end) {
        int id = page_at(begin), next = page_at(begin + kKeys);
        load(begin, id);
        put_k(ks[0]);
        put_v(vs[0]);
        id = page_at(begin + 2 * kKeys);
        load(begin + kKeys, next);
        __syncthreads();
        int buf = 0;
        for (int t0 = begin; t0 < end; t0 += kKeys) {
            if (t0 <= hi_max && t0 + kKeys > lo_min) step(t0, ks[buf], vs[buf]);
            if (t0 + kKeys < end) {
                put_k(ks[buf ^ 1]);
                put_v(vs[buf ^ 1]);
                next = id;
                id = page_at(t0 + 3 * kKeys);
                load(t0 + 2 * kKeys, next);
            }
            __syncthreads();
            buf ^= 1;
        }
    }

    l += __shfl_xor(l, 32);
    if (!valid) return;
    if (limit < 0.0f) M = kNone;
    const int64_t row = sq.q.q0 + tok;
    if (splits > 1) {
        // [split][row][head]: D values, then M and l
        float* p = a.ws + (((int64_t)blockIdx.y * a.b.tokens + row) * a.hq + head) * (D + 2);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const int d = NT * (8 * (k >> 2) + 4 * h + (k & 3));
#pragma unroll
            for (int t = 0; t < NT; t += 2) *reinterpret_cast<float2*>(p + d + t) = make_float2(o[t][k], o[t + 1][k]);
        }
        if (h == 0) *reinterpret_cast<float2*>(p + D) = make_float2(M, l);
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + row * a.ldy + (int64_t)head * D;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const int d = NT * (8 * (k >> 2) + 4 * h + (k & 3));
#pragma unroll
        for (int t = 0; t < NT; t += 2)
            *reinterpret_cast<uint32_t*>(y + d + t) = f32x2_to_16<DT>(o[t][k] * inv, o[t + 1][k] * inv);
    }
    if (a.lse && h == 0) a.lse[row * a.hq + head] = l == 0.0f ? -INFINITY : (M + __log2f(l)) * kLn2;
}

// Joins the parts of each row: D / 8 threads a row.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_attention_prompt_join(AttentionArgs a, int splits) {
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = u / (D / 8);
    const int d = (int)(u - row * (D / 8)) * 8;
    const int64_t rows = (int64_t)a.b.tokens * a.hq;
    if (row >= rows) return;
    const int64_t t = row / a.hq;
    if (a.b.cu_q && (t < a.b.cu_q[0] || t >= a.b.cu_q[a.b.batch])) return;
    const float* p = a.ws + row * (D + 2);
    const int64_t step = rows * (D + 2);
    float M = kNone, l = 0.0f, o[8] = {};
#pragma unroll 8
    for (int w = 0; w < splits; ++w, p += step) {
        const float2 ml = *reinterpret_cast<const float2*>(p + D);
        const float now = fmaxf(M, ml.x), fo = exp2_(M - now), fw = exp2_(ml.x - now);
        M = now;
        l = l * fo + ml.y * fw;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const float2 v = *reinterpret_cast<const float2*>(p + d + k);
            o[k] = o[k] * fo + v.x * fw;
            o[k + 1] = o[k + 1] * fo + v.y * fw;
        }
    }
    const int head = (int)(row - t * a.hq);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint4 w;
    w.x = f32x2_to_16<DT>(o[0] * inv, o[1] * inv);
    w.y = f32x2_to_16<DT>(o[2] * inv, o[3] * inv);
    w.z = f32x2_to_16<DT>(o[4] * inv, o[5] * inv);
    w.w = f32x2_to_16<DT>(o[6] * inv, o[7] * inv);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.y) + t * a.ldy + (int64_t)head * D + d) = w;
    if (a.lse && d == 0) a.lse[row] = l == 0.0f ? -INFINITY : (M + __log2f(l)) * kLn2;
}

int64_t prompt_items(const AttentionArgs& a) {
    const int group = a.hq / a.c.heads, kRows = tile_rows(a.c.dim);
    return a.b.cu_q ? (int64_t)a.b.tokens * group / kRows + a.b.batch
                    : (int64_t)a.b.batch * ((group + kRows - 1) / kRows);
}

template <int DT, int D>
void launch(const AttentionArgs& a, int splits, hipStream_t st) {
    const int64_t items = prompt_items(a);
    const dim3 grid((uint32_t)(items * a.c.heads), splits);
    if (a.softcap > 0.0f) {
        if (a.slopes) k_attention_prompt<DT, D, true, true><<<grid, 64 * waves(D), 0, st>>>(a, items, splits);
        else k_attention_prompt<DT, D, true, false><<<grid, 64 * waves(D), 0, st>>>(a, items, splits);
    } else {
        if (a.slopes) k_attention_prompt<DT, D, false, true><<<grid, 64 * waves(D), 0, st>>>(a, items, splits);
        else k_attention_prompt<DT, D, false, false><<<grid, 64 * waves(D), 0, st>>>(a, items, splits);
    }
    if (splits > 1) {
        const int64_t n = (int64_t)a.b.tokens * a.hq * (D / 8);
        k_attention_prompt_join<DT, D><<<(uint32_t)((n + 255) / 256), 256, 0, st>>>(a, splits);
    }
}

}  // namespace

// Workgroups that the chip holds at once, and row tiles of a batch (of sequences
// of the average length, times heads).
static int64_t slots(int dim) { return 256 * per_simd(dim) * 4 / waves(dim); }
static int64_t tiles(int64_t tokens, int64_t batch, int hq, int hkv, int dim) {
    const int64_t each = (tokens * (hq / hkv) + batch - 1) / batch;
    return (each + tile_rows(dim) - 1) / tile_rows(dim) * batch * hkv;
}

int attention_prompt_most_splits(int64_t tokens, int64_t batch, int hq, int hkv, int dim) {
    return (int)std::min<int64_t>(32, std::max<int64_t>(1, 2 * slots(dim) / tiles(tokens, batch, hq, hkv, dim)));
}

// Parts of the keys that each tile of rows is cut into: the fewest microseconds
// of rounds of workgroups, each some 6 and 2 a step, and of the join, some 4 and
// 0.4 a part.  keys: what the table can name; a window that hides most of them is not
// known here, so windowed chunks are cut more than they need (700 rows, window 128: 31 us, 17 uncut).
// The constants are those of 128 channels and serve 64 and 256 too.  us in 8 / 16 / 32 parts and in the rule's:
//                                  64 channels            128                    256
//   110 tokens, 4842 keys, 1 head  25 / 24 / 31, 19: 23   37 / 31 / 38, 19: 31   50 / 39 / 44, 19: 38
//   512 tokens, 2000 keys, 1 head  19 / 22 / 33, 11: 19   26 / 30 / 42, 11: 27   35 / 38 / 56, 11: 35
//   130 tokens, 16000 keys, 8 (4)  69 / 58 / 66, 18: 55   83 / 97 / 104, 10: 72  122 / 134 / 136, 12: 92
// (key/value heads, each with two query heads, in the last row with four).
int attention_prompt_splits(int64_t tokens, int64_t batch, int hq, int hkv, int dim, int64_t keys) {
    const int most = attention_prompt_most_splits(tokens, batch, hq, hkv, dim);
    const int64_t n = tiles(tokens, batch, hq, hkv, dim), steps = (keys + kKeys - 1) / kKeys;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= most; ++s) {
        const double rounds = (double)((n * s + slots(dim) - 1) / slots(dim));
        const double t = rounds * (6.0 + 2.0 * (double)((steps + s - 1) / s)) + (s > 1 ? 4.0 + 0.4 * s : 0.0);
        if (t < least) {
            least = t;
            best = s;
        }
    }
    return best;
}

int64_t attention_prompt_threads(const AttentionArgs& a, int splits) {
    return std::max(prompt_items(a) * a.c.heads * splits * 64 * waves(a.c.dim), (int64_t)a.b.tokens * a.hq * (a.c.dim / 8));
}

void launch_attention_prompt(const AttentionArgs& a, int dt, int splits, hipStream_t st) {
    if (dt == kBF16) {
        if (a.c.dim == 64) launch<kBF16, 64>(a, splits, st);
        else if (a.c.dim == 128) launch<kBF16, 128>(a, splits, st);
        else launch<kBF16, 256>(a, splits, st);
    } else {
        if (a.c.dim == 64) launch<kF16, 64>(a, splits, st);
        else if (a.c.dim == 128) launch<kF16, 128>(a, splits, st);
        else launch<kF16, 256>(a, splits, st);
    }
}

}  // namespace pdq

// Attention over the paged INT8 key/value cache, many rows for each sequence
// (prompts, chunks of prompts): bound by the matrix products and the softmax
// between them.  include/pdq.h (pdq_kv_attention) states the arithmetic,
// attention_device.h how it is taken.
#include <algorithm>

#include "attention_device.h"

namespace pdq {

namespace {

constexpr int kRows = 128;  // rows of a workgroup: four waves of 32
constexpr int kKeys = 64;   // keys of a step

// LDS of one step's operands, in 16-byte pieces of 8 binary16 values.
// K: piece (c, t) = channels 8 c .. 8 c + 7 of token t.  V: piece (2 u + h, d) =
// channel (D / 32) (d % 32) + d / 32 of the tokens 4 h .. 4 h + 3 and 8 + 4 h .. 8 +
// 4 h + 3 of the u-th 16 tokens, the order in which a lane of half h holds its
// weights.  A lane of a product reads the piece of its own row, a whole half wave
// 512 contiguous bytes; rows of pieces are padded so that the conversion's
// writes (four lanes to a token) fall into different banks too.
template <int D>
struct Stage {
    static constexpr int kPitchK = kKeys * 16 + (D == 64 ? 32 : 16), kPitchV = D * 16 + 16;
    uint8_t k[D / 8 * kPitchK];
    uint8_t v[8 * kPitchV];
    float4 scale[4];  // of each 16 tokens: S_k (0 without a page), log2 S_v, 1 / S_v, 0 or 1: a page is there
};

// One workgroup of four waves takes kRows rows (token, query head of the group)
// of one key/value head over a part of their keys.  Scores are computed
// transposed, keys x rows, in 32x32x16 products, so that a row's scores lie in
// one lane (and the one 32 lanes on) and its weights are the operand of the
// value product as they stand; the output is accumulated transposed too.  Each
// step's codes are loaded a step ahead, converted once for the four waves and
// staged in one of two LDS buffers: one barrier a step.
template <int DT, int D>
__global__ __launch_bounds__(256, D <= 128 ? 2 : 1) void k_attention_prompt(AttentionArgs a, int64_t items, int splits) {
    constexpr int NC = D / 16, NT = D / 32, KW = D / 64, VB = D / 8;  // VB: bytes of a lane's V channels of a quad
    __shared__ Stage<D> stage[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 31, h = lane >> 5;
    const int group = a.hq / a.c.heads;
    const int hk = blockIdx.x % a.c.heads;
    const int64_t item = items - 1 - blockIdx.x / a.c.heads;  // the last rows of a prompt see most: first
    const int s = a.b.cu_q ? item_seq(a.b, item, group, kRows, 1) : (int)(item / ((group + kRows - 1) / kRows));
    const int64_t tile = a.b.cu_q ? item - item_start(a.b, s, group, kRows, 1)
                                  : item - (int64_t)s * ((group + kRows - 1) / kRows);
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
    float M = 0.0f, limit = -INFINITY;  // limit: the exponent less M that moves M; any, before the first visible key
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
            e = top > 0.0f && top < INFINITY ? __builtin_amdgcn_frexp_expf(top) : 14;
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
        f = ldexpf(a.softcap > 0.0f ? 2.0f * kLog2e / a.softcap * a.scale : kLog2e * a.scale, e - 14);
        if (valid) {
            row_keys(a, sq, pos, lo, hi);
            lo_max = lo_min = lo;
            hi_min = hi_max = hi;
            if (a.slopes) slope = a.slopes[head] * kLog2e;
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

    // staging: this wave brings the wave-th 16 tokens of a step
    const int32_t* table = a.b.page_table + (int64_t)s * a.b.ldt;
    const int shift = __builtin_ctz(a.c.page);
    uint4 rk[KW];
    uint2 rv[2][VB / 8];
    float4 rs;
    const int kt = lane >> 2, kj = lane & 3;  // token of the 16, quarter of its channels
    auto page_at = [&](int t0) -> int {
        const int t = t0 + 16 * wave;
        return t < end ? uniform_load(table + (t >> shift)) : -1;
    };
    auto load = [&](int t0, int id) {
        // without a page of the pool page 0 is loaded and not seen (with no pool at all no sequence has keys)
        const bool there = (uint32_t)id < (uint32_t)a.c.pages;
        const int64_t at = (int64_t)(there ? id : 0) * a.c.heads + hk;
        const int64_t base = (at * a.c.page + ((t0 + 16 * wave) & (a.c.page - 1))) * D;
        const uint4* kp = reinterpret_cast<const uint4*>(a.c.k + base + kt * D + kj * (D / 4));
#pragma unroll
        for (int w = 0; w < KW; ++w) rk[w] = kp[w];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint2* vp = reinterpret_cast<const uint2*>(a.c.v + base + (h + 2 * q) * (4 * D) + i * VB);
#pragma unroll
            for (int w = 0; w < VB / 8; ++w) rv[q][w] = vp[w];
        }
        rs = make_float4(uniform_load(a.c.k_scale + at), uniform_load(a.c.v_scale + at), 0.0f, there ? 1.0f : 0.0f);
    };
    auto put = [&](Stage<D>& st) {
        uint8_t* k = st.k + (kj * (D / 32)) * Stage<D>::kPitchK + (16 * wave + kt) * 16;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            *reinterpret_cast<v8h*>(k + (2 * w) * Stage<D>::kPitchK) = join(codes4(rk[w].x), codes4(rk[w].y));
            *reinterpret_cast<v8h*>(k + (2 * w + 1) * Stage<D>::kPitchK) = join(codes4(rk[w].z), codes4(rk[w].w));
        }
        uint8_t* v = st.v + (2 * wave + h) * Stage<D>::kPitchV + i * 16;
#pragma unroll
        for (int w = 0; w < VB / 8; ++w) {
            *reinterpret_cast<v8h*>(v + (2 * w) * 512) = join(codes4(rv[0][w].x), codes4(rv[1][w].x));
            *reinterpret_cast<v8h*>(v + (2 * w + 1) * 512) = join(codes4(rv[0][w].y), codes4(rv[1][w].y));
        }
        if (lane == 0) st.scale[wave] = make_float4(rs.x, __log2f(rs.y), __builtin_amdgcn_rcpf(rs.y), rs.w);
    };

    auto compute = [&](int t0, const Stage<D>& st) {
        v16f z[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < 16; ++k) z[u][k] = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const v8h kf = *reinterpret_cast<const v8h*>(st.k + (2 * c + h) * Stage<D>::kPitchK + (32 * u + i) * 16);
                z[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[c], z[u], 0, 0, 0);
            }
        float4 sc[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) sc[u] = st.scale[u];
        const bool pages = sc[0].w * sc[1].w * sc[2].w * sc[3].w != 0.0f;
        const bool masked = t0 < lo_max || t0 + kKeys - 1 > hi_min || !pages;
        float top = -INFINITY;
        if (a.softcap > 0.0f || a.slopes) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float fs = f * sc[u].x;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float y = z[u >> 1][8 * (u & 1) + k] * fs;
                    if (a.softcap > 0.0f) y = capped(y, cap2);
                    if (a.slopes) y += slope * (float)(t0 + 16 * u + 8 * (k >> 2) + 4 * h + (k & 3) - pos);
                    z[u >> 1][8 * (u & 1) + k] = y + (sc[u].y - M);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float fs = f * sc[u].x, base = sc[u].y - M;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    z[u >> 1][8 * (u & 1) + k] = __builtin_fmaf(z[u >> 1][8 * (u & 1) + k], fs, base);
            }
        }
        if (masked) {
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int key = t0 + 16 * u + 8 * (k >> 2) + 4 * h + (k & 3);
                    const float y = z[u >> 1][8 * (u & 1) + k];
                    z[u >> 1][8 * (u & 1) + k] = key >= lo && key <= hi && sc[u].w != 0.0f ? y : -INFINITY;
                }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int k = 0; k < 16; ++k) top = fmaxf(top, z[u][k]);
        // z is the exponent less M already
        if (__any(top > limit)) {
            top = fmaxf(top, __shfl_xor(top, 32));
            if (top > limit) {
                const float by = ceilf(top) - kLift;
                const float keep = limit < 0.0f ? 0.0f : exp2_(-by);
                limit = kLift + kSlack;
                M += by;
                l *= keep;
#pragma unroll
                for (int t = 0; t < NT; ++t) o[t] *= keep;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int k = 0; k < 16; ++k) z[u][k] -= by;
            }
        }
        v8h pf[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float p[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) p[k] = exp2_(z[u >> 1][8 * (u & 1) + k]);
            const float sum = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
            l += sum == 0.0f ? 0.0f : sum * sc[u].z;  // hidden keys of a page whose scale is not finite: 0
            pf[u] = __builtin_bit_cast(v8h, make_uint4(f32x2_to_16<kF16>(p[0], p[1]), f32x2_to_16<kF16>(p[2], p[3]),
                                                       f32x2_to_16<kF16>(p[4], p[5]), f32x2_to_16<kF16>(p[6], p[7])));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const v8h vf = *reinterpret_cast<const v8h*>(st.v + (2 * u + h) * Stage<D>::kPitchV + (32 * t + i) * 16);
                o[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pf[u], o[t], 0, 0, 0);
            }
    };

    if (begin < end) {
        load(begin, page_at(begin));
        put(stage[0]);
        load(begin + kKeys, page_at(begin + kKeys));
        int id = page_at(begin + 2 * kKeys);
        __syncthreads();
        int buf = 0;
        for (int t0 = begin; t0 < end; t0 += kKeys) {
            if (t0 <= hi_max && t0 + kKeys > lo_min) compute(t0, stage[buf]);
            if (t0 + kKeys < end) {
                put(stage[buf ^ 1]);
                load(t0 + 2 * kKeys, id);
                id = page_at(t0 + 3 * kKeys);
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
    const int group = a.hq / a.c.heads;
    return a.b.cu_q ? (int64_t)a.b.tokens * group / kRows + a.b.batch
                    : (int64_t)a.b.batch * ((group + kRows - 1) / kRows);
}

template <int DT, int D>
void launch(const AttentionArgs& a, int splits, hipStream_t st) {
    const int64_t items = prompt_items(a);
    k_attention_prompt<DT, D><<<dim3((uint32_t)(items * a.c.heads), splits), 256, 0, st>>>(a, items, splits);
    if (splits > 1) {
        const int64_t n = (int64_t)a.b.tokens * a.hq * (D / 8);
        k_attention_prompt_join<DT, D><<<(uint32_t)((n + 255) / 256), 256, 0, st>>>(a, splits);
    }
}

}  // namespace

// Parts of the keys that each tile of rows is cut into: what fills the chip's
// workgroup slots (two a compute unit, one with 256 channels) in the fewest
// rounds of the shortest parts, a part more counted as 2% for its partial
// results.
int attention_prompt_splits(int64_t tokens, int hq, int hkv, int dim) {
    const int64_t slots = dim == 256 ? 256 : 512;
    const int64_t tiles = (tokens * (hq / hkv) + kRows - 1) / kRows * hkv;
    int best = 1;
    double least = 1e30;
    for (int s = 1; s <= 16 && tiles < slots; ++s) {
        const double t = (double)((tiles * s + slots - 1) / slots) / s * (1.0 + 0.02 * s);
        if (t < least) {
            least = t;
            best = s;
        }
    }
    return best;
}

int64_t attention_prompt_threads(const AttentionArgs& a, int splits) {
    return std::max(prompt_items(a) * a.c.heads * splits * 256, (int64_t)a.b.tokens * a.hq * (a.c.dim / 8));
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

// Attention over the paged INT8 key/value cache, few rows for each sequence
// (decode; drafted tokens): bound by reading the cache.  include/pdq.h
// (pdq_kv_attention) states the arithmetic, attention_device.h how it is taken.
#include <algorithm>

#include "attention_device.h"

namespace pdq {

namespace {

constexpr int kStep = 128;  // tokens of a step: four waves of 32

// The work: units of kStep keys, numbered over (sequence, key/value head, tile
// of R rows, step), cut into equal ranges, one for each workgroup,
// whatever the lengths are.  A (sequence, head, row tile) that lies in one range
// is written out by its workgroup; one that is cut leaves a partial result (the
// unnormalised output, M and l of each row) in each range's slot (2 w: the
// range's first segment; 2 w + 1: its last), and the second kernel joins them.
struct Units {
    AttnSeq s;
    int tiles, steps, k0;  // row tiles; steps of one (head, tile); first key, a multiple of 32
    int64_t all;           // heads * tiles * steps
};

template <int R, bool Uniform = false>
__device__ __forceinline__ Units units_of(const AttentionArgs& a, int s) {
    Units u;
    u.s = attn_seq<Uniform>(a, s);
    u.tiles = (u.s.q.n * (a.hq / a.c.heads) + R - 1) / R;
    u.k0 = u.s.k0 & ~31;
    u.steps = u.s.last < u.k0 ? 1 : (u.s.last - u.k0) / kStep + 1;
    u.all = (int64_t)a.c.heads * u.tiles * u.steps;
    return u;
}

// Workgroups of the few-row kernel that the chip holds at once, one range each: as many as a
// compute unit's registers hold without spilling.  With 128 channels two against three and four, joins included: 32
// sequences up to 4096 keys 43 us against 53 and 68, one of 131071 51 against 58 and 99, 96 up to 16384 354 against 355
// and 516.  With 256 channels a lane takes 394 registers; held to the 256 of two workgroups it spills, and 24 sequences of
// up to five rows and 6011 keys take 66 us instead of 51.
constexpr int resident(int D, int NQ) { return D == 256 ? 1 : D == 128 ? 2 : NQ == 1 ? 4 : 2; }
constexpr int ways(int D, int R) { return 256 * resident(D, R / 16); }

// Range w of W: floor(w all / W), or one unit each while there are fewer units
// than ranges.  range_of is the range that holds unit u.
template <int W>
__device__ __forceinline__ int64_t range_start(int64_t all, int w) {
    if (all < W) return min((int64_t)w, all);
    const uint32_t r = (uint32_t)((uint64_t)all % W);
    return w * (int64_t)((uint64_t)all / W) + (uint32_t)(w * r) / W;
}

template <int W>
__device__ __forceinline__ int range_of(int64_t all, int64_t u) {
    if (all < W) return (int)u;
    if (all < (int64_t)0xffffffffu / W) return (int)((uint32_t)((u + 1) * W - 1) / (uint32_t)all);
    return (int)(((u + 1) * W - 1) / all);
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int lane) {
    const int lo = __shfl((int)v, lane), hi = __shfl((int)(v >> 32), lane);
    return (int64_t)hi << 32 | (uint32_t)lo;
}

__device__ __forceinline__ int64_t quotient(int64_t a, int b) {
    return (uint64_t)a >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Inclusive sums over the workgroup's 256 threads, and the total.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* part, int64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t o = shfl64(v, max(lane - d, 0));
        if (lane >= d) v += o;
    }
    __syncthreads();
    if (lane == 63) part[wave] = v;
    __syncthreads();
    total = part[0] + part[1] + part[2] + part[3];
    for (int w = 0; w < wave; ++w) v += part[w];
    return v;
}

// The workspace: for each range two slots of R rows of D values, then M and l of
// each row; then for each segment where its parts are: the slot of the first, and
// the last range (-1: written out whole).
template <int D, int R>
__device__ __forceinline__ float* slot_of(const AttentionArgs& a, int64_t slot) {
    return a.ws + slot * (R * (D + 2));
}

template <int D, int R>
__device__ __forceinline__ int2* parts_of(const AttentionArgs& a, int64_t item, int hk) {
    return reinterpret_cast<int2*>(slot_of<D, R>(a, 2 * ways(D, R))) + item * a.c.heads + hk;
}

// The number of a sequence's first row tile.
template <int R>
__device__ __forceinline__ int64_t first_item(const AttentionArgs& a, int s) {
    return item_start(a.b, s, a.hq / a.c.heads, R, 1);
}

template <int DT, int D>
__device__ __forceinline__ void write_row(const AttentionArgs& a, int64_t row, int head, int d, const float (&o)[8],
                                          float M, float l) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint4 w;
    w.x = f32x2_to_16<DT>(o[0] * inv, o[1] * inv);
    w.y = f32x2_to_16<DT>(o[2] * inv, o[3] * inv);
    w.z = f32x2_to_16<DT>(o[4] * inv, o[5] * inv);
    w.w = f32x2_to_16<DT>(o[6] * inv, o[7] * inv);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.y) + row * a.ldy + (int64_t)head * D + d) = w;
    if (a.lse && d == 0)
        a.lse[row * a.hq + head] = l == 0.0f ? -INFINITY : (M + __log2f(l)) * kLn2;
}

// One workgroup of four waves.  A wave takes every fourth tile of 32 tokens of
// its segment straight from memory into the operands of 16x16x32 products: lane
// (i = lane % 16, g = lane / 16) holds channels g D/4 .. of token i as K, and
// channels i D/16 .. of tokens 4 g .. 4 g + 3 as V; scores come out with a row
// of queries in lane i and tokens 4 g .. 4 g + 3 in its registers, which is the
// weights' operand of the value product as it stands.  The next tile's codes are
// loaded while one is computed, the next segment's first tile while one is
// written out.
//
// Bound by the cache's bytes, 2 D a key and head, at long contexts (one read at
// the card's best, 6.2 TB/s): 96 sequences up to 16384 keys (1.93 GB) 341 us, 5.7
// TB/s; one of 131071 (268 MB) 52 us, 5.2 TB/s, of which some 5 us are its begin:
// lengths, range, page, codes, one after the other.  32 sequences up to 4096 (139
// MB) 38 us, 3.7 TB/s: beside the begin, the 1.5 segments of a workgroup.  The
// equal ranges are what ragged lengths need.  K straight into the operand layout
// keeps LDS out of the loop; converting the codes takes 160 of some 250 vector
// instructions a tile, 22% of the time at most.
template <int DT, int D, int NQ>
__global__ __launch_bounds__(256, resident(D, NQ)) void k_attention_few(AttentionArgs a) {
    constexpr int R = 16 * NQ, W = ways(D, R), DL = D / 4, NC = D / 32, NT = D / 16, W4 = D / 64;
    constexpr int kPitch = D + 4;
    __shared__ float so[4][16][kPitch];
    __shared__ float sM[4][R], sl[4][R];
    __shared__ int64_t part[4];
    __shared__ int64_t found[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), i = lane & 15, g = lane >> 4;
    const int group = a.hq / a.c.heads;

    // this workgroup's range, and the sequence that it begins in
    int64_t total = 0, u0, u1;
    {
        int64_t mine = 0, incl = 0, t;
        for (int base = 0; base < a.b.batch; base += 256) {
            mine = base + tid < a.b.batch ? units_of<R>(a, base + tid).all : 0;
            incl = block_scan(mine, part, t);
            total += t;
        }
        u0 = range_start<W>(total, blockIdx.x);
        u1 = range_start<W>(total, blockIdx.x + 1);
        if (u0 >= u1) return;
        int64_t before = 0;
        for (int base = 0; base < a.b.batch; base += 256) {
            if (a.b.batch > 256) {
                mine = base + tid < a.b.batch ? units_of<R>(a, base + tid).all : 0;
                incl = block_scan(mine, part, t);
            } else {
                t = total;
            }
            if (before + incl > u0 && before + incl - mine <= u0) {
                found[0] = base + tid;
                found[1] = before + incl - mine;
            }
            before += t;
            if (before > u0) break;
        }
        __syncthreads();
    }
    // a segment of the range, or what of it the range holds: steps step0 .. step0 + steps - 1 of row tile `tile`
    // of head hk of sequence s
    struct Segment {
        Units un;
        int64_t from;  // the first unit of the sequence
        int s, hk, tile, step0, steps;
        int begin, end;  // this wave's first tile of 32 keys; the keys' end
        const int32_t* table;
    } sg;
    sg.s = __builtin_amdgcn_readfirstlane((int)found[0]);
    sg.from = found[1];
    sg.un = units_of<R, true>(a, sg.s);
    const int shift = __builtin_ctz(a.c.page);
    auto find = [&](int64_t u) {  // the segment that holds unit u, at or behind the present one
        while (u - sg.from >= sg.un.all) {
            sg.from += sg.un.all;
            sg.s = min(sg.s + 1, a.b.batch - 1);
            sg.un = units_of<R, true>(a, sg.s);
            if (sg.s == a.b.batch - 1) break;  // lengths that changed under the call: stay within the batch
        }
        const int64_t local = u - sg.from;
        const int64_t seg = quotient(local, sg.un.steps);
        sg.step0 = __builtin_amdgcn_readfirstlane((int)(local - seg * sg.un.steps));
        sg.hk = min(__builtin_amdgcn_readfirstlane((int)quotient(seg, max(sg.un.tiles, 1))), a.c.heads - 1);
        sg.tile = (int)min((int64_t)(max(sg.un.tiles, 1) - 1), seg - (int64_t)sg.hk * sg.un.tiles);
        sg.tile = __builtin_amdgcn_readfirstlane(sg.tile);
        sg.steps = __builtin_amdgcn_readfirstlane((int)min((int64_t)(sg.un.steps - sg.step0), u1 - u));
        sg.begin = sg.un.k0 + (sg.step0 * 4 + wave) * 32;
        sg.end = min(sg.un.k0 + (sg.step0 + sg.steps) * kStep, sg.un.s.last + 1);
        sg.table = a.b.page_table + (int64_t)sg.s * a.b.ldt;
    };

    // a tile's two groups of 16 tokens: whether the table names a page of the pool for them (if not, page 0 is loaded
    // and not seen: with no pool at all no sequence has keys), its scales and codes
    struct Tile {
        bool there[2];
        float ks[2], vs[2];
        uint4 k[2][W4], v[2][W4];
    };
    auto pages = [&](int t0, int (&id)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = t0 + 16 * u;
            id[u] = t < sg.end ? uniform_load(sg.table + (t >> shift)) : -1;
        }
    };
    auto load = [&](int t0, const int (&id)[2], Tile& x) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            x.there[u] = (uint32_t)id[u] < (uint32_t)a.c.pages;
            const int64_t at = (int64_t)(x.there[u] ? id[u] : 0) * a.c.heads + sg.hk;
            const int slot = (t0 + 16 * u) & (a.c.page - 1);
            const int64_t base = (at * a.c.page + slot) * D;
            const uint4* kp = reinterpret_cast<const uint4*>(a.c.k + base + i * D + g * DL);
            const uint4* vp = reinterpret_cast<const uint4*>(a.c.v + base + g * (4 * D) + i * DL);
#pragma unroll
            for (int w = 0; w < W4; ++w) x.k[u][w] = kp[w];
#pragma unroll
            for (int w = 0; w < W4; ++w) x.v[u][w] = vp[w];
            x.ks[u] = uniform_load(a.c.k_scale + at);
            x.vs[u] = uniform_load(a.c.v_scale + at);
        }
    };
    // what a segment begins with: its first tile, and its rows' queries
    Tile x, y;
    int id[2];
    Raw8<DT> raw[NQ][DL / 8];
    auto queries = [&]() {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int r = sg.tile * R + n * 16 + i;
            const int tok = r / group, head = sg.hk * group + r - tok * group;
            const uint16_t* row = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(sg.un.s.q.q0 + tok) * a.ldq +
                                  (int64_t)head * D + g * DL;
#pragma unroll
            for (int c = 0; c < DL / 8; ++c) raw[n][c] = tok < sg.un.s.q.n ? load_raw8<DT>(row, c) : zero_raw8<DT>();
        }
    };
    auto ahead = [&]() {
        if (sg.begin < sg.end) {
            pages(sg.begin, id);
            load(sg.begin, id, x);
            pages(sg.begin + kStep, id);
        }
        if (NQ == 1) queries();  // two row tiles have no registers left for it
    };

    bool first_segment = true;
    find(u0);
    ahead();
    for (;;) {
        if (NQ > 1) queries();
        // the tile's rows: queries as binary16 operands (bfloat16 ones as row_exponent says), the keys that each row sees
        v8h qf[NQ][NC];
        int lo[NQ], hi[NQ], pos[NQ];
        float f[NQ], slope[NQ], M[NQ], l[NQ];
        v4f o[NQ][NT];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            const int r = sg.tile * R + n * 16 + i;
            const int tok = r / group, head = sg.hk * group + r - tok * group;
            pos[n] = sg.un.s.q.p0 + tok;
            lo[n] = 1;
            hi[n] = 0;
            slope[n] = 0.0f;
            if (tok < sg.un.s.q.n) {
                row_keys(a, sg.un.s, pos[n], lo[n], hi[n]);
                if (a.slopes) slope[n] = a.slopes[head] * kLog2e;
            }
            float top = 0.0f, v[DL];
#pragma unroll
            for (int c = 0; c < DL / 8; ++c) {
                float w[8];
                widen8<DT>(raw[n][c], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[8 * c + j] = w[j];
                    top = fmaxf(top, fabsf(w[j]));
                }
            }
            int e = 14;
            if constexpr (DT == kBF16) {
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                e = row_exponent(top);
            }
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    qf[n][c][j] = (_Float16)(DT == kBF16 ? ldexpf(v[8 * c + j], 14 - e) : v[8 * c + j]);
            f[n] = ldexpf(a.softcap > 0.0f ? 2.0f * kLog2e / a.softcap * a.scale : kLog2e * a.scale, e - 14);
            M[n] = kNone;
            l[n] = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t) o[n][t] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
        }
        // keys from lo_max to hi_min are seen by all of the tile's rows: the bounds grow with the position
        int lo_max, hi_min, unused;
        {
            const int rows = sg.un.s.q.n * group, r0 = sg.tile * R;
            row_keys(a, sg.un.s, sg.un.s.q.p0 + r0 / group, unused, hi_min);
            row_keys(a, sg.un.s, sg.un.s.q.p0 + (min(r0 + R, rows) - 1) / group, lo_max, unused);
            lo_max = __builtin_amdgcn_readfirstlane(lo_max);
            hi_min = __builtin_amdgcn_readfirstlane(hi_min);
        }
        const float cap2 = a.softcap * kLog2e;

        auto compute = [&](int t0, const Tile& x) {
            v4f z[2][NQ];
            float lv[2], rv[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int n = 0; n < NQ; ++n) z[u][n] = (v4f){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const uint4& w = x.k[u][c >> 1];
                    const v8h kf = (c & 1) ? join(codes4(w.z), codes4(w.w)) : join(codes4(w.x), codes4(w.y));
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        z[u][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[n][c], z[u][n], 0, 0, 0);
                }
                lv[u] = __log2f(x.vs[u]);
                rv[u] = __builtin_amdgcn_rcpf(x.vs[u]);
            }
            const bool masked = t0 < lo_max || t0 + 31 > hi_min || !x.there[0] || !x.there[1];
            v8h pf[NQ];
#pragma unroll
            for (int n = 0; n < NQ; ++n) {
                float e[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) e[u][r] = z[u][n][r] * (f[n] * x.ks[u]);
                if (a.softcap > 0.0f) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r) e[u][r] = capped(e[u][r], cap2);
                }
                if (a.slopes) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r) e[u][r] += slope[n] * (float)(t0 + 16 * u + 4 * g + r - pos[n]);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 4; ++r) e[u][r] += lv[u];
                if (masked) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int key = t0 + 16 * u + 4 * g + r;
                            e[u][r] = key >= lo[n] && key <= hi[n] && x.there[u] ? e[u][r] : -INFINITY;
                        }
                }
                float top = fmaxf(fmaxf(fmaxf(e[0][0], e[0][1]), fmaxf(e[0][2], e[0][3])),
                                  fmaxf(fmaxf(e[1][0], e[1][1]), fmaxf(e[1][2], e[1][3])));
                if (__any(top > M[n] + (kLift + kSlack))) {
                    top = fmaxf(top, __shfl_xor(top, 16));
                    top = fmaxf(top, __shfl_xor(top, 32));
                    if (top > M[n] + (kLift + kSlack)) {
                        const float now = ceilf(top) - kLift;
                        const float keep = exp2_(M[n] - now);
                        M[n] = now;
                        l[n] *= keep;
#pragma unroll
                        for (int t = 0; t < NT; ++t) o[n][t] *= keep;
                    }
                }
                float p[2][4];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) p[u][r] = exp2_(e[u][r] - M[n]);
                    const float sum = (p[u][0] + p[u][1]) + (p[u][2] + p[u][3]);
                    l[n] += sum == 0.0f ? 0.0f : sum * rv[u];  // hidden keys of a page whose scale is not finite: 0
                }
                const uint4 w = make_uint4(f32x2_to_16<kF16>(p[0][0], p[0][1]), f32x2_to_16<kF16>(p[0][2], p[0][3]),
                                           f32x2_to_16<kF16>(p[1][0], p[1][1]), f32x2_to_16<kF16>(p[1][2], p[1][3]));
                pf[n] = __builtin_bit_cast(v8h, w);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const uint32_t w0 = reinterpret_cast<const uint32_t*>(x.v[0])[t];
                const uint32_t w1 = reinterpret_cast<const uint32_t*>(x.v[1])[t];
                const v8h vf = join(codes4(w0), codes4(w1));
#pragma unroll
                for (int n = 0; n < NQ; ++n)
                    o[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[n], o[n][t], 0, 0, 0);
            }
        };

        if (sg.begin < sg.end) {
            for (int t0 = sg.begin;; t0 += 2 * kStep) {
                const bool more = t0 + kStep < sg.end;
                if (more) {
                    load(t0 + kStep, id, y);
                    pages(t0 + 2 * kStep, id);
                }
                compute(t0, x);
                if (!more) break;
                const bool even = t0 + 2 * kStep < sg.end;
                if (even) {
                    load(t0 + 2 * kStep, id, x);
                    pages(t0 + 3 * kStep, id);
                }
                compute(t0 + kStep, y);
                if (!even) break;
            }
        }

        // the next segment's loads run while this one is written out
        const int s = sg.s, hk = sg.hk, tile = sg.tile, step0 = sg.step0, steps = sg.steps;
        const int all_steps = sg.un.steps, n_rows = sg.un.s.q.n, q0 = sg.un.s.q.q0;
        const int64_t u = u0;
        u0 += steps;
        if (u0 < u1) {
            find(u0);
            ahead();
        }

        // join the four waves, 16 rows at a time
        const bool whole = steps == all_steps;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (first_segment ? 0 : 1);
        __syncthreads();
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            l[n] += __shfl_xor(l[n], 16);
            l[n] += __shfl_xor(l[n], 32);
            if (g == 0) {
                sM[wave][n * 16 + i] = M[n];
                sl[wave][n * 16 + i] = l[n];
            }
        }
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
            __syncthreads();
            const int row = n * 16 + i;
            const float top = fmaxf(fmaxf(sM[0][row], sM[1][row]), fmaxf(sM[2][row], sM[3][row]));
            const float keep = exp2_(M[n] - top);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int t = 0; t < NT; t += 4)
                    *reinterpret_cast<float4*>(&so[wave][i][(4 * g + r) * NT + t]) =
                        make_float4(o[n][t][r] * keep, o[n][t + 1][r] * keep, o[n][t + 2][r] * keep, o[n][t + 3][r] * keep);
            __syncthreads();
            for (int c = tid; c < 16 * (D / 8); c += 256) {
                const int j = c / (D / 8), d = c % (D / 8) * 8;
                const int rr = tile * R + n * 16 + j;
                const int tok = rr / group;
                if (tok < n_rows) {
                    const float Mj = fmaxf(fmaxf(sM[0][n * 16 + j], sM[1][n * 16 + j]),
                                           fmaxf(sM[2][n * 16 + j], sM[3][n * 16 + j]));
                    float lj = 0.0f, v[8] = {};
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        lj += sl[w][n * 16 + j] * exp2_(sM[w][n * 16 + j] - Mj);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] += so[w][j][d + k];
                    }
                    if (whole) {
                        write_row<DT, D>(a, q0 + tok, hk * group + rr - tok * group, d, v, Mj, lj);
                    } else {
                        float* p = slot_of<D, R>(a, slot);
                        float4* q = reinterpret_cast<float4*>(p + (n * 16 + j) * D + d);
                        q[0] = make_float4(v[0], v[1], v[2], v[3]);
                        q[1] = make_float4(v[4], v[5], v[6], v[7]);
                        if (d == 0) {
                            p[R * D + n * 16 + j] = Mj;
                            p[R * D + R + n * 16 + j] = lj;
                        }
                    }
                }
            }
        }
        if (step0 == 0 && tid == 0) {
            const int last = whole ? -1 : range_of<W>(total, u + all_steps - 1);
            *parts_of<D, R>(a, first_item<R>(a, s) + tile, hk) = make_int2((int)slot, last);
        }
        if (u0 >= u1) break;
        first_segment = false;
    }
}

// Joins the partial results of a segment that was cut: one workgroup for each
// (row tile of a sequence, head; row), D / 8 threads for each of 2048 / D parts
// at a time.  All latency: 4.7 us for 32 x 4096 and for 1 x 131071 keys, 6.4 for 24 x 6011 with 256 channels.
template <int DT, int D, int R>
__global__ __launch_bounds__(256) void k_attention_join(AttentionArgs a) {
    constexpr int NP = 2048 / D;  // parts taken at once
    __shared__ float sm[NP], sl[NP], so[NP][D];
    const int tid = threadIdx.x, group = a.hq / a.c.heads;
    const int64_t item = blockIdx.x / a.c.heads;
    const int hk = (int)(blockIdx.x - item * a.c.heads), j = blockIdx.y;
    const int2 parts = *parts_of<D, R>(a, item, hk);
    int s;
    int64_t tile;
    // an item that is no tile: nobody wrote its parts, and nothing that they say may be used
    if (!item_of(a.b, item, group, R, 1, s, tile)) return;
    const KvSeq q = kv_seq<true>(a.b, s);
    const int64_t rr = tile * R + j;
    if (rr >= (int64_t)q.n * group) return;
    const int w0 = parts.x >> 1, w1 = parts.y;
    if (w1 < 0) return;

    const int p = tid / (D / 8), d = tid % (D / 8) * 8;
    float M = kNone, l = 0.0f, o[8] = {};
#pragma unroll 4
    for (int w = w0 + p; w <= w1; w += NP) {
        const float* x = slot_of<D, R>(a, w == w0 ? parts.x : 2 * (int64_t)w);
        const float Mw = x[R * D + j], lw_ = x[R * D + R + j];
        const float4 v0 = *reinterpret_cast<const float4*>(x + j * D + d);
        const float4 v1 = *reinterpret_cast<const float4*>(x + j * D + d + 4);
        const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        const float now = fmaxf(M, Mw), fo = exp2_(M - now), fw = exp2_(Mw - now);
        M = now;
        l = l * fo + lw_ * fw;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = o[k] * fo + v[k] * fw;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) so[p][d + k] = o[k];
    if (d == 0) {
        sm[p] = M;
        sl[p] = l;
    }
    __syncthreads();
    if (p != 0) return;
    float top = sm[0];
    for (int w = 1; w < NP; ++w) top = fmaxf(top, sm[w]);
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) o[k] = 0.0f;
#pragma unroll 2
    for (int w = 0; w < NP; ++w) {
        const float keep = exp2_(sm[w] - top);
        l += sl[w] * keep;
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] += so[w][d + k] * keep;
    }
    const int64_t tok = rr / group;
    write_row<DT, D>(a, q.q0 + tok, hk * group + (int)(rr - tok * group), d, o, top, l);
}

// 16-row tiles of the few-row kernel for a batch: enough for the rows that a
// sequence has on average; 0: the prompt kernel.  8 sequences of 4000 keys, this kernel
// against the prompt kernel, us (8 key/value heads; with 256 channels 8 and 2):
//   rows    64 channels   128 channels   256, 8 heads   256, 2 heads
//   24      25 / 25       29 / 34        54 / 62        30 / 47
//   32      28 / 26       31 / 34        56 / 62        32 / 48
//   48      35 / 29       40 / 36        82 / 65        36 / 51
//   64      37 / 30       42 / 37        84 / 68        37 / 54
// With 256 channels the limit of 64 is that of few heads and sequences; with many, 32 would be the better one.
int row_tiles(int64_t tokens, int64_t batch, int hq, int hkv, int dim) {
    const int64_t rows = (tokens * (hq / hkv) + batch - 1) / batch;
    return rows <= 16 ? 1 : rows <= (dim == 256 ? 64 : 32) ? 2 : 0;
}

int64_t few_items(int64_t tokens, int64_t batch, int group, int R, bool ragged) {
    return ragged ? tokens * group / R + batch : batch * ((group + R - 1) / R);
}

int64_t few_items(const AttentionArgs& a, int R) {
    return few_items(a.b.tokens, a.b.batch, a.hq / a.c.heads, R, a.b.cu_q);
}

int prompt_splits(const AttentionArgs& a) {
    return attention_prompt_splits(a.b.tokens, a.b.batch, a.hq, a.c.heads, a.c.dim, (int64_t)a.b.max_pages * a.c.page);
}

template <int DT, int D, int NQ>
void launch_few(const AttentionArgs& a, hipStream_t st) {
    constexpr int R = 16 * NQ;
    const int group = a.hq / a.c.heads;
    k_attention_few<DT, D, NQ><<<ways(D, R), 256, 0, st>>>(a);
    if ((int64_t)a.b.max_pages * a.c.page > kStep)  // else no segment has a second step to be cut at
        k_attention_join<DT, D, R><<<dim3((uint32_t)(few_items(a, R) * a.c.heads), a.b.cu_q ? R : std::min(R, group)),
                                     256, 0, st>>>(a);
}

template <int DT, int D>
void launch(const AttentionArgs& a, int tiles, hipStream_t st) {
    if (tiles == 1) launch_few<DT, D, 1>(a, st);
    else launch_few<DT, D, 2>(a, st);
}

}  // namespace

size_t attention_workspace(int64_t tokens, int64_t batch, int hq, int hkv, int dim) {
    const int tiles = row_tiles(tokens, batch, hq, hkv, dim);
    if (tiles > 0) {
        const int group = hq / hkv, R = 16 * tiles;
        const int64_t items = std::max(few_items(tokens, batch, group, R, true), few_items(tokens, batch, group, R, false));
        return (size_t)2 * ways(dim, R) * R * (dim + 2) * sizeof(float) + items * hkv * sizeof(int2);
    }
    const int splits = attention_prompt_most_splits(tokens, batch, hq, hkv, dim);
    return splits > 1 ? (size_t)splits * tokens * hq * (dim + 2) * sizeof(float) : 0;
}

int64_t attention_threads(const AttentionArgs& a) {
    if (a.b.batch == 0) return 0;
    const int tiles = row_tiles(a.b.tokens, a.b.batch, a.hq, a.c.heads, a.c.dim);
    if (tiles == 0) return attention_prompt_threads(a, prompt_splits(a));
    const int R = 16 * tiles;
    return few_items(a, R) * a.c.heads * (a.b.cu_q ? R : std::min(R, a.hq / a.c.heads)) * 256;
}

void launch_attention(const AttentionArgs& a, int dt, hipStream_t st) {
    const int tiles = row_tiles(a.b.tokens, a.b.batch, a.hq, a.c.heads, a.c.dim);
    if (tiles == 0) {
        launch_attention_prompt(a, dt, prompt_splits(a), st);
    } else if (dt == kBF16) {
        if (a.c.dim == 64) launch<kBF16, 64>(a, tiles, st);
        else if (a.c.dim == 128) launch<kBF16, 128>(a, tiles, st);
        else launch<kBF16, 256>(a, tiles, st);
    } else {
        if (a.c.dim == 64) launch<kF16, 64>(a, tiles, st);
        else if (a.c.dim == 128) launch<kF16, 128>(a, tiles, st);
        else launch<kF16, 256>(a, tiles, st);
    }
}

}  // namespace pdq

// Appending to the paged INT8 key/value cache: position rotation, codes, page
// scales.  include/pdq.h (pdq_kv_append) states the arithmetic.
#include "kv_device.h"

namespace pdq {

namespace {

constexpr float kMinScale = 0x1p-64f;

// A head's row is taken in pairs of 8-channel chunks, dim / 16 of them: the e-th
// is chunks (e, e + rot / 16), whose channels are partners, or with neighbours as
// partners, and behind the rotated channels, chunks (2 e, 2 e + 1).  Either way
// its channels turn by the tables' columns 8 e .. 8 e + 7.
struct Pair {
    int c0, c1;
    bool turned;
};
__device__ __forceinline__ Pair pair_of(const KvAppendArgs& a, int e) {
    const int half = a.rot / 16;  // pairs that are rotated
    const bool turned = a.cos && e < half, halves = turned && !a.interleaved;
    return Pair{halves ? e : 2 * e, halves ? e + half : 2 * e + 1, turned};
}

// The tables' columns of pair e at position pos; a position outside them: NaN.
struct Turn {
    float c[8], s[8];
};
__device__ __forceinline__ Turn turn_of(const KvAppendArgs& a, int e, int pos) {
    Turn t;
    const bool known = (uint32_t)pos < (uint32_t)a.positions;
    const int64_t at = (int64_t)(known ? pos : 0) * (a.rot / 2) + 8 * e;
    const float4* c = reinterpret_cast<const float4*>(a.cos + at);
    const float4* s = reinterpret_cast<const float4*>(a.sin + at);
    const float4 c0 = c[0], c1 = c[1], s0 = s[0], s1 = s[1];
    const float co[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float si[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        t.c[j] = known ? co[j] : __builtin_nanf("");
        t.s[j] = known ? si[j] : __builtin_nanf("");
    }
    return t;
}

// A pair's 16 channels rotated.  The products and the sum are rounded one by one
// (the library is compiled without contraction), so the values are those of the
// same formula in any binary32 arithmetic.
__device__ __forceinline__ void rotate(const Turn& t, bool interleaved, float (&x)[8], float (&y)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float& u = interleaved ? (j < 4 ? x[2 * (j & 3)] : y[2 * (j & 3)]) : x[j];
        float& w = interleaved ? (j < 4 ? x[2 * (j & 3) + 1] : y[2 * (j & 3) + 1]) : y[j];
        const float p = u, q = w;
        u = p * t.c[j] - q * t.s[j];
        w = q * t.c[j] + p * t.s[j];
    }
}

// |x| of 8 values as integers: their order is the values' order, infinities
// above every finite value and NaN above infinity.
__device__ __forceinline__ uint32_t top8(const float (&x)[8], uint32_t m) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[j]) & 0x7fffffffu);
    return m;
}

__device__ __forceinline__ void codes8(const float (&x)[8], float s, float inv, int (&q)[8]) {
    float r[8];
    rne_quotient8<true>(x, s, inv, r);
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = (int)fminf(fmaxf(r[j], -127.0f), 127.0f);
}

__device__ __forceinline__ int moved(int code, float ratio) { return (int)__builtin_rintf((float)code * ratio); }

__device__ __forceinline__ uint32_t moved4(uint32_t w, float ratio) {
    return pack4_i8(moved((int8_t)w, ratio), moved((int8_t)(w >> 8), ratio), moved((int8_t)(w >> 16), ratio),
                    moved((int8_t)(w >> 24), ratio));
}

__device__ __forceinline__ uint2 pack_codes8(const float (&x)[8], float s, float inv, bool finite) {
    int r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (finite) codes8(x, s, inv, r);
    return make_uint2(pack4_i8(r[0], r[1], r[2], r[3]), pack4_i8(r[4], r[5], r[6], r[7]));
}

template <int DT>
__device__ __forceinline__ uint4 round8(const float (&x)[8]) {
    return make_uint4(f32x2_to_16<DT>(x[0], x[1]), f32x2_to_16<DT>(x[2], x[3]), f32x2_to_16<DT>(x[4], x[5]),
                      f32x2_to_16<DT>(x[6], x[7]));
}

constexpr int kHeads = 4;  // query heads of a thread

// The rotated queries of row t, by one wavefront: a thread takes one pair of
// chunks in up to kHeads heads, so that the tables' 64 bytes are read for 128
// bytes of queries.
template <int DT>
__device__ __forceinline__ void rotate_queries(const KvAppendArgs& a, int64_t t) {
    const int lane = threadIdx.x & 63, pairs = a.c.dim / 16;
    if (t >= a.b.tokens) return;
    int s = (int)t;
    if (a.b.cu_q) {
        if (t < uniform_load(a.b.cu_q) || t >= uniform_load(a.b.cu_q + a.b.batch)) return;  // rows of no sequence stay
        s = row_seq(a.b, (int)t);
    }
    const KvSeq q = kv_seq<true>(a.b, s);
    const int pos = q.p0 + (int)t - q.q0;
    const uint16_t* const src = reinterpret_cast<const uint16_t*>(a.q) + t * a.ldq;
    uint16_t* const dst = reinterpret_cast<uint16_t*>(a.q_out) + t * a.ldqo;
    const int per = min(kHeads, max(1, a.hq * pairs / 64));  // heads of a thread
    const int apart = (a.hq + per - 1) / per;
    for (int u = lane; u < apart * pairs; u += 64) {
        const int h = u / pairs, e = u - h * pairs;
        const Pair p = pair_of(a, e);
        Raw8<DT> r0[kHeads], r1[kHeads];
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
            if (k < per && h + k * apart < a.hq) {
                const uint16_t* row = src + (int64_t)(h + k * apart) * a.c.dim;
                r0[k] = load_raw8<DT>(row, p.c0);
                r1[k] = load_raw8<DT>(row, p.c1);
            }
        Turn turn;
        if (p.turned) turn = turn_of(a, e, pos);
#pragma unroll
        for (int k = 0; k < kHeads; ++k)
            if (k < per && h + k * apart < a.hq) {
                float x[8], y[8];
                widen8<DT>(r0[k], x);
                widen8<DT>(r1[k], y);
                if (p.turned) {
                    if (a.interleaved) rotate(turn, true, x, y);
                    else rotate(turn, false, x, y);
                }
                uint4* row = reinterpret_cast<uint4*>(dst + (int64_t)(h + k * apart) * a.c.dim);
                row[p.c0] = round8<DT>(x);
                row[p.c1] = round8<DT>(y);
            }
    }
}

// One workgroup of NT threads for each (touched page, head, keys or values);
// after those, wavefronts that rotate the queries.  Bound by its bytes: seven
// prompts of together 8900 tokens (203 MB, 32 + 8 + 8 heads of 128 channels) 43 us,
// 4.7 TB/s, a large copy's 4.95; one token of one user 4.5 us, all latency, 128 users 6.
// A page's workgroup needs the
// largest magnitude of its new tokens before the first code: what a thread takes
// first of them (up to kKeep pairs of chunks, or quads of tokens) stays in its
// registers, all of a page of 64 tokens x 128 channels; the rest of a larger page
// is read again, from the cache.
template <int DT, int NT>
__global__ __launch_bounds__(NT) void k_kv_append(KvAppendArgs a, int64_t kv_blocks) {
    constexpr int kKeep = 2;
    const int tid = threadIdx.x;
    if (blockIdx.x >= kv_blocks) {
        const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
        rotate_queries<DT>(a, ((int64_t)blockIdx.x - kv_blocks) * (NT / 64) + wave);
        return;
    }
    const bool values = blockIdx.x & 1;
    const int64_t rest = blockIdx.x >> 1;
    const int64_t item = rest / a.c.heads;
    const int h = (int)(rest - item * a.c.heads);
    const int page = a.c.page;
    int s;
    int64_t j;
    if (!item_of(a.b, item, 1, page, 2, s, j)) return;
    const KvSeq q = kv_seq<true>(a.b, s);
    if (q.n == 0) return;
    // the j-th page that the new tokens touch; tokens at negative positions are not written
    const int64_t jj = (int64_t)max(q.p0, 0) / page + j;
    if (jj * page >= q.len || jj >= a.b.max_pages) return;
    const int first = (int)jj * page;
    const int id = uniform_load(a.b.page_table + (int64_t)s * a.b.ldt + jj);
    if ((uint32_t)id >= (uint32_t)a.c.pages) return;
    const int lo = max(q.p0 - first, 0), hi = min(q.len - first, page);  // slots of the new tokens
    const int64_t row0 = (int64_t)q.q0 + first - q.p0;                   // row of slot 0
    const int64_t at = (int64_t)id * a.c.heads + h;
    float* const scale = (values ? a.c.v_scale : a.c.k_scale) + at;
    int8_t* const codes = (values ? a.c.v : a.c.k) + at * page * a.c.dim;
    const int64_t ld = values ? a.ldv : a.ldk;
    const uint16_t* const src = reinterpret_cast<const uint16_t*>(values ? a.v : a.k) + (int64_t)h * a.c.dim;
    const float held = lo > 0 ? *scale : 0.0f;
    const int dc = a.c.dim / 8, pairs = a.c.dim / 16;

    // keys: pair u % pairs of slot lo + u / pairs
    const int key_units = values ? 0 : (hi - lo) * pairs;
    auto key_pair = [&](int u, float (&x)[8], float (&y)[8]) {
        const int slot = lo + u / pairs, e = u % pairs;
        const Pair p = pair_of(a, e);
        const uint16_t* row = src + (row0 + slot) * ld;
        const Raw8<DT> r0 = load_raw8<DT>(row, p.c0), r1 = load_raw8<DT>(row, p.c1);
        if (p.turned) {
            const Turn t = turn_of(a, e, first + slot);
            widen8<DT>(r0, x);
            widen8<DT>(r1, y);
            if (a.interleaved) rotate(t, true, x, y);
            else rotate(t, false, x, y);
        } else {
            widen8<DT>(r0, x);
            widen8<DT>(r1, y);
        }
    };
    // values: chunk u % dc of the four slots from 4 (quad0 + u / dc)
    const int quad0 = lo >> 2;
    const int value_units = values ? (((hi + 3) >> 2) - quad0) * dc : 0;
    auto quad = [&](int u, Raw8<DT> (&r)[4]) {
        const int slot = 4 * (quad0 + u / dc), c = u % dc;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r[i] = slot + i >= lo && slot + i < hi ? load_raw8<DT>(src + (row0 + slot + i) * ld, c) : zero_raw8<DT>();
    };

    uint32_t top = 0;
    float kx[kKeep][8], ky[kKeep][8];
    Raw8<DT> vr[kKeep][4];
    if (!values) {
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (tid + k * NT < key_units) {
                key_pair(tid + k * NT, kx[k], ky[k]);
                top = top8(ky[k], top8(kx[k], top));
            }
        for (int u = tid + kKeep * NT; u < key_units; u += NT) {
            float x[8], y[8];
            key_pair(u, x, y);
            top = top8(y, top8(x, top));
        }
    } else {
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (tid + k * NT < value_units) quad(tid + k * NT, vr[k]);
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (tid + k * NT < value_units) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[8];
                    widen8<DT>(vr[k][i], x);
                    top = top8(x, top);
                }
            }
        for (int u = tid + kKeep * NT; u < value_units; u += NT) {
            Raw8<DT> r[4];
            quad(u, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float x[8];
                widen8<DT>(r[i], x);
                top = top8(x, top);
            }
        }
    }
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, m));
    if constexpr (NT > 64) {
        __shared__ uint32_t part[NT / 64];
        if ((tid & 63) == 0) part[tid >> 6] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NT / 64; ++i) top = max(top, part[i]);
    }
    const bool finite = top < 0x7f800000u && fabsf(held) < INFINITY;
    const float need = fmaxf(__uint_as_float(top) * (1.0f / 127.0f), kMinScale);
    const float now = finite ? fmaxf(held, need) : __builtin_nanf("");
    const float inv = 1.0f / now;
    const bool move = lo > 0 && finite && now > held;
    const float ratio = held / now;
    if (tid == 0 && !(lo > 0 && now == held)) *scale = now;

    if (!values) {
        auto put = [&](int u, const float (&x)[8], const float (&y)[8]) {
            const int slot = lo + u / pairs;
            const Pair p = pair_of(a, u % pairs);
            uint2* row = reinterpret_cast<uint2*>(codes + (int64_t)slot * a.c.dim);
            row[p.c0] = pack_codes8(x, now, inv, finite);
            row[p.c1] = pack_codes8(y, now, inv, finite);
        };
#pragma unroll
        for (int k = 0; k < kKeep; ++k)
            if (tid + k * NT < key_units) put(tid + k * NT, kx[k], ky[k]);
        for (int u = tid + kKeep * NT; u < key_units; u += NT) {
            float x[8], y[8];
            key_pair(u, x, y);
            put(u, x, y);
        }
        if (move) {
            for (int u = tid; u < lo * dc; u += NT) {
                uint2* p = reinterpret_cast<uint2*>(codes) + u;
                *p = make_uint2(moved4(p->x, ratio), moved4(p->y, ratio));
            }
        }
        return;
    }
    // quads of four slots, of which the first may hold older tokens and the last tokens to come
    auto put = [&](int u, const Raw8<DT> (&r)[4]) {
        const int slot = 4 * (quad0 + u / dc), c = u % dc;
        uint4* p = reinterpret_cast<uint4*>(codes + ((int64_t)slot * a.c.dim + 32 * c));
        const bool whole = slot >= lo && slot + 4 <= hi;
        uint2 q8[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x[8];
            widen8<DT>(r[i], x);
            q8[i] = pack_codes8(x, now, inv, finite);
        }
        uint32_t w[8];
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            const int b = 8 * (d & 3);
            const uint32_t c0 = d < 4 ? q8[0].x : q8[0].y, c1 = d < 4 ? q8[1].x : q8[1].y;
            const uint32_t c2 = d < 4 ? q8[2].x : q8[2].y, c3 = d < 4 ? q8[3].x : q8[3].y;
            w[d] = (c0 >> b & 0xff) | (c1 >> b & 0xff) << 8 | (c2 >> b & 0xff) << 16 | (c3 >> b) << 24;
        }
        if (!whole) {
            const uint4 o0 = p[0], o1 = p[1];
            const uint32_t o[8] = {o0.x, o0.y, o0.z, o0.w, o1.x, o1.y, o1.z, o1.w};
            uint32_t fresh = 0, older = 0;  // bytes of new tokens, of older ones
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (slot + i >= lo && slot + i < hi) fresh |= 0xffu << (8 * i);
                if (slot + i < lo) older |= 0xffu << (8 * i);
            }
            if (!move) older = 0;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                const uint32_t m = older ? (moved4(o[d], ratio) & older) | (o[d] & ~older) : o[d];
                w[d] = (w[d] & fresh) | (m & ~fresh);
            }
        }
        p[0] = make_uint4(w[0], w[1], w[2], w[3]);
        p[1] = make_uint4(w[4], w[5], w[6], w[7]);
    };
#pragma unroll
    for (int k = 0; k < kKeep; ++k)
        if (tid + k * NT < value_units) put(tid + k * NT, vr[k]);
    for (int u = tid + kKeep * NT; u < value_units; u += NT) {
        Raw8<DT> r[4];
        quad(u, r);
        put(u, r);
    }
    if (move) {  // the quads before them
        for (int u = tid; u < quad0 * dc; u += NT) {
            uint4* p = reinterpret_cast<uint4*>(codes) + 2 * u;
            const uint4 o0 = p[0], o1 = p[1];
            p[0] = make_uint4(moved4(o0.x, ratio), moved4(o0.y, ratio), moved4(o0.z, ratio), moved4(o0.w, ratio));
            p[1] = make_uint4(moved4(o1.x, ratio), moved4(o1.y, ratio), moved4(o1.z, ratio), moved4(o1.w, ratio));
        }
    }
}

// A wavefront for a page with one new token, four for the many of a prompt (128
// single tokens 6.1 us against 8.9 with four; prompts of 8900 tokens 39.0 against 41.0
// with one, replayed on the same data).
int threads(const KvAppendArgs& a) { return a.b.cu_q ? 256 : 64; }

int64_t kv_blocks(const KvAppendArgs& a) {
    const int64_t items = a.b.cu_q ? (int64_t)a.b.tokens / a.c.page + 2 * (int64_t)a.b.batch : a.b.batch;
    return items * a.c.heads * 2;
}

int64_t q_blocks(const KvAppendArgs& a) {
    const int waves = threads(a) / 64;  // a row each
    return a.q ? ((int64_t)a.b.tokens + waves - 1) / waves : 0;
}

}  // namespace

int64_t kv_append_threads(const KvAppendArgs& a) { return (kv_blocks(a) + q_blocks(a)) * threads(a); }

void launch_kv_append(const KvAppendArgs& a, int dt, hipStream_t st) {
    const int64_t kv = kv_blocks(a);
    const dim3 grid((uint32_t)(kv + q_blocks(a)));
    if (a.b.cu_q) {
        if (dt == kBF16) k_kv_append<kBF16, 256><<<grid, 256, 0, st>>>(a, kv);
        else k_kv_append<kF16, 256><<<grid, 256, 0, st>>>(a, kv);
    } else {
        if (dt == kBF16) k_kv_append<kBF16, 64><<<grid, 64, 0, st>>>(a, kv);
        else k_kv_append<kF16, 64><<<grid, 64, 0, st>>>(a, kv);
    }
}

}  // namespace pdq

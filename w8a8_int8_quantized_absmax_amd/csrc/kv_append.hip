// Appending to the paged INT8 key/value cache: position rotation, codes, page
// scales.  include/pdq.h (pdq_kv_append) states the arithmetic.
#include "kv_device.h"

namespace pdq {

namespace {

constexpr float kMinScale = 0x1p-64f;

// 8 channels [8 c, 8 c + 8) of one head's row at `row`, rotated by the tables'
// row `pos` (outside the tables: NaN).  The products and the sum are rounded
// one by one (the library is compiled without contraction), so the values are
// those of the same formula in any binary32 arithmetic.
template <int DT>
__device__ __forceinline__ void load_rotated(const KvAppendArgs& a, const uint16_t* row, int c, int pos,
                                             float (&x)[8]) {
    widen8<DT>(load_raw8<DT>(row, c), x);
    if (!a.cos || 8 * c >= a.rot) return;
    const int half = a.rot / 2;
    const bool known = (uint32_t)pos < (uint32_t)a.positions;
    const int64_t at = (int64_t)(known ? pos : 0) * half;
    const float nan = __builtin_nanf("");
    if (a.interleaved) {
        const float4 cs = *reinterpret_cast<const float4*>(a.cos + at + 4 * c);
        const float4 sn = *reinterpret_cast<const float4*>(a.sin + at + 4 * c);
        const float co[4] = {cs.x, cs.y, cs.z, cs.w}, si[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = x[2 * j], w = x[2 * j + 1];
            x[2 * j] = known ? u * co[j] - w * si[j] : nan;
            x[2 * j + 1] = known ? w * co[j] + u * si[j] : nan;
        }
        return;
    }
    const int hc = half / 8;           // 8-channel chunks of a half
    const bool second = c >= hc;       // the partner of the second half's channel j is j - half
    const int f = second ? c - hc : c;
    float o[8];
    widen8<DT>(load_raw8<DT>(row, second ? f : c + hc), o);
    const float4* cs = reinterpret_cast<const float4*>(a.cos + at + 8 * f);
    const float4* sn = reinterpret_cast<const float4*>(a.sin + at + 8 * f);
    const float4 c0 = cs[0], c1 = cs[1], s0 = sn[0], s1 = sn[1];
    const float co[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float si[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float p = x[j] * co[j], r = o[j] * si[j];
        x[j] = known ? (second ? p + r : p - r) : nan;
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

// One workgroup of NT threads for each (touched page, head, keys or values);
// after those, workgroups that rotate the queries.  A page's workgroup goes over
// its new tokens twice, once for the largest magnitude, once for the codes.
template <int DT, int NT>
__global__ __launch_bounds__(NT) void k_kv_append(KvAppendArgs a, int64_t kv_blocks) {
    const int tid = threadIdx.x;
    const int dc = a.c.dim / 8;  // 8-channel chunks of a head
    if (blockIdx.x >= kv_blocks) {
        const int64_t u = ((int64_t)blockIdx.x - kv_blocks) * NT + tid;
        const int64_t row = u / dc;
        const int c = (int)(u - row * dc);
        const int64_t t = row / a.hq;
        if (t >= a.b.tokens) return;
        const int h = (int)(row - t * a.hq);
        if (a.b.cu_q && (t < a.b.cu_q[0] || t >= a.b.cu_q[a.b.batch])) return;  // rows of no sequence stay
        const int s = row_seq(a.b, (int)t);
        const KvSeq q = kv_seq(a.b, s);
        float x[8];
        load_rotated<DT>(a, reinterpret_cast<const uint16_t*>(a.q) + t * a.ldq + (int64_t)h * a.c.dim, c,
                         q.p0 + (int)t - q.q0, x);
        uint4 o;
        o.x = f32x2_to_16<DT>(x[0], x[1]);
        o.y = f32x2_to_16<DT>(x[2], x[3]);
        o.z = f32x2_to_16<DT>(x[4], x[5]);
        o.w = f32x2_to_16<DT>(x[6], x[7]);
        reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.q_out) + t * a.ldqo + (int64_t)h * a.c.dim)[c] = o;
        return;
    }
    const bool values = blockIdx.x & 1;
    const int64_t rest = blockIdx.x >> 1;
    const int64_t item = rest / a.c.heads;
    const int h = (int)(rest - item * a.c.heads);
    const int page = a.c.page;
    int s, j;
    if (a.b.cu_q) {
        s = item_seq(a.b, item, 1, page, 2);
        j = (int)min(item - item_start(a.b, s, 1, page, 2), (int64_t)1 << 30);
    } else {
        s = (int)item;
        j = 0;
    }
    const KvSeq q = kv_seq(a.b, s);
    if (q.n == 0) return;
    // the j-th page that the new tokens touch; tokens at negative positions are not written
    const int64_t jj = (int64_t)max(q.p0, 0) / page + j;
    if (jj * page >= q.len || jj >= a.b.max_pages) return;
    const int first = (int)jj * page;
    const int id = kv_page(a.c, a.b, s, (int)jj);
    if (id < 0) return;
    const int lo = max(q.p0 - first, 0), hi = min(q.len - first, page);  // slots of the new tokens
    const int64_t pos0 = first, row0 = (int64_t)q.q0 + first - q.p0;     // position and row of slot 0
    const int64_t at = (int64_t)id * a.c.heads + h;
    float* const scale = (values ? a.c.v_scale : a.c.k_scale) + at;
    int8_t* const codes = (values ? a.c.v : a.c.k) + at * page * a.c.dim;
    const int64_t ld = values ? a.ldv : a.ldk;
    const uint16_t* const src = reinterpret_cast<const uint16_t*>(values ? a.v : a.k) + (int64_t)h * a.c.dim;
    const float held = lo > 0 ? *scale : 0.0f;

    uint32_t top = 0;
    for (int u = tid; u < (hi - lo) * dc; u += NT) {
        const int slot = lo + u / dc, c = u % dc;
        const uint16_t* row = src + (row0 + slot) * ld;
        float x[8];
        if (values) widen8<DT>(load_raw8<DT>(row, c), x);
        else load_rotated<DT>(a, row, c, (int)pos0 + slot, x);
        top = top8(x, top);
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
    const bool finite = top < 0x7f800000u && held == held;
    const float need = fmaxf(__uint_as_float(top) * (1.0f / 127.0f), kMinScale);
    const float now = finite ? fmaxf(held, need) : __builtin_nanf("");
    const float inv = 1.0f / now;
    const bool move = lo > 0 && finite && now > held;
    const float ratio = held / now;
    if (tid == 0 && !(lo > 0 && now == held)) *scale = now;

    if (!values) {
        for (int u = tid; u < (hi - lo) * dc; u += NT) {
            const int slot = lo + u / dc, c = u % dc;
            float x[8];
            load_rotated<DT>(a, src + (row0 + slot) * ld, c, (int)pos0 + slot, x);
            int r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (finite) codes8(x, now, inv, r);
            *reinterpret_cast<uint2*>(codes + (int64_t)slot * a.c.dim + 8 * c) =
                make_uint2(pack4_i8(r[0], r[1], r[2], r[3]), pack4_i8(r[4], r[5], r[6], r[7]));
        }
        if (move) {
            for (int u = tid; u < lo * dc; u += NT) {
                uint2* p = reinterpret_cast<uint2*>(codes) + u;
                *p = make_uint2(moved4(p->x, ratio), moved4(p->y, ratio));
            }
        }
        return;
    }
    // values: quads of four slots, of which the first may hold older tokens and the last tokens to come
    const int quad0 = move ? 0 : lo >> 2, quads = ((hi + 3) >> 2) - quad0;
    for (int u = tid; u < quads * dc; u += NT) {
        const int quad = quad0 + u / dc, c = u % dc;
        uint32_t* p = reinterpret_cast<uint32_t*>(codes + ((int64_t)quad * a.c.dim + 8 * c) * 4);
        uint32_t w[8];
        const bool whole = 4 * quad >= lo && 4 * quad + 4 <= hi;
        if (!whole) {
#pragma unroll
            for (int d = 0; d < 8; ++d) w[d] = p[d];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int slot = 4 * quad + i;
            const uint32_t keep = ~(0xffu << (8 * i));
            if (slot >= lo && slot < hi) {
                float x[8];
                widen8<DT>(load_raw8<DT>(src + (row0 + slot) * ld, c), x);
                int r[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (finite) codes8(x, now, inv, r);
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    const uint32_t b = (uint32_t)(r[d] & 0xff) << (8 * i);
                    w[d] = whole && i == 0 ? b : (w[d] & keep) | b;
                }
            } else if (slot < lo && move) {
#pragma unroll
                for (int d = 0; d < 8; ++d)
                    w[d] = (w[d] & keep) | (uint32_t)(moved((int8_t)(w[d] >> (8 * i)), ratio) & 0xff) << (8 * i);
            }
        }
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

int threads(const KvAppendArgs& a) { return a.b.cu_q ? 256 : 64; }

int64_t kv_blocks(const KvAppendArgs& a) {
    const int64_t items = a.b.cu_q ? (int64_t)a.b.tokens / a.c.page + 2 * (int64_t)a.b.batch : a.b.batch;
    return items * a.c.heads * 2;
}

int64_t q_blocks(const KvAppendArgs& a) {
    const int nt = threads(a);
    return a.q ? ((int64_t)a.b.tokens * a.hq * (a.c.dim / 8) + nt - 1) / nt : 0;
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

// Attention over the paged INT8 key/value cache.  include/pdq.h
// (pdq_kv_attention) states the arithmetic.
#include "kv_device.h"

namespace pdq {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// One workgroup of four waves for each (row, query head): a wave takes groups of
// 16 tokens in turn with its own running maximum and sum, and the four are
// joined at the end.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_attention_rows(AttentionArgs a) {
    constexpr int DL = D / 4;   // channels of a lane in the score product
    constexpr int DV = D / 64;  // channels of a lane in the value product
    __shared__ float sm[4], sl[4], so[4][D];
    const int t = blockIdx.x / a.hq, h = blockIdx.x % a.hq;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15, g = lane >> 4;
    if (a.b.cu_q && (t < a.b.cu_q[0] || t >= a.b.cu_q[a.b.batch])) return;
    const int s = row_seq(a.b, t);
    const KvSeq q = kv_seq(a.b, s);
    const int hk = h / (a.hq / a.c.heads);
    const int pos = q.p0 + t - q.q0;
    const int last = min(min(a.prefix ? max(pos, a.prefix[s] - 1) : pos, q.len - 1), a.b.max_pages * a.c.page - 1);
    const int first = a.window ? max(pos - a.window + 1, 0) : 0;
    float x[DL], o[DV] = {}, m = -INFINITY, l = 0.0f;
    {
        const uint16_t* row = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)t * a.ldq + (int64_t)h * D + g * DL;
#pragma unroll
        for (int c = 0; c < DL / 8; ++c) {
            float v[8];
            widen8<DT>(load_raw8<DT>(row, c), v);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[8 * c + j] = v[j];
        }
    }
    for (int t0 = (first & ~15) + 16 * wave; t0 <= last; t0 += 64) {
        const int id = kv_page(a.c, a.b, s, t0 / a.c.page);
        if (id < 0) continue;
        const int64_t at = (int64_t)id * a.c.heads + hk;
        const int slot = t0 & (a.c.page - 1);
        const int8_t* k = a.c.k + (at * a.c.page + slot + i) * D + g * DL;
        float dot = 0.0f;
#pragma unroll
        for (int d = 0; d < DL; ++d) dot += x[d] * (float)k[d];
        dot += __shfl_xor(dot, 16);
        dot += __shfl_xor(dot, 32);
        float z = dot * (a.scale * a.c.k_scale[at]);
        if (a.softcap > 0.0f) z = a.softcap * tanhf(z / a.softcap);
        const int key = t0 + i;
        if (a.slopes) z += a.slopes[h] * (float)(key - pos);
        if (key < first || key > last) z = -INFINITY;
        float top = z;
#pragma unroll
        for (int w = 8; w >= 1; w >>= 1) top = fmaxf(top, __shfl_xor(top, w));
        const float mn = fmaxf(m, top);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float keep = exp2f((m - base) * kLog2e);
        const float p = exp2f((z - base) * kLog2e);
        l *= keep;
#pragma unroll
        for (int d = 0; d < DV; ++d) o[d] *= keep;
        m = mn;
        const float sv = a.c.v_scale[at];
        const int8_t* v = a.c.v + at * a.c.page * D + (int64_t)slot * D;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float pj = __shfl(p, j);
            l += pj;
            if (pj != 0.0f) {
#pragma unroll
                for (int d = 0; d < DV; ++d)
                    o[d] += pj * (sv * (float)v[((int64_t)(j >> 2) * D + lane * DV + d) * 4 + (j & 3)]);
            }
        }
    }
    if (lane == 0) {
        sm[wave] = m;
        sl[wave] = l;
    }
#pragma unroll
    for (int d = 0; d < DV; ++d) so[wave][lane * DV + d] = o[d];
    __syncthreads();
    const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const float base = top == -INFINITY ? 0.0f : top;
    float f[4], total = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        f[w] = exp2f((sm[w] - base) * kLog2e);
        total += sl[w] * f[w];
    }
    for (int d = threadIdx.x; d < D; d += 256) {
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) y += so[w][d] * f[w];
        y = total == 0.0f ? 0.0f : y / total;
        reinterpret_cast<uint16_t*>(a.y)[(int64_t)t * a.ldy + (int64_t)h * D + d] =
            DT == kBF16 ? f32_to_bf16(y) : f32_to_f16(y);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(int64_t)t * a.hq + h] = total == 0.0f ? -INFINITY : base + log2f(total) * kLn2;
}

template <int DT>
void launch(const AttentionArgs& a, hipStream_t st) {
    const dim3 grid((uint32_t)((int64_t)a.b.tokens * a.hq));
    if (a.c.dim == 64) k_attention_rows<DT, 64><<<grid, 256, 0, st>>>(a);
    else if (a.c.dim == 128) k_attention_rows<DT, 128><<<grid, 256, 0, st>>>(a);
    else k_attention_rows<DT, 256><<<grid, 256, 0, st>>>(a);
}

}  // namespace

size_t attention_workspace(int64_t tokens, int64_t batch, int hq, int hkv, int dim) { return 0; }

int64_t attention_threads(const AttentionArgs& a) { return (int64_t)a.b.tokens * a.hq * 256; }

void launch_attention(const AttentionArgs& a, int dt, hipStream_t st) {
    if (dt == kBF16) launch<kBF16>(a, st);
    else launch<kF16>(a, st);
}

}  // namespace pdq

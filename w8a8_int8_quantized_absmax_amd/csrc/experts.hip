// The experts' layer on 8-bit floating-point weights (gfx950): for each sorted
// row (a token at one of its experts) h = silu(Gate x) * (Up x), coded in groups of
// 128 as x is, then Down h times the row's weight, and a token's rows summed in the
// order of its slots.

#include "fp8_device.h"

namespace pdq {

namespace {

constexpr int kDirect = 8, kDirectValues = 32768;  // rows; values that a workgroup codes

template <bool F32S>
struct BlockScale {
    float f;
    uint32_t b;
};

template <bool F32S>
__device__ __forceinline__ BlockScale<F32S> block_scale(const void* s, int64_t at) {
    BlockScale<F32S> r{};
    if constexpr (F32S) r.f = static_cast<const float*>(s)[at];
    else r.b = static_cast<const uint8_t*>(s)[at];
    return r;
}

template <bool F32S>
__device__ __forceinline__ v4f mac16(v8i w, v8i x, v4f c, BlockScale<F32S> s, uint32_t sx) {
    if constexpr (F32S) {
        const Fp8Split both = fp8_split(s.f);
        const v4f p = fp8_mfma16(w, x, v4f{}, both.b, sx);
#pragma unroll
        for (int r = 0; r < 4; ++r) c[r] = __fmaf_rn(p[r], both.f, c[r]);
        return c;
    } else {
        return fp8_mfma16(w, x, c, s.b, sx);
    }
}

// What gate and up are made of in the kernels that the weight's bytes bound: a difference of their last
// bits moves some of h's codes, by a step each, so that every bit of the sum counts.  x: widened by fp8_by of its scale, sx:
// what is left of that.
template <bool F32S>
__device__ __forceinline__ v4f mac16_wide(v8i w, const Fp8Wide& x, v4f c, BlockScale<F32S> s, float sx) {
    const v4f p = fp8_mfma16_wide(fp8_widen(w, 1.0f), x);
    const float both = __fmul_rn(sx, F32S ? s.f : fp8_scale_value(s.b));
#pragma unroll
    for (int r = 0; r < 4; ++r) c[r] = __fmaf_rn(p[r], both, c[r]);
    return c;
}

// ---- a token or two: no more than kDirect rows, taken as they are ----
//
// Bound by reading the chosen experts' weights; two launches, no sorting and nothing in between but
// h, in binary32.  Both kernels code what they multiply (a row of x; the rows of h of a token) into
// LDS while their first weights are on their way.

// h of one row (a token at one of its experts) and 16 inner channels a workgroup; its four
// wavefronts take the groups of the hidden channels in turn.
template <bool F32S, int DT>
__global__ __launch_bounds__(256) void k_fp8_gate_up_direct(Fp8ExpertsArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t codes[kDirectValues], scales[kDirectValues / kGroup];
    __shared__ v4f red[2][4][4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int flat = blockIdx.y, expert = a.ids[flat];
    if ((uint32_t)expert >= (uint32_t)a.sorted.experts) return;
    const int G = (int)fp8_groups(a.hidden), IG = (int)fp8_groups(a.inner), ngroups = a.inner / 16;
    const int64_t pitch = fp8_scale_pitch(a.hidden);
    const uint8_t* wp[2];
    int64_t srow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t mat = 2 * (int64_t)expert + i;
        wp[i] = a.gate_up + (mat * ngroups + blockIdx.x) * G * kGroupBytes;
        srow[i] = (mat * IG + blockIdx.x / 8) * pitch;
    }
    constexpr int U = 4;
    v8i w[2][U][2];  // [set][group][gate, up]
    BlockScale<F32S> s[2][U][2];
    auto load = [&](int set, int g0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = min(g0 + 4 * u, G - 1);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                w[set][u][i] = fp8_fragment(wp[i] + (int64_t)g * kGroupBytes, lane);
                s[set][u][i] = block_scale<F32S>(a.gate_up_s, srow[i] + g);
            }
        }
    };
    load(0, wave);
    fp8_code_rows<DT>(static_cast<const char*>(a.raw) + flat / a.sorted.k * a.ldx * 2, 0, 1, a.hidden, codes, scales, 0);
    __syncthreads();
    v4f acc[2] = {v4f{}, v4f{}};
    auto add = [&](int set, int g0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = g0 + 4 * u;
            if (g >= G) break;
            const Fp8By sx = fp8_by(scales[g]);
            const Fp8Wide x = fp8_widen(fp8_row_fragment(codes, g, lane), sx.by);
#pragma unroll
            for (int i = 0; i < 2; ++i) acc[i] = mac16_wide<F32S>(w[set][u][i], x, acc[i], s[set][u][i], sx.rest);
        }
    };
    for (int g = wave; g < G; g += 8 * U) {
        load(1, g + 4 * U);
        add(0, g);
        load(0, g + 8 * U);
        add(1, g + 4 * U);
    }
    // every column of the product is the row: the first one's four lanes
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        fp8_settle(acc[i]);
        if ((lane & 15) == 0) red[i][wave][lane >> 4] = acc[i];
    }
    __syncthreads();
    if (threadIdx.x < 4) {
        v4f v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v[i] = red[i][0][threadIdx.x] + red[i][1][threadIdx.x] + red[i][2][threadIdx.x] + red[i][3][threadIdx.x];
        v4f h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = fp8_silu_mul(v[0][r], v[1][r]);
        *reinterpret_cast<v4f*>(a.partial + (int64_t)flat * a.inner + blockIdx.x * 16 + threadIdx.x * 4) = h;
    }
}

// y of one token and 16 hidden channels a workgroup: its rows of h one after the other, the groups
// of each dealt to the wavefronts.
template <bool F32S, int OUT>
__global__ __launch_bounds__(256) void k_fp8_down_direct(Fp8ExpertsArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t codes[kDirectValues], scales[kDirectValues / kGroup];
    __shared__ v4f red[4][4];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int k = a.sorted.k, token = blockIdx.y;
    const int G = (int)fp8_groups(a.inner), HG = (int)fp8_groups(a.hidden), ngroups = a.hidden / 16;
    const int64_t pitch = fp8_scale_pitch(a.inner);
    const int steps = k * G;  // (slot, group) pairs, taken in turn
    constexpr int U = 8;
    v8i w[U];
    BlockScale<F32S> s[U];
    float weight[U];
    auto load = [&](int p0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = min(p0 + 4 * u, steps - 1), j = p / G, g = p - j * G;
            const int expert = a.ids[token * k + j];
            const bool there = p0 + 4 * u < steps && (uint32_t)expert < (uint32_t)a.sorted.experts;
            const int64_t e = there ? expert : 0;
            w[u] = fp8_fragment(a.down + ((e * ngroups + blockIdx.x) * G + g) * kGroupBytes, lane);
            s[u] = block_scale<F32S>(a.down_s, (e * HG + blockIdx.x / 8) * pitch + g);
            weight[u] = there ? a.weights[token * k + j] : 0.0f;
        }
    };
    load(wave);
    fp8_code_rows<kF32>(a.partial + (int64_t)token * k * a.inner, a.inner, k, a.inner, codes, scales, G * kGroup);
    __syncthreads();
    v4f y = v4f{};
    for (int p0 = wave; p0 < steps; p0 += 4 * U) {
        if (p0 != wave) load(p0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + 4 * u;
            if (p >= steps) break;
            const int j = p / G, g = p - j * G;
            if ((uint32_t)a.ids[token * k + j] >= (uint32_t)a.sorted.experts) continue;  // (its h is not there)
            v4f v = mac16<F32S>(w[u], fp8_row_fragment(codes + j * G * kGroup, g, lane), v4f{}, s[u], scales[p]);
            fp8_settle(v);
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = __fmaf_rn(v[r], weight[u], y[r]);
        }
    }
    if ((lane & 15) == 0) red[wave][lane >> 4] = y;
    __syncthreads();
    if (threadIdx.x < 4) {
        const v4f v = red[0][threadIdx.x] + red[1][threadIdx.x] + red[2][threadIdx.x] + red[3][threadIdx.x];
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + token * a.ldy + blockIdx.x * 16 + threadIdx.x * 4) =
            make_uint2(f32x2_to_16<OUT>(v[0], v[1]), f32x2_to_16<OUT>(v[2], v[3]));
    }
}

// ---- blocks of 16 sorted rows ----

// One block of 16 rows and 128 inner channels a workgroup; wavefront w computes
// gate and up of the channels 32 w .. 32 w + 31.
template <bool F32S>
__global__ __launch_bounds__(256) void k_fp8_gate_up(Fp8ExpertsArgs a) {
    __shared__ uint32_t tops[4][16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Fp8Tile t = fp8_tile<16>(a.sorted, blockIdx.x, lane);
    if (t.expert < 0) return;
    const int G = (int)fp8_groups(a.hidden), pitch = (int)fp8_scale_pitch(a.hidden);
    const int IG = (int)fp8_groups(a.inner), ngroups = a.inner / 16;
    const uint8_t* xb = a.x + (int64_t)blockIdx.x * G * kGroupBytes;
    const uint8_t* xs = a.xs + ((int64_t)blockIdx.x * 16 + (lane & 15)) * pitch;
    v4f acc[2][2];
    const uint8_t* wp[2][2];
    int64_t srow[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int64_t mat = 2 * (int64_t)t.expert + i;
        srow[i] = (mat * IG + blockIdx.y) * pitch;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            wp[i][j] = a.gate_up + (mat * ngroups + min((int)blockIdx.y * 8 + 2 * wave + j, ngroups - 1)) * G * kGroupBytes;
            acc[i][j] = v4f{};
        }
    }
    for (int g = 0; g < G; ++g) {
        const Fp8By sx = fp8_by(xs[g]);
        const Fp8Wide x = fp8_widen(fp8_fragment(xb + (int64_t)g * kGroupBytes, lane), sx.by);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const BlockScale<F32S> s = block_scale<F32S>(a.gate_up_s, srow[i] + g);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = mac16_wide<F32S>(fp8_fragment(wp[i][j] + (int64_t)g * kGroupBytes, lane), x, acc[i][j], s, sx.rest);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) fp8_settle(acc[i][j]);
    float h[2][4];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            h[j][r] = (int)blockIdx.y * 8 + 2 * wave + j < ngroups ? fp8_silu_mul(acc[0][j][r], acc[1][j][r]) : 0.0f;
            top = max(top, magnitude(h[j][r]));
        }
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    if (lane < 16) tops[wave][lane] = top;
    __syncthreads();
    const int row = lane & 15;
    const uint32_t b = fp8_scale_byte(max(max(tops[0][row], tops[1][row]), max(tops[2][row], tops[3][row])));
    const float inv = fp8_inverse(b);
    uint8_t* hb = a.h + ((int64_t)blockIdx.x * IG + blockIdx.y) * kGroupBytes;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int c = 2 * wave + j;  // chunk of 16 channels in the group
#pragma unroll
        for (int r = 0; r < 4; ++r) h[j][r] *= inv;  // (whatever a group with a NaN scale holds is NaN)
        *reinterpret_cast<uint32_t*>(hb + (c >> 2) * kWBlock + fp8_pos(row, c & 3) + 4 * (lane >> 4)) =
            fp8_pack4(h[j][0], h[j][1], h[j][2], h[j][3]);
    }
    if (threadIdx.x < 16) a.hs[((int64_t)blockIdx.x * 16 + row) * fp8_scale_pitch(a.inner) + blockIdx.y] = (uint8_t)b;
}

// One block of 16 rows and 64 hidden channels a workgroup, 16 a wavefront.
template <bool F32S>
__global__ __launch_bounds__(256) void k_fp8_down(Fp8ExpertsArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Fp8Tile t = fp8_tile<16>(a.sorted, blockIdx.x, lane);
    const int ngroups = a.hidden / 16, n16 = blockIdx.y * 4 + wave;
    if (t.expert < 0 || n16 >= ngroups) return;
    const int G = (int)fp8_groups(a.inner), pitch = (int)fp8_scale_pitch(a.inner);
    const uint8_t* xb = a.h + (int64_t)blockIdx.x * G * kGroupBytes;
    const uint8_t* xs = a.hs + ((int64_t)blockIdx.x * 16 + (lane & 15)) * pitch;
    const uint8_t* wp = a.down + ((int64_t)t.expert * ngroups + n16) * G * kGroupBytes;
    const int64_t srow = ((int64_t)t.expert * fp8_groups(a.hidden) + n16 / 8) * pitch;
    constexpr int U = 4;  // groups loaded together, two sets of them on their way
    v8i w[2][U], x[2][U];
    BlockScale<F32S> s[2][U];
    uint32_t sx[2][U];
    auto load = [&](int set, int g0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = min(g0 + u, G - 1);
            w[set][u] = fp8_fragment(wp + (int64_t)g * kGroupBytes, lane);
            x[set][u] = fp8_fragment(xb + (int64_t)g * kGroupBytes, lane);
            s[set][u] = block_scale<F32S>(a.down_s, srow + g);
            sx[set][u] = xs[g];
        }
    };
    v4f acc = v4f{};
    auto add = [&](int set, int g0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g0 + u < G) acc = mac16<F32S>(w[set][u], x[set][u], acc, s[set][u], sx[set][u]);
    };
    load(0, 0);
    for (int g = 0; g < G; g += 2 * U) {
        load(1, g + U);
        add(0, g);
        load(0, g + 2 * U);
        add(1, g + U);
    }
    fp8_settle(acc);
    const int flat = fp8_sorted_row(a.sorted, t, lane & 15);
    if (flat < 0) return;
    const float weight = a.weights[flat];
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = __fmul_rn(acc[r], weight);
    *reinterpret_cast<v4f*>(a.partial + (int64_t)flat * a.hidden + n16 * 16 + 4 * (lane >> 4)) = acc;
}

// A token's rows, in the order of its slots; slots without an expert add nothing.
template <int OUT>
__global__ __launch_bounds__(256) void k_fp8_combine(Fp8ExpertsArgs a) {
    const int n = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int64_t token = blockIdx.x;
    if (n >= a.hidden) return;
    v4f y = v4f{};
    for (int j = 0; j < a.sorted.k; ++j) {
        const int64_t flat = token * a.sorted.k + j;
        if ((uint32_t)a.ids[flat] >= (uint32_t)a.sorted.experts) continue;
        const v4f p = *reinterpret_cast<const v4f*>(a.partial + flat * a.hidden + n);
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = __fadd_rn(y[r], p[r]);
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + token * a.ldy + n) =
        make_uint2(f32x2_to_16<OUT>(y[0], y[1]), f32x2_to_16<OUT>(y[2], y[3]));
}

template <bool F32S>
void launch_products(const Fp8ExpertsArgs& a, int dt, hipStream_t st) {
    // Rows of a tile by the average rows of an expert: a tile that is not full costs as much as a
    // full one.  Below 12 one block of 16 rows at a time.  Measured (us, blocks of 16 / tiles of 64 / 128 /
    // 256), 4 of 32 experts of 4096 x 1360, average rows 8: 129 / 131 / 138 / 163, 16: 154 / 137 / 146 / 171,
    // 32: 221 / 154 / 156 / 177, 64: 389 / 189 / 175 / 194, 128: - / 262 / 227 / 237, 191: 818 / 293 / 248-259 / 239-240,
    // 512: 1617 / 631 / 511 / 451; 2 of 8 of 4096 x 14336, 128: 1684 / 522 / 370 / 410, 256: 2768 / 769 / 644 / 504.
    const int64_t each = a.sorted.total / a.sorted.experts;
    const int large = F32S ? 192 : 256;
    const int rows = each >= 160 ? large : each >= 48 ? 128 : each >= 12 ? 64 : 0;
    if (rows > 0) {
        Fp8TileArgs t{};
        t.x = a.x;
        t.xs = a.xs;
        t.w = a.gate_up;
        t.ws = a.gate_up_s;
        t.ws_f32 = F32S;
        t.N = a.inner;
        t.groups = (int)fp8_groups(a.hidden);
        t.pitch = (int)fp8_scale_pitch(a.hidden);
        t.sorted = a.sorted;
        t.h = a.h;
        t.hs = a.hs;
        t.h_pitch = (int)fp8_scale_pitch(a.inner);
        // Widened products take 256 registers for less of a tile: 64 rows, or 128 from an average of 150.  Measured
        // (us, all in tiles of 64 / 128, binary16), the 32 experts above, 32: 159 / 202, 64: 200 / 225, 128: 281 / 300,
        // 191: 362 / 339; the 8, 64: 359 / 429.
        const bool wide = dt == kF16;
        launch_fp8_gate_up_tiles(t, wide, !wide ? rows : each >= 150 ? 128 : 64, st);
        t.x = a.h;
        t.xs = a.hs;
        t.w = a.down;
        t.ws = a.down_s;
        t.N = a.hidden;
        t.groups = (int)fp8_groups(a.inner);
        t.pitch = (int)fp8_scale_pitch(a.inner);
        t.y = a.partial;
        t.ldy = a.hidden;
        t.weights = a.weights;
        // Down in large tiles or, below, two of 128 x 128 a compute unit.  Measured (us, 128 x 256 / 128 x 128): the 8
        // experts, 64: 318 / 287, 256: 512 / 567 (256 x 256 / 128 x 128); the 32, 16: 135 / 135, 64: 162 / 161.
        launch_fp8_down_tiles(t, rows == large ? Fp8TileShape{large, 256} : Fp8TileShape{128, 128}, st);
        return;
    }
    const uint32_t blocks = (uint32_t)fp8_blocks(a.sorted.total, a.sorted.experts);
    hipLaunchKernelGGL((k_fp8_gate_up<F32S>), dim3(blocks, (uint32_t)fp8_groups(a.inner)), dim3(256), 0, st, a);
    hipLaunchKernelGGL((k_fp8_down<F32S>), dim3(blocks, (a.hidden + 63) / 64), dim3(256), 0, st, a);
}

template <bool F32S>
void launch_direct(const Fp8ExpertsArgs& a, int dt, hipStream_t st) {
    const dim3 up(a.inner / 16, a.sorted.total), down(a.hidden / 16, (uint32_t)a.tokens), block(256);
    if (dt == kF16) {
        hipLaunchKernelGGL((k_fp8_gate_up_direct<F32S, kF16>), up, block, 0, st, a);
        hipLaunchKernelGGL((k_fp8_down_direct<F32S, kF16>), down, block, 0, st, a);
    } else {
        hipLaunchKernelGGL((k_fp8_gate_up_direct<F32S, kBF16>), up, block, 0, st, a);
        hipLaunchKernelGGL((k_fp8_down_direct<F32S, kBF16>), down, block, 0, st, a);
    }
}

}  // namespace

bool fp8_experts_direct(int64_t rows, int64_t k, int64_t hidden, int64_t inner) {
    return rows <= kDirect && fp8_groups(hidden) * kGroup <= kDirectValues && k * fp8_groups(inner) * kGroup <= kDirectValues;
}

void launch_fp8_experts_direct(const Fp8ExpertsArgs& a, int dt, hipStream_t st) {
    if (a.ws_f32) launch_direct<true>(a, dt, st);
    else launch_direct<false>(a, dt, st);
}

void launch_fp8_experts(const Fp8ExpertsArgs& a, int out_dt, hipStream_t st) {
    if (a.ws_f32) launch_products<true>(a, out_dt, st);
    else launch_products<false>(a, out_dt, st);
    const dim3 grid((uint32_t)a.tokens, (a.hidden + 1023) / 1024);
    if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_combine<kF16>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_fp8_combine<kBF16>), grid, dim3(256), 0, st, a);
}

}  // namespace pdq

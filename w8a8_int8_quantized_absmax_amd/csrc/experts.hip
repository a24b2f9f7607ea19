// The experts' layer on 8-bit floating-point weights (gfx950): for each sorted
// row (a token at one of its experts) h = silu(Gate x) * (Up x), coded in groups of
// 128 as x is, then Down h times the row's weight, and a token's rows summed in the
// order of its slots.

#include "fp8_device.h"

namespace pdq {

namespace {

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
        const v4f p = fp8_mfma16(w, x, v4f{}, 127, sx);
#pragma unroll
        for (int r = 0; r < 4; ++r) c[r] = __fmaf_rn(p[r], s.f, c[r]);
        return c;
    } else {
        return fp8_mfma16(w, x, c, s.b, sx);
    }
}

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
        const v8i x = fp8_fragment(xb + (int64_t)g * kGroupBytes, lane);
        const uint32_t sx = xs[g];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const BlockScale<F32S> s = block_scale<F32S>(a.gate_up_s, srow[i] + g);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                acc[i][j] = mac16<F32S>(fp8_fragment(wp[i][j] + (int64_t)g * kGroupBytes, lane), x, acc[i][j], s, sx);
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
        for (int r = 0; r < 4; ++r) h[j][r] = fp8_scaled(h[j][r], inv);
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
    v4f acc = v4f{};
    for (int g = 0; g < G; ++g)
        acc = mac16<F32S>(fp8_fragment(wp + (int64_t)g * kGroupBytes, lane), fp8_fragment(xb + (int64_t)g * kGroupBytes, lane),
                          acc, block_scale<F32S>(a.down_s, srow + g), xs[g]);
    fp8_settle(acc);
    const int flat = fp8_sorted_row(a.sorted, t, lane & 15);
    if (flat < 0) return;
    const float w = a.weights[flat];
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = __fmul_rn(acc[r], w);
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
void launch_products(const Fp8ExpertsArgs& a, hipStream_t st) {
    // Rows of a tile by the average rows of an expert: a tile that is not full costs as much as a
    // full one.  Below 24 one block of 16 rows at a time.
    const int64_t each = a.sorted.total / a.sorted.experts;
    const int rows = each >= 200 ? (F32S ? 192 : 256) : each >= 64 ? 128 : each >= 24 ? 64 : 0;
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
        launch_fp8_expert_tiles(t, true, rows, st);
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
        launch_fp8_expert_tiles(t, false, rows, st);
        return;
    }
    const uint32_t blocks = (uint32_t)fp8_blocks(a.sorted.total, a.sorted.experts);
    hipLaunchKernelGGL((k_fp8_gate_up<F32S>), dim3(blocks, (uint32_t)fp8_groups(a.inner)), dim3(256), 0, st, a);
    hipLaunchKernelGGL((k_fp8_down<F32S>), dim3(blocks, (a.hidden + 63) / 64), dim3(256), 0, st, a);
}

}  // namespace

void launch_fp8_experts(const Fp8ExpertsArgs& a, int out_dt, hipStream_t st) {
    if (a.ws_f32) launch_products<true>(a, st);
    else launch_products<false>(a, st);
    const dim3 grid((uint32_t)a.tokens, (a.hidden + 1023) / 1024);
    if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_combine<kF16>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((k_fp8_combine<kBF16>), grid, dim3(256), 0, st, a);
}

}  // namespace pdq

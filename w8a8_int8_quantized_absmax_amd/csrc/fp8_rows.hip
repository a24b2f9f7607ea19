// Product of 8-bit floating-point codes for few activation rows (gfx950):
//   y[m, n] = sum over groups g of 128: S_x[m, g] S_w[n / 128, g] sum xq wq (+ bias[n]),
// every sum in binary32, one rounding to 16 bits.
//
// Bound by reading the weight.  A workgroup owns 16 NG weight channels and 16 MB
// activation rows; its four wavefronts take the groups in turn, and a group of 16
// channels is one contiguous 2 KB run of the packed weight, which lane by lane is
// the operand of one 16x16x128 product: no LDS before the sum of the four partial
// results.  The e8m0 scales go into the product itself; binary32 block scales
// multiply its result, one multiply-add a value.

#include "fp8_device.h"

namespace pdq {

namespace {

template <int NG, int MB, bool F32S>
struct Step {  // one group's operands
    v8i w[NG], x[MB];
    uint32_t sx[MB];
    float sw;      // F32S
    uint32_t swb;  // else
};

template <int NG, int MB, bool F32S, int OUT>
__global__ __launch_bounds__(256) void k_fp8_rows(Fp8GemmArgs a) {
    __shared__ v4f red[4][NG * MB][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = a.groups;
    const int n0 = blockIdx.x * 16 * NG, m0 = blockIdx.y * 16 * MB;
    const int lastw = (a.N + 15) / 16 - 1, lastx = (a.M + 15) / 16 - 1;
    const uint8_t* wp[NG];
    const uint8_t* xp[MB];
    const uint8_t* xsp[MB];
    const int off = 16 * lane;
#pragma unroll
    for (int i = 0; i < NG; ++i) wp[i] = a.w + (int64_t)min(n0 / 16 + i, lastw) * G * kGroupBytes + off;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        xp[i] = a.x + (int64_t)min(m0 / 16 + i, lastx) * G * kGroupBytes + off;
        xsp[i] = a.xs + (int64_t)min(m0 + 16 * i + (lane & 15), a.M - 1) * a.pitch;
    }
    const int64_t srow = (int64_t)(n0 / 128) * a.pitch;
    auto load = [&](Step<NG, MB, F32S>& s, int g) {
        g = min(g, G - 1);
        auto frag = [&](const uint8_t* p) {
            const v4i lo = *reinterpret_cast<const v4i*>(p + (int64_t)g * kGroupBytes);
            const v4i hi = *reinterpret_cast<const v4i*>(p + (int64_t)g * kGroupBytes + kWBlock);
            return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        };
#pragma unroll
        for (int i = 0; i < NG; ++i) s.w[i] = frag(wp[i]);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            s.x[i] = frag(xp[i]);
            s.sx[i] = xsp[i][g];
        }
        if constexpr (F32S) s.sw = static_cast<const float*>(a.ws)[srow + g];
        else s.swb = static_cast<const uint8_t*>(a.ws)[srow + g];
    };
    v4f acc[NG][MB];
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = v4f{};
    auto add = [&](const Step<NG, MB, F32S>& s) {
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                if constexpr (F32S) {
                    const v4f p = fp8_mfma16(s.w[i], s.x[j], v4f{}, 127, s.sx[j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = __fmaf_rn(p[r], s.sw, acc[i][j][r]);
                } else {
                    acc[i][j] = fp8_mfma16(s.w[i], s.x[j], acc[i][j], s.swb, s.sx[j]);
                }
            }
    };
    constexpr int U = 4 / (NG > MB ? NG : MB);  // groups loaded together
    Step<NG, MB, F32S> cur[U], nxt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(cur[u], wave + 4 * u);
    for (int g = wave; g < G; g += 4 * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(nxt[u], g + 4 * (U + u));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (g + 4 * u < G) add(cur[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) cur[u] = nxt[u];
    }
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            fp8_settle(acc[i][j]);
            red[wave][i * MB + j][lane] = acc[i][j];
        }
    __syncthreads();
    const bool vec = (reinterpret_cast<uintptr_t>(a.y) & 7) == 0 && a.ldy % 4 == 0;
#pragma unroll
    for (int b = 0; b < NG * MB; ++b) {
        if (b % 4 != wave) continue;
        v4f v = red[0][b][lane] + red[1][b][lane] + red[2][b][lane] + red[3][b][lane];
        const int n = n0 + 16 * (b / MB) + 4 * (lane >> 4), m = m0 + 16 * (b % MB) + (lane & 15);
        if (m >= a.M || n >= a.N) continue;
        if (a.bias) {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = __fadd_rn(v[r], a.bias[min(n + r, a.N - 1)]);
        }
        const uint32_t lo = f32x2_to_16<OUT>(v[0], v[1]), hi = f32x2_to_16<OUT>(v[2], v[3]);
        uint16_t* y = static_cast<uint16_t*>(a.y) + (int64_t)m * a.ldy + n;
        if (vec && n + 4 <= a.N) {
            *reinterpret_cast<uint2*>(y) = make_uint2(lo, hi);
        } else {
            const uint16_t e[4] = {(uint16_t)lo, (uint16_t)(lo >> 16), (uint16_t)hi, (uint16_t)(hi >> 16)};
            for (int r = 0; r < 4 && n + r < a.N; ++r) y[r] = e[r];
        }
    }
}

template <int NG, int MB>
void launch(const Fp8GemmArgs& a, int out_dt, hipStream_t st) {
    const dim3 grid((a.N + 16 * NG - 1) / (16 * NG), (a.M + 16 * MB - 1) / (16 * MB)), block(256);
    if (a.ws_f32 && out_dt == kF16) hipLaunchKernelGGL((k_fp8_rows<NG, MB, true, kF16>), grid, block, 0, st, a);
    else if (a.ws_f32) hipLaunchKernelGGL((k_fp8_rows<NG, MB, true, kBF16>), grid, block, 0, st, a);
    else if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_rows<NG, MB, false, kF16>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_fp8_rows<NG, MB, false, kBF16>), grid, block, 0, st, a);
}

}  // namespace

void launch_fp8_rows(const Fp8GemmArgs& a, int out_dt, hipStream_t st) {
    if (a.M <= 16) launch<1, 1>(a, out_dt, st);
    else if (a.M <= 32) launch<1, 2>(a, out_dt, st);
    else launch<2, 4>(a, out_dt, st);
}

}  // namespace pdq

// Product of 8-bit floating-point codes for few activation rows (gfx950):
//   y[m, n] = sum over groups g of 128: S_x[m, g] S_w[n / 128, g] sum xq wq (+ bias[n]),
// every sum in binary32, one rounding to 16 bits.
//
// FUSED: the activations are coded within the kernel (a few thousand values: every
// workgroup codes them all, into LDS, while its first weights are on their way), which
// saves a launch where launches are most of the time.
//
// Bound by reading the weight.  A workgroup owns 16 NG weight channels and 16 MB
// activation rows; its four wavefronts take the groups in turn, and a group of 16
// channels is one contiguous 2 KB run of the packed weight, which lane by lane is
// the operand of one 16x16x128 product: no LDS before the sum of the four partial
// results.  The e8m0 scales go into the product itself, of binary32 block scales the
// exponents; what is left of those multiplies its result, one multiply-add a value.

#include "fp8_device.h"

namespace pdq {

namespace {

constexpr int kFusedBytes = 20480;  // codes and scales of 16384 values in at most 16 padded rows

template <int NG, int MB>
struct Step {  // one group's operands
    v8i w[NG], x[MB];
    uint32_t sx[MB];
    float sw;      // F32S
    uint32_t swb;  // else
};

template <int NG, int MB, bool F32S, int OUT, bool FUSED, int W>
__global__ __launch_bounds__(64 * W) void k_fp8_rows(Fp8GemmArgs a) {
    __shared__ v4f red[W][NG * MB][64];
    __shared__ __attribute__((aligned(16))) uint8_t fused[FUSED ? kFusedBytes : 16];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = a.groups;
    const int n0 = blockIdx.x * 16 * NG, m0 = blockIdx.y * 16 * MB;
    const int lastw = (a.N + 15) / 16 - 1, lastx = (a.M + 15) / 16 - 1;
    const uint8_t* wp[NG];
    const uint8_t* xp[MB];
    const uint8_t* xsp[MB];
#pragma unroll
    for (int i = 0; i < NG; ++i) wp[i] = a.w + (int64_t)min(n0 / 16 + i, lastw) * G * kGroupBytes + 16 * lane;
    const int pitch = G * kGroup + 16;  // FUSED
    uint8_t* const scales = fused + a.M * pitch;
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int m = min(m0 + 16 * i + (lane & 15), a.M - 1);
        xp[i] = FUSED ? fused + m * pitch + (lane >> 4) * 16
                      : a.x + (int64_t)min(m0 / 16 + i, lastx) * G * kGroupBytes + 16 * lane;
        xsp[i] = FUSED ? scales + m * G : a.xs + (int64_t)m * a.pitch;
    }
    constexpr int kStep = FUSED ? kGroup : kGroupBytes, kHalf = FUSED ? kGroup / 2 : kWBlock;
    const int64_t srow = (int64_t)(n0 / 128) * a.pitch;
    auto frag = [&](const uint8_t* p, int step, int half) {
        const v4i lo = *reinterpret_cast<const v4i*>(p + step);
        const v4i hi = *reinterpret_cast<const v4i*>(p + step + half);
        return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    auto load = [&](Step<NG, MB>& s, int g) {
        g = min(g, G - 1);
#pragma unroll
        for (int i = 0; i < NG; ++i) s.w[i] = frag(wp[i] + (int64_t)g * kGroupBytes, 0, kWBlock);
        if constexpr (!FUSED) {
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                s.x[i] = frag(xp[i] + (int64_t)g * kStep, 0, kHalf);
                s.sx[i] = xsp[i][g];
            }
        }
        if constexpr (F32S) s.sw = static_cast<const float*>(a.ws)[srow + g];
        else s.swb = static_cast<const uint8_t*>(a.ws)[srow + g];
    };
    auto load_fused = [&](Step<NG, MB>& s, int g) {
        g = min(g, G - 1);
#pragma unroll
        for (int i = 0; i < MB; ++i) {
            s.x[i] = frag(xp[i] + g * kStep, 0, kHalf);
            s.sx[i] = xsp[i][g];
        }
    };
    v4f acc[NG][MB];
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = v4f{};
    auto add = [&](const Step<NG, MB>& s) {
        const Fp8Split sw = F32S ? fp8_split(s.sw) : Fp8Split{};
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j) {
                if constexpr (F32S) {
                    const v4f p = fp8_mfma16(s.w[i], s.x[j], v4f{}, sw.b, s.sx[j]);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[i][j][r] = __fmaf_rn(p[r], sw.f, acc[i][j][r]);
                } else {
                    acc[i][j] = fp8_mfma16(s.w[i], s.x[j], acc[i][j], s.swb, s.sx[j]);
                }
            }
    };
    constexpr int U = 4 / (NG > MB ? NG : MB);  // groups loaded together
    Step<NG, MB> cur[U], nxt[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(cur[u], wave + W * u);
    if constexpr (FUSED) {
        if (a.raw_dt == kF32) fp8_code_rows<kF32>(a.raw, a.ldx, a.M, a.K, fused, scales, pitch);
        else if (a.raw_dt == kBF16) fp8_code_rows<kBF16>(a.raw, a.ldx, a.M, a.K, fused, scales, pitch);
        else fp8_code_rows<kF16>(a.raw, a.ldx, a.M, a.K, fused, scales, pitch);
        __syncthreads();
    }
    for (int g = wave; g < G; g += W * U) {
#pragma unroll
        for (int u = 0; u < U; ++u) load(nxt[u], g + W * (U + u));
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if constexpr (FUSED) load_fused(cur[u], g + W * u);
            if (g + W * u < G) add(cur[u]);
        }
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
        if (b % W != wave) continue;
        v4f v = red[0][b][lane];
#pragma unroll
        for (int w = 1; w < W; ++w) v += red[w][b][lane];
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

template <int NG, int MB, bool FUSED, int W>
void launch(const Fp8GemmArgs& a, int out_dt, hipStream_t st) {
    const dim3 grid((a.N + 16 * NG - 1) / (16 * NG), (a.M + 16 * MB - 1) / (16 * MB)), block(64 * W);
    if (a.ws_f32 && out_dt == kF16) hipLaunchKernelGGL((k_fp8_rows<NG, MB, true, kF16, FUSED, W>), grid, block, 0, st, a);
    else if (a.ws_f32) hipLaunchKernelGGL((k_fp8_rows<NG, MB, true, kBF16, FUSED, W>), grid, block, 0, st, a);
    else if (out_dt == kF16) hipLaunchKernelGGL((k_fp8_rows<NG, MB, false, kF16, FUSED, W>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_fp8_rows<NG, MB, false, kBF16, FUSED, W>), grid, block, 0, st, a);
}

}  // namespace

// Up to 16 rows of together as many values as a workgroup codes in the time that a launch takes.
bool fp8_fusable(int64_t M, int64_t K) {
    const int64_t groups = fp8_groups(K);
    return M <= 16 && M * groups * kGroup <= 16384 && M * (groups * kGroup + 16 + groups) <= kFusedBytes;
}

// Channels of a workgroup (16 or 32, 64 with 33 rows or more), and whether eight wavefronts share its
// groups instead of four.  Wide workgroups read the activations less often, narrow ones keep all
// 256 compute units at the weight.  Measured with K = 4096 (us; 16 / 32 channels, four wavefronts):
//   8 rows:  N 4096 5.9 / 7.0, 8192 9.3 / 8.7, 11008 12.6 / 12.5, 16384 16.7 / 14.1, 28672 28.1 / 24.0
//   24 rows: N 4096 7.3 / 8.7, 8192 12.0 / 10.0, 11008 16.5 / 14.9, 28672 35.7 / 29.2
//   64 rows (16 with eight wavefronts / 32 / 64): N 4096 10.5 / 11.3 / 14.7, 8192 18.8 / 12.9 / 15.6,
//            11008 27.0 / 20.2 / 17.2, 28672 60.2 / 37.2 / 30.6
//   coded within (16 with eight / 16 / 32): N 4096 5.9 / 6.3 / 7.0, 11008 12.4 / 10.7 / 11.9,
//            16384 15.6 / 14.5 / 14.5, 28672 25.8 / 23.1 / 21.9; K = 11008, N 4096: 11.9 / 14.4 / 16.3
void launch_fp8_rows(const Fp8GemmArgs& a, int out_dt, hipStream_t st) {
    const int groups = (a.N + 15) / 16;  // of 16 channels
    if (a.raw) {
        if (groups < 512) launch<1, 1, true, 8>(a, out_dt, st);
        else if (groups < 1024) launch<1, 1, true, 4>(a, out_dt, st);
        else launch<2, 1, true, 4>(a, out_dt, st);
    } else if (a.M <= 16) {
        if (groups < 512) launch<1, 1, false, 4>(a, out_dt, st);
        else launch<2, 1, false, 4>(a, out_dt, st);
    } else if (a.M <= 32) {
        if (groups < 512) launch<1, 2, false, 4>(a, out_dt, st);
        else launch<2, 2, false, 4>(a, out_dt, st);
    } else {
        const int width = fp8_rows_width(a.M, a.N);
        if (width == 1) launch<1, 4, false, 8>(a, out_dt, st);
        else if (width == 2) launch<2, 4, false, 4>(a, out_dt, st);
        else launch<4, 4, false, 4>(a, out_dt, st);
    }
}

// Groups of 16 channels of a workgroup for 33 rows or more: as many as leave some 170 workgroups.
int fp8_rows_width(int64_t M, int64_t N) {
    const int64_t units = (N + 15) / 16 * ((M + 63) / 64);
    return units >= 680 ? 4 : units >= 384 ? 2 : 1;
}

}  // namespace pdq

// 8-bit floating-point codes with a scale for each group of 128 (gfx950).
//
// Activations: for each row and group of 128 K values C = max |x|, S the
// smallest power of two with C <= 448 S, code = e4m3(x / S).  The division is
// exact, so that a code is off by half a step of e4m3 and nothing else, and the
// matrix instructions take S as it is (the e8m0 operand of the scaled products):
// no arithmetic on the accumulators between groups.
// Weights: the same with one scale for 128 rows x 128 K values.
//
// Bound by memory: one read of x, codes and scales written once.

#include "fp8_device.h"
#include "pdq_kernels.h"

namespace pdq {

namespace {

// A workgroup codes 16 rows x 4 groups (8 KB of packed codes, one dword of scales a
// row): wavefront w the rows 4 w .. 4 w + 3, 16 lanes a row, 8 values a lane and
// group, the row's maximum by lane permutations within its 16 lanes.  A wavefront's
// loads are 4 rows x 256 bytes; the codes take their places in LDS and leave as one
// contiguous run.
template <int DT>
__global__ __launch_bounds__(256) void k_fp8_quant(Fp8QuantArgs a) {
    __shared__ __attribute__((aligned(16))) uint8_t image[4 * kGroupBytes];
    const int lane = threadIdx.x & 63, r = threadIdx.x >> 4;  // row of the 16-row block
    const int gpieces = (a.groups + 3) / 4;
    const int64_t block = blockIdx.x / gpieces;
    const int g0 = (int)(blockIdx.x % gpieces) * 4;
    const int64_t row = block * 16 + r;
    int64_t src = row < a.M ? row : -1;
    if (a.sorted.offsets) {
        const Fp8Tile tile = fp8_tile<16>(a.sorted, (int)block, lane);
        const int flat = fp8_sorted_row(a.sorted, tile, r);
        src = flat < 0 ? -1 : flat / a.sorted.k;
    }
    const bool live = src >= 0;
    const char* xr = static_cast<const char*>(a.x) + (live ? src * a.ldx : 0) * Elem<DT>::bytes;
    const int c8 = lane & 15;  // chunk of 8 values in the group
    Raw8<DT> raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int k = (g0 + i) * kGroup + c8 * 8;
        raw[i] = live && k < a.K ? load_raw8<DT>(xr, k / 8) : zero_raw8<DT>();
    }
    uint32_t scales = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (g0 + i >= a.groups) break;
        float v[8];
        widen8<DT>(raw[i], v);
        const uint32_t b = fp8_scale_byte(row16_max(fp8_top8(v)));
        const int c16 = c8 >> 1;
        *reinterpret_cast<uint2*>(image + i * kGroupBytes + (c16 >> 2) * kWBlock + fp8_pos(r, c16 & 3) + 8 * (c8 & 1)) =
            fp8_code8(v, b);
        scales |= b << (8 * i);
    }
    if (c8 == 0 && (a.sorted.offsets || row < a.M))
        *reinterpret_cast<uint32_t*>(a.scale + row * a.pitch + g0) = scales;
    __syncthreads();
    uint4* out = reinterpret_cast<uint4*>(a.q + (block * a.groups + g0) * kGroupBytes);
    const int chunks = min(a.groups - g0, 4) * (kGroupBytes / 16);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int c = threadIdx.x + 256 * i;
        if (c < chunks) out[c] = reinterpret_cast<const uint4*>(image)[c];
    }
}

// One block of 128 x 128 weights a workgroup: its values stay in registers (8
// rows of 8 values a thread) between the maximum and the codes.
template <int DT>
__global__ __launch_bounds__(256) void k_fp8_weight(Fp8WeightArgs a) {
    __shared__ uint32_t tops[4];
    const int groups = (int)fp8_groups(a.K), nblocks = (int)fp8_groups(a.N), pitch = (int)fp8_scale_pitch(a.K);
    const int g = blockIdx.x % groups;
    const int nb = (int)(blockIdx.x / groups % nblocks);
    const int64_t mat = blockIdx.x / ((int64_t)groups * nblocks);
    const int r16 = threadIdx.x >> 4, c8 = threadIdx.x & 15, k = g * kGroup + c8 * 8;
    const char* w = static_cast<const char*>(a.w) + mat * a.stride * Elem<DT>::bytes;
    Raw8<DT> raw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t n = nb * 128 + i * 16 + r16;
        raw[i] = n < a.N && k < a.K ? load_raw8<DT>(w + n * a.ldw * Elem<DT>::bytes, k / 8) : zero_raw8<DT>();
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        widen8<DT>(raw[i], v);
        top = max(top, fp8_top8(v));
    }
    top = row16_max(top);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
    __syncthreads();
    const uint32_t b = fp8_scale_byte(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
    const int64_t ngroups = (a.N + 15) / 16;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t g16 = nb * 8 + i;
        if (g16 >= ngroups) break;
        float v[8];
        widen8<DT>(raw[i], v);
        const int c16 = c8 >> 1;
        uint8_t* blk = a.q + ((mat * ngroups + g16) * groups + g) * kGroupBytes + (c16 >> 2) * kWBlock;
        *reinterpret_cast<uint2*>(blk + fp8_pos(r16, c16 & 3) + 8 * (c8 & 1)) = fp8_code8(v, b);
    }
    // the row's padding up to the pitch: scales of 1
    uint8_t* s = a.scale + (mat * nblocks + nb) * pitch;
    if (threadIdx.x == 0) s[g] = (uint8_t)b;
    if (g == groups - 1 && (int)threadIdx.x > 0 && groups - 1 + (int)threadIdx.x < pitch) s[g + threadIdx.x] = 127;
}

// Codes of another tool, row-major, to the packed layout: 16 bytes a thread.
__global__ __launch_bounds__(256) void k_fp8_pack(Fp8PackArgs a, int64_t chunks) {
    const int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (t >= chunks) return;
    const int64_t groups = fp8_groups(a.K), ngroups = (a.N + 15) / 16;
    // t: the chunk in the packed image, blocks of 64 chunks
    const int in = (int)(t & 63), r = in & 15, c = in >> 4;
    const int64_t blk = t >> 6, kt = blk % (2 * groups), g16 = blk / (2 * groups) % ngroups, mat = blk / (2 * groups * ngroups);
    const int64_t n = g16 * 16 + r, k = kt * kWTileK + c * 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n < a.N && k < a.K) v = *reinterpret_cast<const uint4*>(a.codes + (mat * a.N + n) * a.K + k);
    reinterpret_cast<uint4*>(a.q)[t] = v;
}

// A weight's block scales, dense, to rows of a whole number of four.
template <typename T>
__global__ __launch_bounds__(256) void k_fp8_scales(const T* in, T* out, int64_t rows, int groups, int pitch, T one) {
    const int64_t t = blockIdx.x * (int64_t)256 + threadIdx.x;
    if (t >= rows * pitch) return;
    const int64_t row = t / pitch;
    const int g = (int)(t % pitch);
    out[t] = g < groups ? in[row * groups + g] : one;
}

}  // namespace

void launch_fp8_quant(const Fp8QuantArgs& a, int dt, int64_t blocks, hipStream_t st) {
    const dim3 grid((uint32_t)(blocks * ((a.groups + 3) / 4)));
    if (dt == kF32)
        hipLaunchKernelGGL((k_fp8_quant<kF32>), grid, dim3(256), 0, st, a);
    else if (dt == kBF16)
        hipLaunchKernelGGL((k_fp8_quant<kBF16>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_fp8_quant<kF16>), grid, dim3(256), 0, st, a);
}

void launch_fp8_weight(const Fp8WeightArgs& a, int dt, hipStream_t st) {
    const dim3 grid((uint32_t)(a.count * fp8_groups(a.N) * fp8_groups(a.K)));
    if (dt == kF32)
        hipLaunchKernelGGL((k_fp8_weight<kF32>), grid, dim3(256), 0, st, a);
    else if (dt == kBF16)
        hipLaunchKernelGGL((k_fp8_weight<kBF16>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((k_fp8_weight<kF16>), grid, dim3(256), 0, st, a);
}

void launch_fp8_pack(const Fp8PackArgs& a, hipStream_t st) {
    const int64_t groups = fp8_groups(a.K), pitch = fp8_scale_pitch(a.K);
    const int64_t chunks = a.count * ((a.N + 15) / 16) * groups * (kGroupBytes / 16);
    hipLaunchKernelGGL(k_fp8_pack, dim3((uint32_t)((chunks + 255) / 256)), dim3(256), 0, st, a, chunks);
    const int64_t rows = a.count * fp8_groups(a.N);
    const dim3 grid((uint32_t)((rows * pitch + 255) / 256));
    if (a.f32)
        hipLaunchKernelGGL((k_fp8_scales<float>), grid, dim3(256), 0, st, static_cast<const float*>(a.scale),
                           static_cast<float*>(a.scale_out), rows, (int)groups, (int)pitch, 1.0f);
    else
        hipLaunchKernelGGL((k_fp8_scales<uint8_t>), grid, dim3(256), 0, st, static_cast<const uint8_t*>(a.scale),
                           static_cast<uint8_t*>(a.scale_out), rows, (int)groups, (int)pitch, (uint8_t)127);
}

}  // namespace pdq

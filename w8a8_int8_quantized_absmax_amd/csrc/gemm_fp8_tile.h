// Tiled product of 8-bit floating-point codes (gfx950): the kernel of gemm_fp8.hip (power-of-two
// scales of the weights), gemm_fp8_f32.hip (binary32 ones) and gemm_fp8_wide.hip (widened codes).
//
//   acc[m, n] = sum over groups g of 128: S_x[m, g] S_w[n / 128, g] sum xq wq
//
// on the scaled products v_mfma_scale_f32_16x16x128: a group is one instruction, both
// scales are operands of it, and nothing else touches the accumulators: an FP8 product
// with a scale for each block of 128 costs what one without scales does.
//
// A tile of 64 NA rows x 64 NB channels a workgroup of four wavefronts, 2 x 2, each 32 NA rows x 32 NB
// channels.  NA = NB = 4, or 2 and 4: one workgroup a compute unit; 2 and 2: two, which fill each other's begins
// and ends, where a compute unit has few tiles.  Bound by the matrix unit (at NA = 4 by the power that it draws:
// 16x16x128 runs 8% faster than 32x32x64 there, 4.29 against 3.96 PFLOP/s from registers
// alone), so that all else has to run beside it:
// - K in steps of a group.  Operands come through LDS, without registers: a packed block of 16
//   rows x 128 K values (2 KB) is its own LDS image, free of bank conflicts (fp8_device.h).
// - A wavefront's rows and channels are two halves each; a step is four quadrants of products,
//   Alo F, Alo S, Ahi S, Ahi F, with F and S the channels' halves, first lo, hi, in the next step
//   hi, lo.  Each quadrant uses one operand half of the quadrant before and a new one, which is
//   read from LDS during the quadrant before: 128 registers of operands hold it all.
// - Two steps are in LDS.  What a step has read twice two quadrants ago is refilled, for the step
//   after the next, after each barrier: two barriers a step, every load sent 1.5 steps
//   (some 3000 clocks) before it is needed.
// - The scales of four groups are one dword a row; they come through LDS too.
// - The outputs leave from the accumulators (through LDS, for longer runs of a row together: the same time).
// What one tile of a compute unit costs beside its steps (1.5 us each at NA = NB = 4): some 5 us, 7 for gate and
// up, of it 3 and 5 the vector unit's in the epilogue, which no other tile's products run beside.

#pragma once

#include <type_traits>

#include "fp8_device.h"

namespace pdq {

namespace {

constexpr int kXcds = 8;

typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int waitcnt_imm(int vm, int lgkm) { return (vm & 15) | ((vm >> 4) << 14) | (7 << 4) | (lgkm << 8); }

// At most VM of this wavefront's loads still on their way, its LDS reads done, then the
// workgroup's barrier (by builtins, which the compiler's own waits count on).
template <int VM>
__device__ __forceinline__ void wait_loads_and_sync() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(VM, 0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Consecutive workgroups run on different XCDs, each with an L2 of its own: every XCD
// takes a contiguous run of tiles, walked in groups of kGroupM tile rows: 4, of the experts 8
// (2 / 4 / 8 / 16: 8192 tokens to 2 of 8 of 4096 x 14336 2667 / 2548 / 2509 / 2566 us; 4096 x 11008 x 4096 177 / 177 / 179 /
// 187; 8192 x 4096 x 14336, binary32 scales 512 / 502 / 501 / 508).
template <int kGroupM>
__device__ __forceinline__ void tile_of(int bid, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int num = tiles_m * tiles_n;
    const int q = num / kXcds, r = num % kXcds;
    const int xcd = bid % kXcds, local = bid / kXcds;
    const int id = xcd < r ? xcd * (q + 1) + local : r * (q + 1) + (xcd - r) * q + local;
    const int per_group = kGroupM * tiles_n;
    const int first = id / per_group * kGroupM;
    const int size = min(tiles_m - first, kGroupM);
    const int in = id - first * tiles_n;
    tm = first + in % size;
    tn = in / size;
}

// (fp8_mfma16 with both scales from byte B of their dwords)
template <int B>
__device__ __forceinline__ v4f mfma(v8i w, v8i x, v4f c, int sw, int sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, B, sw, B, sx);
}

// A buffer that begins at p (the same in every lane), for loads by 32-bit offsets: a tile's
// operands are at most 16 blocks of 16 rows x 65536 bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const uint8_t* p) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, 0x7fffffff, 0x00027000);
}

// What a tile of outputs becomes.
enum { kDense = 0, kGateUp = 1, kDown = 2 };

// EPI kDense: 16-bit y, type OUT.  The experts' products take the rows of a tile from one
// expert's sorted rows; kGateUp: 128 channels of gate and the same 128 of up, 64 of each the
// halves of a wavefront's channels, so that a lane holds both of a channel, and h's codes come
// out; kDown: weighted binary32 rows at their token and slot.
//
// F32S: binary32 block scales.  Their exponents go into the product (fp8_split), and what is left, 1 to 2, multiplies a group's
// product, a multiply-add a value: with them the vector unit is busy for 39% of the clocks (20% without), the matrix unit for
// 47%, and a SIMD's one wavefront, there for 86%, mostly waits for one of the two.  The accumulators are in
// vector registers (NA at most 3: 192 of 256), the products' results wait kLag products for theirs.  (With
// NA = NB = 2 one workgroup multiplies while the other adds: 1024 x 4096 x 4096 in 23 us where 128 x 256 took 33.)
//
// WIDE (gate and up of binary16 rows, NA at most 2): the codes are widened between LDS and the product, and 16-bit
// products take their place (fp8_widen); a group's sum is multiplied by both scales.  The FP8 products'
// alignment moves a few of h's codes by a step (2^-3 of them): unseen beside a bfloat16 rounding, but
// six times a binary16 one.
template <int EPI, int OUT, int NA, int NB, bool F32S, bool WIDE = false>
__global__ __launch_bounds__(256, NB == 4 ? 1 : 2) void k_fp8_tile(Fp8TileArgs a) {
    constexpr int BN = 64 * NB;
    // [step % 2][half], each an object of its own: the compiler then knows which loads into LDS
    // a read has to wait for.  Behind the first, four groups' scales.
    constexpr int kARegion = 4 * NA * kWBlock, kBRegion = 4 * NB * kWBlock, kScaleWords = 512;
    __shared__ __attribute__((aligned(1024))) uint8_t A00[kARegion + 4 * kScaleWords], A01[kARegion], A10[kARegion], A11[kARegion];
    __shared__ __attribute__((aligned(1024))) uint8_t B00[kBRegion], B01[kBRegion], B10[kBRegion], B11[kBRegion];
    __shared__ __attribute__((aligned(16))) float s_aux[256];  // kDense: bias; kDown: the rows' weights
    __shared__ int32_t s_flat[EPI == kDown ? 256 : 1];
    uint32_t* const sc = reinterpret_cast<uint32_t*>(A00 + kARegion);
    auto regionA = [&](auto buf, auto half) -> uint8_t* {
        constexpr int b = decltype(buf)::value & 1, h = decltype(half)::value;
        if constexpr (b == 0 && h == 0) return A00;
        else if constexpr (b == 0) return A01;
        else if constexpr (h == 0) return A10;
        else return A11;
    };
    auto regionB = [&](auto buf, auto half) -> uint8_t* {
        constexpr int b = decltype(buf)::value & 1, h = decltype(half)::value;
        if constexpr (b == 0 && h == 0) return B00;
        else if constexpr (b == 0) return B01;
        else if constexpr (h == 0) return B10;
        else return B11;
    };
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    constexpr int kRows = 64 * NA;  // of this tile
    const int tiles_n = EPI == kGateUp ? (a.N + 127) / 128 : (a.N + BN - 1) / BN;
    int tm, tn;
    Fp8Tile t{};
    int m0;
    if constexpr (EPI == kDense) {
        tile_of<4>(blockIdx.x, (a.M + kRows - 1) / kRows, tiles_n, tm, tn);
        m0 = tm * kRows;
    } else {
        const int tiles_m = fp8_tiles<kRows>(a.sorted, lane);
        if ((int)blockIdx.x >= tiles_m * tiles_n) return;
        tile_of<8>(blockIdx.x, tiles_m, tiles_n, tm, tn);
        t = fp8_tile<kRows>(a.sorted, tm, lane);
        m0 = t.block * 16;
    }
    const int n0 = tn * (EPI == kGateUp ? 128 : BN);
    const int G = a.groups;

    v4f acc[8][8];  // 2 NA rows, 2 NB columns used
#pragma unroll
    for (int i = 0; i < 2 * NA; ++i)
#pragma unroll
        for (int j = 0; j < 2 * NB; ++j) {
            acc[i][j] = v4f{};
            // accumulation registers: the products then work on them in place
            if constexpr (!F32S && !WIDE) asm volatile("" : "+a"(acc[i][j]));
        }
    if constexpr (EPI == kDense) {
        if (tid < BN) s_aux[tid] = a.bias && n0 + tid < a.N ? a.bias[n0 + tid] : 0.0f;
    } else if constexpr (EPI == kDown) {
        const int flat = fp8_sorted_row(a.sorted, t, tid);
        s_flat[tid] = flat;
        s_aux[tid] = flat < 0 ? 0.0f : a.weights[flat];
    }
    __syncthreads();

    // Loads of a half of a step: 4 NA blocks of 1 KB of the rows, 4 NB of the channels, of which a
    // wavefront sends NA and NB.  Offsets are from the tile's first block; blocks past the last of
    // the operand are the last one's: they only feed outputs that are not stored.
    const int blocks_n = (a.N + 15) / 16;  // of one matrix
    const int lasta = EPI == kDense ? (a.M - 1) / 16 : t.block + (t.rows - 1) / 16;
    const auto xrsrc = resource(a.x + (int64_t)(m0 / 16) * G * kGroupBytes);
    const uint8_t* const wbase =
        a.w + ((EPI == kGateUp ? 2 : 1) * (int64_t)t.expert * blocks_n + n0 / 16) * G * kGroupBytes;
    const auto wrsrc = resource(wbase);
    const auto ursrc = resource(EPI == kGateUp ? wbase + (int64_t)blocks_n * G * kGroupBytes : wbase);
    int oa[2][4], ob[2][4];  // [half]; 4 of them whatever NA and NB are: an array of a dependent size loses the host's stub
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < NA; ++i) {
            const int piece = wave * NA + i, b = piece >> 1;  // block b % NA of wavefront row b / NA
            oa[h][i] = min(b / NA * 2 * NA + h * NA + b % NA, lasta - m0 / 16) * (G * kGroupBytes) +
                       (piece & 1) * kWBlock + lane * 16;
        }
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int piece = wave * NB + i, b = piece >> 1;  // block b % NB of wavefront column b / NB
            const int at = EPI == kGateUp ? b : b / NB * 2 * NB + h * NB + b % NB;
            ob[h][i] = min(at, blocks_n - 1 - n0 / 16) * (G * kGroupBytes) + (piece & 1) * kWBlock + lane * 16;
        }
    }
    constexpr int kLoads = NA + NB;
    auto issue = [&](auto buf, auto ha, auto hb, int g, int q) {  // load q of the halves ha of the rows, hb of the channels
        const int at = min(g, G - 1) * kGroupBytes;
        constexpr int A = decltype(ha)::value, B = decltype(hb)::value;
        if (q < NA)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(xrsrc, (lds_ptr_t)(regionA(buf, ha) + (wave * NA + q) * kWBlock), 16,
                                                     oa[A][q < NA ? q : 0], at, 0, 0);
        else
            __builtin_amdgcn_raw_ptr_buffer_load_lds(B ? ursrc : wrsrc,
                                                     (lds_ptr_t)(regionB(buf, hb) + (wave * NB + q - NA) * kWBlock), 16,
                                                     ob[B][q < NA ? 0 : q - NA], at, 0, 0);
    };
    // Four groups' scales: of the activation row `tid`, and of the tile's two blocks of
    // weight rows in turn, for each wavefront its own copy.  (Sent every second step, for the next
    // two: where those are of the same four, with the values that are there.)
    const int last_row = EPI == kDense ? a.M - 1 : lasta * 16 + 15;
    const int blocks_w = (a.N + 127) / 128;
    const uint8_t* ps = a.xs + (int64_t)min(m0 + tid, last_row) * a.pitch;
    auto scale_row = [&](int b) {  // of the tile's block b of weight rows
        if constexpr (EPI == kGateUp) return ((2 * (int64_t)t.expert + b) * blocks_w + tn) * a.pitch;
        else return ((int64_t)t.expert * blocks_w + min((n0 + 32 * NB * b) / 128, blocks_w - 1)) * a.pitch;
    };
    const uint8_t* pw = static_cast<const uint8_t*>(a.ws) + (F32S ? 0 : scale_row(lane & 1));
    auto issue_scales = [&](int g) {
        const int at = min(g, G - 1) & ~3;
        __builtin_amdgcn_global_load_lds(ps + at, (lds_ptr_t)(sc + wave * 64), 4, 0, 0);
        if constexpr (!F32S) __builtin_amdgcn_global_load_lds(pw + at, (lds_ptr_t)(sc + 256 + wave * 64), 4, 0, 0);
    };
    const int off = 16 * lane;
    v4i fa[2][4][2], fb[2][4][2];  // [half][block][K half]
    auto read_a = [&](auto buf, auto half, int q) {
        fa[decltype(half)::value][q >> 1][q & 1] =
            *reinterpret_cast<const v4i*>(regionA(buf, half) + (wm * NA + (q >> 1)) * kGroupBytes + (q & 1) * kWBlock + off);
    };
    auto read_b = [&](auto buf, auto half, int q) {
        fb[decltype(half)::value][q >> 1][q & 1] =
            *reinterpret_cast<const v4i*>(regionB(buf, half) + (wn * NB + (q >> 1)) * kGroupBytes + (q & 1) * kWBlock + off);
    };
    auto whole = [](const v4i (&f)[2]) { return v8i{f[0][0], f[0][1], f[0][2], f[0][3], f[1][0], f[1][1], f[1][2], f[1][3]}; };
    int sx[8], sw[2] = {0, 0};
    auto read_scales = [&](int g) {  // of steps g and g + 1 (g even) in the low bytes
        const int shift = 8 * (g & 2), width = g + 1 < G ? 16 : 8;
        auto two = [&](uint32_t four) { return (int)__builtin_amdgcn_ubfe(four, shift, width); };
#pragma unroll
        for (int i = 0; i < 2 * NA; ++i) sx[i] = two(sc[(wm * 2 * NA + i) * 16 + (lane & 15)]);
        if constexpr (!F32S) {
            sw[0] = two(sc[256 + wave * 64 + (EPI == kGateUp ? 0 : wn)]);
            sw[1] = EPI == kGateUp ? two(sc[256 + wave * 64 + 1]) : sw[0];
        }
    };
    // F32S: the scales (their factors: fp8_split) of step g of the wavefront's halves of channels, and of the step before
    float ws[2] = {0.0f, 0.0f}, before[2] = {0.0f, 0.0f}, next[2][2];
    const float* pf[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) pf[h] = static_cast<const float*>(a.ws) + (F32S ? scale_row(EPI == kGateUp ? h : wn) : 0);
    // The next step's, split between this one's products, the factors in scalar registers: with vector registers in each
    // multiply-add 8192 x 14336 -> 4096 takes 515 us instead of 502.
    Fp8Split ahead[2] = {};
    auto split_ahead = [&](int s, int h) {
        const Fp8Split split = fp8_split(next[s][h]);
        ahead[h].f = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(split.f)));
        ahead[h].b = split.b;
    };
    auto fetch_f32 = [&](int g) {  // g even; a group beyond the last counts nothing
        const int at = min(g, G - 1) & ~1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            next[0][h] = uniform_load(pf[h] + at);
            next[1][h] = g + 1 < G ? uniform_load(pf[h] + at + 1) : 0.0f;
        }
    };
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    issue_scales(0);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) issue(I0{}, I0{}, I0{}, 0, q);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) issue(I0{}, I1{}, I1{}, 0, q);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) issue(I1{}, I0{}, I1{}, 1, q);
#pragma unroll
    for (int q = 0; q < kLoads; ++q) issue(I1{}, I1{}, I0{}, 1, q);
    wait_loads_and_sync<3 * kLoads>();
    read_scales(0);
    if constexpr (F32S) {
        fetch_f32(0);
#pragma unroll
        for (int h = 0; h < 2; ++h) split_ahead(0, h);
    }
#pragma unroll
    for (int q = 0; q < 2 * NA; ++q) read_a(I0{}, I0{}, q);
#pragma unroll
    for (int q = 0; q < 2 * NB; ++q) read_b(I0{}, I0{}, q);

    // Half a step: the rows' half HA by the channels' HB, then by the other.  The first products run
    // ahead of the barrier behind which `load` may refill what was read and `read1`, `read2` (n1,
    // n2 reads of 16 bytes a lane) find what the next two quadrants take.  Reads and loads go
    // evenly between the products: four wavefronts' reads behind each other's products would
    // keep LDS busy for longer than the products take.
    constexpr int kLag = 4, kRing = 8;
    v4f part_sum[kRing];  // WIDE: [row % 2][channels' block]
    v8bf wide_b[4][4];
    // Of binary16 rows S_x is 2^-32 to 2^8.  Its codes are widened by 2^16, which its scale lacks then: so no S_x S_w
    // passes 2^128 where the sum is 0.
    constexpr uint32_t kWideBy = 16;
    float both[2];
#pragma unroll
    for (int q = 0; q < kRing; ++q) part_sum[q] = v4f{};
    auto half = [&](auto HA, auto HB, auto BYTE, auto&& load, auto&& read1, auto N1, auto&& read2, auto N2) {
        constexpr int ha = decltype(HA)::value, kByte = decltype(BYTE)::value;
        constexpr int n1 = decltype(N1)::value, n2 = decltype(N2)::value;
        constexpr int L = NB * NA;                      // products of a quadrant
        constexpr int kAhead = NA == 4 ? 2 : 1;         // products before the barrier
        constexpr int kSpan1 = L - kAhead - L / 4, kSpan2 = L - L / 4;  // the last reads' latency under the last quarter
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 2 * L; ++q) {
            const int i = q % L / NB, j = q % NB, hb = q < L ? decltype(HB)::value : 1 - decltype(HB)::value;
            if (q == kAhead) {
                wait_loads_and_sync<2 * kLoads>();
                __builtin_amdgcn_sched_barrier(0);
            }
            if constexpr (WIDE) {
                // a quarter (j) of the group's K values: row block i by the half's four blocks of channels
                const int at = i & 1;
                if (j == 0) {
                    const uint32_t byte = (uint32_t)sx[ha * NA + i] >> 8 * kByte & 255;
                    // (byte 0: the group behind an odd last one)
                    const float s = __uint_as_float(byte == 255u ? 0x7fc00000u : __builtin_elementwise_sub_sat(byte, kWideBy) << 23);
                    both[at] = __fmul_rn(s, ws[hb]);
                }
                if (i == 0 && !(ha == 1 && q < L)) {  // (those of the quadrant before are the same ones)
#pragma unroll
                    for (int b = 0; b < 4; ++b)
                        wide_b[b][j] = fp8_widen8(fb[hb][b][j >> 1][2 * (j & 1)], fb[hb][b][j >> 1][2 * (j & 1) + 1], 1.0f);
                }
                const v8bf wide_a = fp8_widen8(fa[ha][i][j >> 1][2 * (j & 1)], fa[ha][i][j >> 1][2 * (j & 1) + 1], (float)(1 << kWideBy));
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    v4f& to = part_sum[at * 4 + b];
                    to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wide_b[b][j], wide_a, j ? to : v4f{}, 0, 0, 0);
                    asm volatile("" : "+v"(to));
                }
                auto add = [&](int pa, int ph, int row) {  // the sums of row block `row`, in half ph of the channels
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        v4f& to = acc[pa * NA + row][ph * 4 + b];
#pragma unroll
                        for (int r = 0; r < 4; ++r) to[r] = __fmaf_rn(part_sum[(row & 1) * 4 + b][r], both[row & 1], to[r]);
                        asm volatile("" : "+v"(to));
                    }
                };
                if (NA == 2 && j == 1 && q >= 4) {  // the row block before, its products done by now
                    const int before_q = q - 4;
                    add(ha, before_q < L ? decltype(HB)::value : 1 - decltype(HB)::value, before_q % L / 4);
                }
                if (j == 3 && (NA == 1 || q == 2 * L - 1)) add(ha, hb, i);
            } else if constexpr (F32S) {
                part_sum[q % kRing] = mfma<kByte>(whole(fb[hb][j]), whole(fa[ha][i]), v4f{}, sw[hb], sx[ha * NA + i]);
                asm volatile("" : "+v"(part_sum[q % kRing]));  // here: not where its value is first asked for
                // the product kLag before: of this half, of the step's first, or of the step before
                const int p = (q - kLag + 2 * L) % (2 * L), pa = q < kLag ? 1 - ha : ha;
                const int pb = q >= kLag ? (p < L ? decltype(HB)::value : 1 - decltype(HB)::value)
                                         : (ha ? decltype(HB)::value : 1 - decltype(HB)::value);
                const float s = q < kLag && ha == 0 ? before[pb] : ws[pb];
                v4f& to = acc[pa * NA + p % L / NB][pb * NB + p % NB];
#pragma unroll
                for (int r = 0; r < 4; ++r) to[r] = __fmaf_rn(part_sum[(q + kRing - kLag) % kRing][r], s, to[r]);
                asm volatile("" : "+v"(to));
            } else {
                acc[ha * NA + i][hb * NB + j] =
                    mfma<kByte>(whole(fb[hb][j]), whole(fa[ha][i]), acc[ha * NA + i][hb * NB + j], sw[hb], sx[ha * NA + i]);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (r < n1 && q == kAhead + r * kSpan1 / n1) read1(r);
                if (r < n2 && q == L + r * kSpan2 / n2) read2(r);
                if (r < kLoads && q == kAhead + r * (2 * L - kAhead) / kLoads) load(r);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    auto step = [&](auto S, int g) {
        constexpr int s = decltype(S)::value;
        using Buf = std::integral_constant<int, s & 1>;
        using Nxt = std::integral_constant<int, (s + 1) & 1>;
        using F = std::integral_constant<int, s & 1>;        // the half of the channels that comes first
        using O = std::integral_constant<int, (s + 1) & 1>;  // the other, the next step's first
        using ReadsA = std::integral_constant<int, 2 * NA>;
        using ReadsB = std::integral_constant<int, 2 * NB>;
        if constexpr (WIDE && !F32S) {
#pragma unroll
            for (int h = 0; h < 2; ++h) ws[h] = fp8_scale_value((uint32_t)sw[h] >> 8 * s & 255);
        }
        if constexpr (F32S) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                before[h] = ws[h];
                if constexpr (WIDE) {
                    ws[h] = next[s][h];
                } else {
                    ws[h] = ahead[h].f;
                    sw[h] = ahead[h].b << 8 * s;
                }
            }
            if constexpr (s == 1) fetch_f32(g + 1);
        }
        half(I0{}, F{}, S,
             [&](int q) {
                 if (s == 0 && q == 0) issue_scales(g + 2);
                 issue(Buf{}, I0{}, F{}, g + 2, q);
             },
             [&](int q) { read_b(Buf{}, O{}, q); }, ReadsB{}, [&](int q) { read_a(Buf{}, I1{}, q); }, ReadsA{});
        half(I1{}, O{}, S,
             [&](int q) {
                 if (F32S && !WIDE && q < 2) split_ahead(1 - s, q);  // of the next step, between products
                 issue(Buf{}, I1{}, O{}, g + 2, q);
             },
             [&](int q) { read_a(Nxt{}, I0{}, q); }, ReadsA{}, [&](int q) { read_b(Nxt{}, O{}, q); }, ReadsB{});
        if constexpr (s == 1) read_scales(g + 1);
    };
    // Two steps without a branch: the compiler tells the regions apart within a block only, and
    // waits for every load before a read where it cannot.  Behind an odd last group the second
    // multiplies that group again by scales of 2^-254: zeros.
    int g = 0;
    do {
        step(I0{}, g);
        step(I1{}, g + 1);
        g += 2;
    } while (g < G);
    wait_loads_and_sync<0>();  // the regions are no longer read or written
    if constexpr (F32S && !WIDE) {  // the last step's last products
#pragma unroll
        for (int p = NB * NA - kLag; p < NB * NA; ++p)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                v4f& to = acc[NA + p / NB][NB + p % NB];
                to[r] = __fmaf_rn(part_sum[(NB * NA + p) % kRing][r], ws[1], to[r]);
            }
    }

    // Lane l's accumulators: weight rows 4 (l / 16) + r of block j, activation row l % 16 of block
    // i: four neighbouring outputs of a row.
    const int el = (int)__builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    const int row0 = el & 15, quad = el >> 4;
    const int rbase = wm * 32 * NA;
    if constexpr (EPI == kDense) {
        // Two blocks' quads are swapped between neighbouring rows of 16 lanes, so that a lane has eight outputs of one
        // block, 64 bytes of a row together.
        uint16_t* y = static_cast<uint16_t*>(a.y);
        const bool vec = (reinterpret_cast<uintptr_t>(y) & 15) == 0 && a.ldy % 8 == 0;
        const int nl = 16 * (quad & 1) + 8 * (quad >> 1);  // within the two blocks
#pragma unroll
        for (int j = 0; j < 2 * NB; j += 2) {
            const int n = n0 + wn * 32 * NB + 16 * j + nl;
            const v4f b0 = *reinterpret_cast<const v4f*>(s_aux + wn * 32 * NB + 16 * j + 4 * quad);
            const v4f b1 = *reinterpret_cast<const v4f*>(s_aux + wn * 32 * NB + 16 * (j + 1) + 4 * quad);
#pragma unroll
            for (int i = 0; i < 2 * NA; ++i) {
                const v4f v0 = acc[i][j], v1 = acc[i][j + 1];
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const auto s = __builtin_amdgcn_permlane16_swap(
                        f32x2_to_16<OUT>(__fadd_rn(v0[2 * e], b0[2 * e]), __fadd_rn(v0[2 * e + 1], b0[2 * e + 1])),
                        f32x2_to_16<OUT>(__fadd_rn(v1[2 * e], b1[2 * e]), __fadd_rn(v1[2 * e + 1], b1[2 * e + 1])), false, false);
                    w[e] = s[0];
                    w[2 + e] = s[1];
                }
                const int m = m0 + rbase + 16 * i + row0;
                if (m >= a.M || n >= a.N) continue;
                uint16_t* dst = y + (int64_t)m * a.ldy + n;
                if (vec && n + 8 <= a.N) {
                    *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    for (int e = 0; e < 8 && n + e < a.N; ++e) dst[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                }
            }
        }
    } else if constexpr (EPI == kGateUp) {
        uint32_t* const tops = sc;  // [2][256]
#pragma unroll
        for (int i = 0; i < 2 * NA; ++i) {
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool there = n0 + wn * 64 + 16 * j < a.N;  // a multiple of 16
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    acc[i][j][r] = there ? fp8_silu_mul(acc[i][j][r], acc[i][j + 4][r]) : 0.0f;
                    most = larger(most, acc[i][j][r]);
                }
            }
            uint32_t top = magnitude(most);
            top = max(top, (uint32_t)__shfl_xor((int)top, 16));
            top = max(top, (uint32_t)__shfl_xor((int)top, 32));
            tops[wn * 256 + rbase + 16 * i + row0] = top;
        }
        __syncthreads();
        // the codes as the packed blocks that they are in memory, a wavefront row's in one region
        uint8_t* const image = wm ? A01 : A00;
#pragma unroll
        for (int i = 0; i < 2 * NA; ++i) {
            const int row = rbase + 16 * i + row0;
            const uint32_t b = fp8_scale_byte(max(tops[row], tops[256 + row]));
            const float inv = fp8_inverse(b);
            if (wn == 0 && el < 16 && row < (t.rows + 15) / 16 * 16)
                a.hs[(int64_t)(m0 + row) * a.h_pitch + tn] = (uint8_t)b;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * inv;  // (whatever a group with a NaN scale holds is NaN)
                *reinterpret_cast<uint32_t*>(image + i * kGroupBytes + wn * kWBlock + fp8_pos(row0, j) + 4 * quad) =
                    fp8_pack4(v[0], v[1], v[2], v[3]);
            }
        }
        __syncthreads();
        const int blocks = (t.rows + 15) / 16;
        for (int c = tid; c < blocks * (kGroupBytes / 16); c += 256) {
            const int b = c >> 7;
            const uint8_t* src = (b < 2 * NA ? A00 : A01) + (b % (2 * NA)) * kGroupBytes + (c & 127) * 16;
            *reinterpret_cast<uint4*>(a.h + ((int64_t)(t.block + b) * tiles_n + tn) * kGroupBytes + (c & 127) * 16) =
                *reinterpret_cast<const uint4*>(src);
        }
    } else {
        float* y = static_cast<float*>(a.y);
#pragma unroll
        for (int i = 0; i < 2 * NA; ++i) {
            const int row = rbase + 16 * i + row0, flat = s_flat[row];
            const float w = s_aux[row];
            if (flat < 0) continue;
            float* const to = y + (int64_t)flat * a.ldy + n0 + wn * 32 * NB + 4 * quad;
#pragma unroll
            for (int j = 0; j < 2 * NB; ++j) {
                v4f v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = __fmul_rn(acc[i][j][e], w);
                if (n0 + wn * 32 * NB + 16 * j < a.N) *reinterpret_cast<v4f*>(to + 16 * j) = v;
            }
        }
    }
}

}  // namespace

}  // namespace pdq

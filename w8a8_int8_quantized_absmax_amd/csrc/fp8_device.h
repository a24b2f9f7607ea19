// Device-side helpers of the 8-bit floating-point products (gfx950): codes are
// e4m3 values (OCP: 448 the largest, no infinity), scales of activation groups
// powers of two in the e8m0 format (byte b stands for 2^(b - 127), 255 for NaN).
#pragma once

#include "pdq_device.h"
#include "pdq_kernels.h"

namespace pdq {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// K values of one scale: of a row's group and, with as many rows, of a weight's block.
constexpr int kGroup = 128;

// The packed operand: blocks of 16 rows x 64 K values as the INT8 one's (pdq_device.h), two blocks
// that follow each other for a group: 2 KB, one fragment of a 16x16x128 product.  Within a block
// the 16-byte chunks go by chunk, then row, so that lane l's, row l % 16 and chunk l / 16, is the
// l-th: 1 KB by 64 lanes in order, from memory as from LDS, free of bank conflicts.  (In the
// INT8 order, rows of 64 bytes with their chunks turned, these reads count as many conflict
// clocks as clocks.)
__host__ __device__ __forceinline__ int fp8_pos(int r, int c) { return c * 256 + r * 16; }
constexpr int kGroupBytes = 2 * kWBlock;
__host__ __device__ __forceinline__ int64_t fp8_groups(int64_t K) { return (K + kGroup - 1) / kGroup; }
// Groups in a row of scales: a multiple of 4, so that four scales are one aligned load.
__host__ __device__ __forceinline__ int64_t fp8_scale_pitch(int64_t K) { return (fp8_groups(K) + 3) / 4 * 4; }

// The e8m0 byte of a group whose largest magnitude has the bits `top` (the
// maximum of the magnitudes' bits, so that infinities and NaN win): the smallest
// power of two S with |x| <= 448 S.  448 = 1.75 * 2^8, so that S = 2^(E - 8), E
// the magnitude's exponent, or twice that if its mantissa is above 1.75;
// 2^-127, the format's smallest, where that is below it; 1 for zeros.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t top) {
    const int e = (int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    const uint32_t b = (uint32_t)max(e, 0);
    return top == 0 ? 127u : top >= 0x7f800000u ? 255u : b;
}

// 1 / S as binary32, exact: 2^(127 - b) for b <= 247 (E <= 254 above); 0 for NaN,
// whose codes are zeros.
__device__ __forceinline__ float fp8_inverse(uint32_t b) { return b == 255u ? 0.0f : __uint_as_float((254u - b) << 23); }

// Four codes, rounded to nearest even (v_cvt_pk_fp8_f32; |v| <= 448).
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    return (uint32_t)r;
}

// Maximum over the 16 lanes of a row of lanes, by lane permutations.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xf, 0xf, false);
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, dpp_u32<0xB1>(v));   // quad_perm [1, 0, 3, 2]
    v = max(v, dpp_u32<0x4E>(v));   // quad_perm [2, 3, 0, 1]
    v = max(v, dpp_u32<0x141>(v));  // row_half_mirror
    return max(v, dpp_u32<0x140>(v));  // row_mirror
}

// The larger magnitude, NaN if one is.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(fabsf(a), fabsf(b)); }
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The bits of the largest magnitude of eight values (maxima of three that keep a NaN: four instructions), and their
// codes at scale byte b.
__device__ __forceinline__ uint32_t fp8_top8(const float (&v)[8]) {
    float m = larger(v[0], v[1]);
#pragma unroll
    for (int j = 2; j < 8; ++j) m = larger(m, v[j]);
    return magnitude(m);
}
__device__ __forceinline__ uint2 fp8_code8(const float (&v)[8], uint32_t b) {
    const float inv = fp8_inverse(b);
    const uint2 c = make_uint2(fp8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                               fp8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    return b == 255u ? make_uint2(0, 0) : c;  // (infinities and NaN times 0 are not 0)
}

// A lane's 32 bytes of a fragment of 16 rows x 128 K values: row lane % 16, the
// chunk lane / 16 of each of the two blocks.  The order of K values within a
// group is the same for both operands of a product, so that any will do.
__device__ __forceinline__ v8i fp8_fragment(const uint8_t* group, int lane) {
    const uint8_t* p = group + 16 * lane;
    const v4i lo = *reinterpret_cast<const v4i*>(p);
    const v4i hi = *reinterpret_cast<const v4i*>(p + kWBlock);
    return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// c += 2^(sw - 127) 2^(sx - 127) W X^T for fragments of 16 weight rows and 16
// activation rows: lane l's scale byte is its own row's (l % 16); all 128
// products of an output share a scale.  Output r of lane l: weight row
// 4 (l / 16) + r, activation row l % 16.
__device__ __forceinline__ v4f fp8_mfma16(v8i w, v8i x, v4f c, int sw, int sx) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, 0, 0, 0, sw, 0, sx);
}

// The same product on 16-bit operands, with every product whole and the sum binary32: the codes are
// widened (exactly, v_cvt_scalef32_pk_bf16_fp8), the activation's by its scale, and the weight's multiplies the sum.  The FP8
// products align eight products to the largest of their exponents and keep 13 bits behind it, some 2^-16
// of a sum; this one is off by some 2^-25.  At half the rate (16 x 16 x 32 in 16 clocks, for 16 x 16 x 128 in 32), and the codes are
// widened by the vector unit: where reading the weight is what takes the time.
struct Fp8Wide {
    v8bf v[4];
};
__device__ __forceinline__ v8bf fp8_widen8(unsigned a, unsigned b, float by) {  // by: a power of two
    v8bf w;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const auto lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(j ? b : a, by, false);
        const auto hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(j ? b : a, by, true);
        w[4 * j] = lo[0];
        w[4 * j + 1] = lo[1];
        w[4 * j + 2] = hi[0];
        w[4 * j + 3] = hi[1];
    }
    return w;
}
__device__ __forceinline__ Fp8Wide fp8_widen(v8i f, float by) {
    Fp8Wide w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w.v[i] = fp8_widen8((unsigned)f[2 * i], (unsigned)f[2 * i + 1], by);
    return w;
}
__device__ __forceinline__ v4f fp8_mfma16_wide(const Fp8Wide& w, const Fp8Wide& x) {
    v4f c = v4f{};
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.v[i], x.v[i], c, 0, 0, 0);
    return c;
}

// A binary32 scale as a power of two in the e8m0 format, an operand of the matrix instruction, and the factor that is left, 1 to
// 2 (less for scales below 2^-126): S_x times a sum of codes alone may pass 2^128 where the result does not.  Exact for
// every value; infinities and NaN stay in the factor, and so does 0.
struct Fp8Split {
    float f;
    int b;
};
__device__ __forceinline__ Fp8Split fp8_split(float s) {
    const int e = (int)(__float_as_uint(s) >> 23 & 255u), b = e == 255 ? 127 : e;
    return Fp8Split{__builtin_ldexpf(s, 127 - b), b};
}

// What an e8m0 byte stands for.
__device__ __forceinline__ float fp8_scale_value(uint32_t b) {
    return __uint_as_float(b == 255u ? 0x7fc00000u : b == 0u ? 0x00400000u : b << 23);
}

// An activation's scale as what its codes are widened by, 2^-100 to 2^100, and what is left, which multiplies the weight's: as one
// factor of the sum both might pass 2^128 where that is 0 (there: from S_w = 2^108 on, under an S_x beyond 2^100).
struct Fp8By {
    float by, rest;
};
__device__ __forceinline__ Fp8By fp8_by(uint32_t b) {
    const uint32_t e = min(max(b, 27u), 227u);
    return Fp8By{__uint_as_float(e << 23), __uint_as_float(b == 255u ? 0x7fc00000u : (b + 127u - e) << 23)};
}

// A few rows' codes and scales, by the whole workgroup into LDS: rows of `pitch` bytes (K padded to whole
// groups, and 16 bytes so that 16 rows' chunks lie in different banks), and a scale byte a group.
template <int DT>
__device__ __forceinline__ void fp8_code_rows(const void* x, int64_t ldx, int rows, int K, uint8_t* codes, uint8_t* scales,
                                              int pitch) {
    const int groups = (int)fp8_groups(K), c8 = threadIdx.x & 15, pieces = rows * groups, each = blockDim.x >> 4;
    constexpr int U = 4;  // loads sent together
    for (int p0 = threadIdx.x >> 4; p0 < (pieces + each - 1) / each * each; p0 += U * each) {  // a row's group by 16 lanes
        Raw8<DT> raw[U];
        int m[U], g[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = p0 + u * each;
            m[u] = min(p / groups, rows - 1);
            g[u] = p - p / groups * groups;
            const int k = g[u] * kGroup + c8 * 8;
            raw[u] = p < pieces && k < K ? load_raw8<DT>(static_cast<const char*>(x) + m[u] * ldx * Elem<DT>::bytes, k / 8)
                                         : zero_raw8<DT>();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (p0 + u * each >= pieces) break;  // (the same in the 16 lanes)
            float v[8];
            widen8<DT>(raw[u], v);
            const uint32_t b = fp8_scale_byte(row16_max(fp8_top8(v)));
            *reinterpret_cast<uint2*>(codes + m[u] * pitch + g[u] * kGroup + c8 * 8) = fp8_code8(v, b);
            if (c8 == 0) scales[m[u] * groups + g[u]] = (uint8_t)b;
        }
    }
}

// A lane's fragment of a row coded there: any row, the chunk lane / 16 of each half of the group.
__device__ __forceinline__ v8i fp8_row_fragment(const uint8_t* row, int g, int lane) {
    const uint8_t* p = row + g * kGroup + (lane >> 4) * 16;
    const v4i lo = *reinterpret_cast<const v4i*>(p);
    const v4i hi = *reinterpret_cast<const v4i*>(p + kGroup / 2);
    return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}

// A product's result, for every lane, here: the compiler may otherwise move the
// instruction into a branch that only some lanes take, and with it the writes of
// its scale operands, which the lanes outside then lack.
__device__ __forceinline__ void fp8_settle(v4f& v) { asm volatile("" : "+v"(v)); }

// A tile of kRows sorted rows, all of one expert: the `index`-th of all, in the
// order of the experts.
struct Fp8Tile {
    int expert;  // -1: there is no such tile
    int first;   // its first sorted row
    int rows;    // 1 .. kRows
    int block;   // its first block of 16 rows
};

// Expert e's sorted rows.  What the offsets hold cannot be checked on the host: they are clamped to
// rows that are there, and where they do not ascend there are no tiles (from that run of 64 experts
// on), so that all tiles together never hold more rows, or blocks, than there are.
struct Fp8Span {
    int lo, count;
    bool descends;
};
__device__ __forceinline__ Fp8Span fp8_span(const Fp8Sorted& s, int e) {  // e at most s.experts
    const int lo = min(max(s.offsets[e], 0), s.total);
    const int hi = min(max(s.offsets[min(e + 1, s.experts)], 0), s.total);
    return Fp8Span{lo, hi - lo, hi < lo};
}

// Every lane of the wavefront takes part and gets the same answer.
template <int kRows>
__device__ __forceinline__ Fp8Tile fp8_tile(const Fp8Sorted& s, int index, int lane) {
    int tiles0 = 0, blocks0 = 0;
    for (int e0 = 0; e0 < s.experts; e0 += 64) {
        const Fp8Span span = fp8_span(s, min(e0 + lane, s.experts));
        if (__ballot(span.descends)) break;
        const int lo = span.lo, count = span.count, blocks = (count + 15) / 16, tiles = (count + kRows - 1) / kRows;
        int bsum = blocks, tsum = tiles;  // inclusive sums over the lanes
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int b = __shfl_up(bsum, d), t = kRows == 16 ? 0 : __shfl_up(tsum, d);
            if (lane >= d) {
                bsum += b;
                tsum += t;
            }
        }
        if (kRows == 16) tsum = bsum;
        const uint64_t past = __ballot(tiles0 + tsum > index);
        if (past) {
            const int l = __builtin_ctzll(past);
            const int at = index - tiles0 - (__builtin_amdgcn_readlane(tsum, l) - __builtin_amdgcn_readlane(tiles, l));
            const int n = __builtin_amdgcn_readlane(count, l);
            return Fp8Tile{e0 + l, __builtin_amdgcn_readlane(lo, l) + at * kRows, min(n - at * kRows, kRows),
                           blocks0 + __builtin_amdgcn_readlane(bsum, l) - __builtin_amdgcn_readlane(blocks, l) +
                               at * (kRows / 16)};
        }
        tiles0 += __builtin_amdgcn_readlane(tsum, 63);
        blocks0 += __builtin_amdgcn_readlane(bsum, 63);
    }
    return Fp8Tile{-1, 0, 0, 0};
}

// How many tiles of kRows sorted rows there are; none if the offsets descend anywhere.
template <int kRows>
__device__ __forceinline__ int fp8_tiles(const Fp8Sorted& s, int lane) {
    int n = 0;
    for (int e0 = 0; e0 < s.experts; e0 += 64) {
        const Fp8Span span = fp8_span(s, min(e0 + lane, s.experts));
        if (__ballot(span.descends)) return 0;
        n += (span.count + kRows - 1) / kRows;
    }
    return __builtin_amdgcn_readfirstlane(wave_sum(n));
}

// silu(g) * u = g u / (1 + e), e = 2^(-g log2 e), by the hardware's exp2 and reciprocal (where e is beyond 2^126 or
// infinite, 0).  Off by (1.3 |g| + 7) 2^-24 of it: the constant and its product 1.22 |g|, exp2 and the reciprocal a unit each, 2, the
// sum and two products 1 each.
__device__ __forceinline__ float fp8_silu_mul(float g, float u) {
    const float e = __builtin_amdgcn_exp2f(g * -1.4426950408889634f);
    return g * __builtin_amdgcn_rcpf(1.0f + e) * u;
}

// The token and slot of row r of a tile, -1 where there is none (or the entry is not a row of the call).
__device__ __forceinline__ int fp8_sorted_row(const Fp8Sorted& s, const Fp8Tile& t, int r) {
    if (t.expert < 0 || r >= t.rows) return -1;
    const int flat = s.rows[t.first + r];
    return (uint32_t)flat < (uint32_t)s.total ? flat : -1;
}

}  // namespace pdq

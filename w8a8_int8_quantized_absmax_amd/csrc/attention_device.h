// What the attention kernels over the INT8 key/value cache share.
//
// Both take K codes and V codes as binary16 matrix operands (integers up to 127
// are exact there) and leave the scales outside the products: a score is
// (q . codes) * S_k, and the value scale goes into the weight's exponent,
//   p = 2^(z log2 e + log2 S_v - M),   O = sum p * codes,   l = sum p / S_v,
// so that a weight, rounded to binary16 for the value product, keeps its 11 bits
// whatever the scales are, and a page's scale costs one addition a score.
//
// M is an integer, kLift below the largest exponent where it was set, and moved
// only when weights pass 2^(kLift + kSlack), by the row itself, whatever the other
// rows do: moving it multiplies what is accumulated by a power of two, exactly,
// and most tiles need no maximum across lanes.  A weight under 2^-14 (2^-19 of the
// largest when M was set) is subnormal in binary16: off by 2^-25 at most.
#pragma once

#include "kv_device.h"

namespace pdq {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v4h __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLift = 5.0f, kSlack = 8.0f;  // weights stay below 2^13
constexpr float kNone = -3e38f;               // M before the first visible key

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Four codes as binary16: the byte b ^ 0x80 under the exponent byte 0x64 is
// 1024 + 128 + code, exactly; subtracting 1152 is exact too.
__device__ __forceinline__ v4h codes4(uint32_t w) {
    w ^= 0x80808080u;
    const v2h lo = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, 0x04010400u));
    const v2h hi = __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, w, 0x04030402u));
    const v2h off = {(_Float16)1152.0f, (_Float16)1152.0f};
    const v2h a = lo - off, b = hi - off;
    return __builtin_shufflevector(a, b, 0, 1, 2, 3);
}

__device__ __forceinline__ v8h join(v4h a, v4h b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// The score (q . codes) * f, capped or not, in units of log2: cap2 = softcap *
// log2 e, and f = scale * S_k * log2 e without a cap, 2 log2 e * scale * S_k /
// softcap with one: tanh(x) = 1 - 2 / (2^(2 x log2 e) + 1), exact at both ends,
// off by an ulp of 1 between.
__device__ __forceinline__ float capped(float x2, float cap2) {
    const float r = __builtin_amdgcn_rcpf(exp2_(x2) + 1.0f);
    return cap2 * (1.0f - 2.0f * r);
}

// A row of bfloat16 queries with the largest magnitude `top` becomes binary16 times
// 2^(14 - e): the largest lies in [2^13, 2^14), and what binary16 rounds away is at most
// 2^-25, 2^-38 of it.  A row below 2^-96 takes 2^109, which makes every bfloat16 number,
// a multiple of 2^-133, one of binary16's, exactly: its factor scale * 2^(e - 14) stays
// among binary32's normal numbers (from a scale of 2^-17 on), whatever page scales follow.
__device__ __forceinline__ int row_exponent(float top) {
    return top > 0.0f && top < INFINITY ? max(__builtin_amdgcn_frexp_expf(top), -95) : 14;
}

// A sequence's rows and keys as a tile of R rows takes them: rows are (token,
// query head of the group), the keys seen by any of its rows k0 .. last.
struct AttnSeq {
    KvSeq q;
    int len;       // min(length, what the table can name); 0 without a pool
    int prefix;    // keys that every row sees (0: none)
    int k0, last;  // keys that some row sees (last < k0: none)
};

template <bool Uniform = false>
__device__ __forceinline__ AttnSeq attn_seq(const AttentionArgs& a, int s) {
    AttnSeq r;
    r.q = kv_seq<Uniform>(a.b, s);
    r.len = a.c.pages > 0 ? min(r.q.len, a.b.max_pages * a.c.page) : 0;
    r.prefix = a.prefix ? max(load_as<Uniform>(a.prefix + s), 0) : 0;
    r.k0 = a.window ? (int)max((int64_t)r.q.p0 - a.window + 1, (int64_t)0) : 0;
    r.last = min(max(r.q.p0 + r.q.n, r.prefix), r.len) - 1;
    return r;
}

// The keys lo .. hi that a row at position pos sees.
__device__ __forceinline__ void row_keys(const AttentionArgs& a, const AttnSeq& s, int pos, int& lo, int& hi) {
    lo = a.window ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
    hi = min(max(pos + 1, s.prefix), s.len) - 1;
}

// attention_prompt.hip: many rows for each sequence.  splits: parts of the keys,
// joined through the workspace ([splits, tokens, hq, dim + 2] floats) beyond one.
int attention_prompt_most_splits(int64_t tokens, int64_t batch, int hq, int hkv, int dim);
int attention_prompt_splits(int64_t tokens, int64_t batch, int hq, int hkv, int dim, int64_t keys);
int64_t attention_prompt_threads(const AttentionArgs& a, int splits);
void launch_attention_prompt(const AttentionArgs& a, int dt, int splits, hipStream_t st);

}  // namespace pdq

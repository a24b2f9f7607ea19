// The C entry points of libpdq: host-side argument checks, then the kernel
// launches of each operation on the caller's stream.  Declared and
// documented in include/pdq.h.

#include <math.h>

#include <algorithm>
#include <mutex>

#include "pdq.h"
#include "fp8_device.h"
#include "pdq_device.h"
#include "pdq_kernels.h"

using namespace pdq;

#define PDQ_TRY(expr)                         \
    do {                                      \
        const pdq_status s_ = (expr);         \
        if (s_ != PDQ_OK) return s_;          \
    } while (0)


namespace {

constexpr int64_t kMaxK = 65536;        // |sum_k (q_x - Z) q_w| < 255 * 127 * K stays in int32
// Rows of any operand (M activation rows, N weight rows = output channels).
// Together with the two products below this keeps every launch grid inside
// the dispatch limits with room to spare: the skinny GEMM's second grid
// dimension is rows / 64, the per-token quantizers run 256 threads per row,
// the static quantizer one thread per 8 values, the tiled GEMM 256 threads
// per 256 x 256 output tile.
constexpr int64_t kMaxRows = int64_t(1) << 21;
constexpr int64_t kMaxValues = int64_t(1) << 34;   // M x K of one operand
constexpr int64_t kMaxOutputs = int64_t(1) << 39;  // M x N of one product
// Which kernel runs an M x N INT8 GEMM, whichever quantization scheme
// produced the codes: the skinny (weight-streaming) kernel of decode.hip or
// the 256 x 256-tile GEMM.  The skinny kernel's work is ceil(N / 16) x
// ceil(M / 64) units, each one pass over the K tiles of 16 weight channels
// for up to 64 activation rows, and costs about 4 us plus 4.7 us per 256 of
// them with 16 channels per workgroup, 3.6 us with more; the tiled GEMM costs
// about 52 us per round of 256 tiles, however few tiles the round holds (all
// measured on MI355X at K = 4096; K scales both alike).  Up to 64 rows the
// skinny kernel always runs.
bool skinny_gemm(int64_t M, int64_t N) {
    if (M <= 64) return true;
    const double units = (double)((N + 15) / 16) * (double)((M + 63) / 64);
    const double tiles = (double)((M + 255) / 256) * (double)((N + 255) / 256);
    const double per256 = decode_groups(M, N) > 1 ? 3.6 : 4.7;
    return 4.0 + per256 * units / 256.0 < 52.0 * ceil(tiles / 256.0);
}

int elem_bytes(int dt) { return dt == PDQ_F32 ? 4 : 2; }
bool dtype_ok(int dt) { return dt == PDQ_F32 || dt == PDQ_BF16 || dt == PDQ_F16; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Shape rules shared by every K-wide operand.  K == 0 is refused: the kernels
// read at least one 16-value chunk of every row they touch.
pdq_status check_mk(int64_t M, int64_t K, int64_t ld) {
    if (M < 0 || K <= 0 || M > kMaxRows || K > kMaxK || K % 16 != 0) return PDQ_ERR_SHAPE;
    if (M * K > kMaxValues) return PDQ_ERR_SHAPE;
    if (ld < K || ld < 0) return PDQ_ERR_SHAPE;
    return PDQ_OK;
}

// A [rows, K] operand with `ebytes`-byte elements and row pitch `ld`.
pdq_status check_operand(const void* p, int ebytes, int64_t rows, int64_t K, int64_t ld) {
    pdq_status s = check_mk(rows, K, ld);
    if (s != PDQ_OK) return s;
    if (rows > 0 && K > 0 && !p) return PDQ_ERR_NULL;
    if (!aligned(p, 16) || (ld * ebytes) % 16 != 0) return PDQ_ERR_ALIGN;
    return PDQ_OK;
}

pdq_status launched() { return hipGetLastError() == hipSuccess ? PDQ_OK : PDQ_ERR_HIP; }

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

int64_t side_pitch(int64_t max_out) { return (max_out + 15) / 16 * 16; }

}  // namespace

// Scratch of pdq_linear_int8_outlier_noalloc: one copy per device, held until
// the process ends.  Host code never passes `scratch` itself to a kernel (on
// the host it names a stand-in, not device memory): the device address comes
// from hipGetSymbolAddress, looked up once per device with that device current
// and kept in scratch_ptr[device].
namespace {

constexpr size_t kScratchBytes = size_t(8) << 20;
static __device__ __align__(256) uint8_t scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex scratch_mu;
char* scratch_ptr[kMaxDevices] = {};

// The scratch address on the device of `st` (the current device: a stream of
// another device is refused).
pdq_status scratch_for_stream(hipStream_t st, char** out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return PDQ_ERR_HIP;
    if (st) {
        int sdev = -1;
        if (hipStreamGetDevice(st, &sdev) != hipSuccess) return PDQ_ERR_HIP;
        if (sdev != dev) return PDQ_ERR_UNSUPPORTED;
    }
    std::lock_guard<std::mutex> lock(scratch_mu);
    if (!scratch_ptr[dev]) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return PDQ_ERR_HIP;
        scratch_ptr[dev] = static_cast<char*>(p);
    }
    *out = scratch_ptr[dev];
    return PDQ_OK;
}

// Host-side checks of the LLM.int8 call, shared by both of its entry points
// (no HIP call).
pdq_status check_int8_outlier(const void* x, pdq_dtype dt, int64_t M, int64_t K, int64_t ldx, float threshold,
                              const int8_t* wq, const float* w_scale, const void* w16, int64_t ldw,
                              const float* bias, int64_t N, void* y, int64_t ldy, int8_t* xq, float* x_scale,
                              int32_t* outlier_idx, int32_t* n_outlier, int64_t max_outliers, int32_t* acc_out) {
    if (dt != PDQ_F16 && dt != PDQ_BF16) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(dt), M, K, ldx));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N || ldw < K) return PDQ_ERR_SHAPE;
    if (max_outliers < 0 || max_outliers > K) return PDQ_ERR_SHAPE;
    if (isnan(threshold)) return PDQ_ERR_UNSUPPORTED;
    if (!n_outlier || (max_outliers > 0 && !outlier_idx)) return PDQ_ERR_NULL;
    if (N > 0 && (!w_scale || (K > 0 && !w16))) return PDQ_ERR_NULL;
    if (M > 0 && ((K > 0 && !xq) || !x_scale)) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
        !aligned(y, 2) || !aligned(w16, 2) || !aligned(acc_out, 4) || !aligned(outlier_idx, 4) ||
        !aligned(n_outlier, 4))
        return PDQ_ERR_ALIGN;
    return PDQ_OK;
}

// The launches of the LLM.int8 call on a workspace of at least
// pdq_linear_int8_outlier_workspace(M, N, K, max_outliers) bytes, 256-byte
// aligned: predicates per row block -> mask, index list, count and the W
// gather -> INT8 codes of the regular columns with the X gather -> INT8 GEMM
// with the 16-bit side product in its epilogue.  Every byte of the workspace
// that is read is first written by the same call.
void run_int8_outlier(const void* x, pdq_dtype dt, int64_t M, int64_t K, int64_t ldx, float threshold,
                      const int8_t* wq, const float* w_scale, const void* w16, int64_t ldw, const float* bias,
                      int64_t N, void* y, int64_t ldy, int8_t* xq, float* x_scale, int32_t* outlier_idx,
                      int32_t* n_outlier, int64_t max_outliers, char* ws, int32_t* acc_out, hipStream_t st) {
    const int64_t P = side_pitch(max_outliers);
    const size_t pitch = (size_t)outlier_partial_pitch(K);
    uint8_t* partial = reinterpret_cast<uint8_t*>(ws);
    ws += align256((size_t)outlier_row_blocks(M) * pitch);
    uint8_t* mask = reinterpret_cast<uint8_t*>(ws);
    ws += align256(pitch);
    uint16_t* xo = reinterpret_cast<uint16_t*>(ws);
    ws += align256((size_t)(M * P * 2));
    uint16_t* wo = reinterpret_cast<uint16_t*>(ws);

    launch_outlier_partial(x, dt, M, K, ldx, threshold, partial, st);
    launch_outlier_index(partial, M, K, mask, outlier_idx, n_outlier, max_outliers, st);
    if (M > 0) {
        // the regular-column quantizer; extra workgroups of its launch gather
        // W_out (at most 256 of them)
        OutlierSkip skip{};
        skip.mask = mask;
        skip.idx = outlier_idx;
        skip.count = n_outlier;
        skip.max_out = (int)max_outliers;
        skip.xo = xo;
        skip.P = (int)P;
        skip.w16 = static_cast<const uint16_t*>(w16);
        skip.ldw = ldw;
        skip.N = N;
        skip.wo = wo;
        skip.wrows = (int)std::max<int64_t>(64, (N + 255) / 256);
        launch_quant_rows(x, dt, M, K, ldx, xq, x_scale, nullptr, &skip, st);
    }
    GemmArgs g{};
    g.A = xq;
    g.B = wq;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.sa = x_scale;
    g.sb = w_scale;
    g.bias = bias;
    g.y = y;
    g.ldy = ldy;
    g.acc_out = acc_out;
    g.xo = xo;
    g.wo = wo;
    g.P = (int)P;
    g.count = n_outlier;
    g.max_count = (int)max_outliers;
    launch_gemm_i8(g, dt, true, st);
}

}  // namespace

extern "C" {

const char* pdq_status_string(pdq_status s) {
    switch (s) {
        case PDQ_OK: return "ok";
        case PDQ_ERR_NULL: return "required pointer is NULL";
        case PDQ_ERR_SHAPE:
            return "invalid shape (negative or too large size, K not a positive multiple of 16 up to 65536, or ld "
                   "too small)";
        case PDQ_ERR_DTYPE: return "dtype not accepted by this entry point";
        case PDQ_ERR_ALIGN: return "pointer or row pitch not 16-byte aligned";
        case PDQ_ERR_UNSUPPORTED: return "argument value out of range";
        case PDQ_ERR_WORKSPACE: return "workspace missing or too small";
        case PDQ_ERR_HIP: return "HIP launch error";
        default: return "unknown status";  // any other value, the range sentinels included
    }
}

size_t pdq_weight_bytes(int64_t N, int64_t K) {
    if (N < 0 || K < 0) return 0;
    return (size_t)((N + kWGroup - 1) / kWGroup) * (size_t)((K + kWTileK - 1) / kWTileK) * kWBlock;
}

size_t pdq_act_bytes(int64_t M, int64_t K) { return pdq_weight_bytes(M, K); }

int pdq_gemm_kernel(int64_t M, int64_t N) {
    if (M < 1 || N < 1) return -1;
    return skinny_gemm(M, N) ? PDQ_GEMM_SKINNY : PDQ_GEMM_TILED;
}

int pdq_skinny_channels(int64_t M, int64_t N) {
    if (M < 1 || N < 1 || M > kMaxRows || N > kMaxRows) return -1;
    return 16 * decode_groups(M, N);
}

pdq_status pdq_pack_int8(const int8_t* src, int64_t rows, int64_t K, int64_t ld, int8_t* packed, void* stream) {
    PDQ_TRY(check_operand(src, 1, rows, K, ld));
    if (rows > 0 && !packed) return PDQ_ERR_NULL;
    if (!aligned(packed, 16)) return PDQ_ERR_ALIGN;
    if (rows == 0) return PDQ_OK;
    launch_pack_int8(src, rows, K, ld, packed, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_unpack_int8(const int8_t* packed, int64_t rows, int64_t K, int8_t* dst, int64_t ld, void* stream) {
    PDQ_TRY(check_operand(dst, 1, rows, K, ld));
    if (rows > 0 && !packed) return PDQ_ERR_NULL;
    if (!aligned(packed, 16)) return PDQ_ERR_ALIGN;
    if (rows == 0) return PDQ_OK;
    launch_unpack_int8(packed, rows, K, dst, ld, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_quantize_weight(const void* w, pdq_dtype w_dt, int64_t N, int64_t K, int64_t ldw,
                               int8_t* wq, float* w_scale, int32_t* w_colsum, void* stream) {
    if (!dtype_ok(w_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(w, elem_bytes(w_dt), N, K, ldw));
    if (N > 0 && ((K > 0 && !wq) || !w_scale)) return PDQ_ERR_NULL;
    if (!aligned(wq, 16) || !aligned(w_scale, 4) || !aligned(w_colsum, 4)) return PDQ_ERR_ALIGN;
    if (N == 0) return PDQ_OK;
    launch_quant_rows(w, w_dt, N, K, ldw, wq, w_scale, w_colsum, nullptr, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_calibrate_static(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                float* minmax, float* a_scale, int32_t* a_zp, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (!minmax) return PDQ_ERR_NULL;
    if ((a_scale == nullptr) != (a_zp == nullptr)) return PDQ_ERR_NULL;
    if (!aligned(minmax, 4) || !aligned(a_scale, 4) || !aligned(a_zp, 4)) return PDQ_ERR_ALIGN;
    hipStream_t st = static_cast<hipStream_t>(stream);
    launch_minmax(x, x_dt, M, K, ldx, minmax, st);
    if (a_scale) launch_minmax_finalize(minmax, a_scale, a_zp, st);
    return launched();
}

pdq_status pdq_quantize_per_token(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                  int8_t* xq, float* x_scale, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (M > 0 && ((K > 0 && !xq) || !x_scale)) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4)) return PDQ_ERR_ALIGN;
    if (M == 0) return PDQ_OK;
    launch_quant_rows(x, x_dt, M, K, ldx, xq, x_scale, nullptr, nullptr, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_gemm_per_token(const int8_t* xq, const float* x_scale, int64_t M, int64_t K,
                              const int8_t* wq, const float* w_scale, const float* bias, int64_t N,
                              uint16_t* y, int64_t ldy, int32_t* acc_out, void* stream) {
    PDQ_TRY(check_operand(xq, 1, M, K, K));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (N > 0 && !w_scale) return PDQ_ERR_NULL;
    if (M > 0 && !x_scale) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) || !aligned(y, 2) ||
        !aligned(acc_out, 4))
        return PDQ_ERR_ALIGN;
    if (M == 0 || N == 0) return PDQ_OK;
    if (skinny_gemm(M, N)) {
        DecodeArgs d{};
        d.xq = xq;
        d.wq = wq;
        d.M = (int)M;
        d.N = (int)N;
        d.K = (int)K;
        d.sa = x_scale;
        d.sw = w_scale;
        d.bias = bias;
        d.y = y;
        d.ldy = ldy;
        d.acc_out = acc_out;
        launch_decode_gemv(d, static_cast<hipStream_t>(stream));
        return launched();
    }
    GemmArgs g{};
    g.A = xq;
    g.B = wq;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.sa = x_scale;
    g.sb = w_scale;
    g.bias = bias;
    g.y = y;
    g.ldy = ldy;
    g.acc_out = acc_out;
    launch_gemm_i8(g, PDQ_BF16, false, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_linear_prefill(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                              const int8_t* wq, const float* w_scale, const float* bias, int64_t N,
                              int8_t* xq, float* x_scale, uint16_t* y, int64_t ldy,
                              int32_t* acc_out, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (N > 0 && !w_scale) return PDQ_ERR_NULL;
    if (M > 0 && ((K > 0 && !xq) || !x_scale)) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
        !aligned(y, 2) || !aligned(acc_out, 4))
        return PDQ_ERR_ALIGN;
    PDQ_TRY(pdq_quantize_per_token(x, x_dt, M, K, ldx, xq, x_scale, stream));
    return pdq_gemm_per_token(xq, x_scale, M, K, wq, w_scale, bias, N, y, ldy, acc_out, stream);
}

pdq_status pdq_silu_mul_quantize_per_token(const void* gate, const void* up, pdq_dtype dt, int64_t M,
                                           int64_t K, int64_t ldg, int64_t ldu, int8_t* xq,
                                           float* x_scale, uint16_t* h, int64_t ldh, void* stream) {
    if (dt != PDQ_BF16 && dt != PDQ_F16) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(gate, 2, M, K, ldg));
    PDQ_TRY(check_operand(up, 2, M, K, ldu));
    if (h) PDQ_TRY(check_operand(h, 2, M, K, ldh));
    if (M > 0 && ((K > 0 && !xq) || !x_scale)) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4)) return PDQ_ERR_ALIGN;
    if (M == 0) return PDQ_OK;
    launch_silu_mul_quant(gate, ldg, up, ldu, dt, M, K, xq, x_scale, h, ldh, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_linear_prefill_silu_mul(const void* gate, const void* up, pdq_dtype dt, int64_t M, int64_t K,
                                       int64_t ldg, int64_t ldu, const int8_t* wq, const float* w_scale,
                                       const float* bias, int64_t N, int8_t* xq, float* x_scale,
                                       uint16_t* y, int64_t ldy, int32_t* acc_out, void* stream) {
    if (dt != PDQ_BF16 && dt != PDQ_F16) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(gate, 2, M, K, ldg));
    PDQ_TRY(check_operand(up, 2, M, K, ldu));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (N > 0 && !w_scale) return PDQ_ERR_NULL;
    if (M > 0 && ((K > 0 && !xq) || !x_scale)) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(bias, 4) ||
        !aligned(y, 2) || !aligned(acc_out, 4))
        return PDQ_ERR_ALIGN;
    PDQ_TRY(pdq_silu_mul_quantize_per_token(gate, up, dt, M, K, ldg, ldu, xq, x_scale, nullptr, 0, stream));
    return pdq_gemm_per_token(xq, x_scale, M, K, wq, w_scale, bias, N, y, ldy, acc_out, stream);
}

pdq_status pdq_quantize_per_token_asym(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                       int8_t* xq, float* x_scale, int32_t* x_zp, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (M > 0 && ((K > 0 && !xq) || !x_scale || !x_zp)) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(x_zp, 4)) return PDQ_ERR_ALIGN;
    if (M == 0) return PDQ_OK;
    launch_quant_rows_asym(x, x_dt, M, K, ldx, xq, x_scale, x_zp, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_gemm_per_token_asym(const int8_t* xq, const float* x_scale, const int32_t* x_zp, int64_t M,
                                   int64_t K, const int8_t* wq, const float* w_scale,
                                   const int32_t* w_colsum, const float* bias, int64_t N, uint16_t* y,
                                   int64_t ldy, int32_t* acc_out, void* stream) {
    PDQ_TRY(check_operand(xq, 1, M, K, K));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (N > 0 && (!w_scale || !w_colsum)) return PDQ_ERR_NULL;
    if (M > 0 && (!x_scale || !x_zp)) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(x_scale, 4) || !aligned(x_zp, 4) || !aligned(w_scale, 4) || !aligned(w_colsum, 4) ||
        !aligned(bias, 4) || !aligned(y, 2) || !aligned(acc_out, 4))
        return PDQ_ERR_ALIGN;
    if (M == 0 || N == 0) return PDQ_OK;
    if (skinny_gemm(M, N)) {
        DecodeArgs d{};
        d.xq = xq;
        d.wq = wq;
        d.M = (int)M;
        d.N = (int)N;
        d.K = (int)K;
        d.sa = x_scale;
        d.za = x_zp;
        d.sw = w_scale;
        d.colsum = w_colsum;
        d.bias = bias;
        d.y = y;
        d.ldy = ldy;
        d.acc_out = acc_out;
        launch_decode_gemv(d, static_cast<hipStream_t>(stream));
        return launched();
    }
    GemmArgs g{};
    g.A = xq;
    g.B = wq;
    g.M = (int)M;
    g.N = (int)N;
    g.K = (int)K;
    g.sa = x_scale;
    g.za = x_zp;
    g.colsum = w_colsum;
    g.sb = w_scale;
    g.bias = bias;
    g.y = y;
    g.ldy = ldy;
    g.acc_out = acc_out;
    launch_gemm_i8(g, PDQ_BF16, false, static_cast<hipStream_t>(stream), 2);
    return launched();
}

pdq_status pdq_linear_prefill_asym(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                   const int8_t* wq, const float* w_scale, const int32_t* w_colsum,
                                   const float* bias, int64_t N, int8_t* xq, float* x_scale, int32_t* x_zp,
                                   uint16_t* y, int64_t ldy, int32_t* acc_out, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (N > 0 && (!w_scale || !w_colsum)) return PDQ_ERR_NULL;
    if (M > 0 && ((K > 0 && !xq) || !x_scale || !x_zp)) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4) || !aligned(x_zp, 4) || !aligned(w_scale, 4) ||
        !aligned(w_colsum, 4) || !aligned(bias, 4) || !aligned(y, 2) || !aligned(acc_out, 4))
        return PDQ_ERR_ALIGN;
    PDQ_TRY(pdq_quantize_per_token_asym(x, x_dt, M, K, ldx, xq, x_scale, x_zp, stream));
    return pdq_gemm_per_token_asym(xq, x_scale, x_zp, M, K, wq, w_scale, w_colsum, bias, N, y, ldy, acc_out,
                                   stream);
}

pdq_status pdq_quantize_static(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                               float a_scale, int32_t a_zp, int8_t* xq, uint32_t* sat_count,
                               void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (!(a_scale > 0.0f) || !isfinite(a_scale) || a_zp < -128 || a_zp > 127)
        return PDQ_ERR_UNSUPPORTED;
    if (M > 0 && K > 0 && !xq) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(sat_count, 4)) return PDQ_ERR_ALIGN;
    if (M == 0) return PDQ_OK;
    launch_quant_static(x, x_dt, M, K, ldx, a_scale, a_zp, xq, sat_count,
                        static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_gemm_static(const int8_t* xq, int64_t M, int64_t K, float a_scale, int32_t a_zp,
                           const int8_t* wq, const float* w_scale, const int32_t* w_colsum,
                           const float* bias, int64_t N, uint16_t* y, int64_t ldy, int32_t* acc_out,
                           void* stream) {
    PDQ_TRY(check_operand(xq, 1, M, K, K));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (!(a_scale > 0.0f) || !isfinite(a_scale) || a_zp < -128 || a_zp > 127)
        return PDQ_ERR_UNSUPPORTED;
    if (N > 0 && (!w_scale || (a_zp != 0 && !w_colsum))) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(w_scale, 4) || !aligned(w_colsum, 4) || !aligned(bias, 4) || !aligned(y, 2) ||
        !aligned(acc_out, 4))
        return PDQ_ERR_ALIGN;
    if (M == 0 || N == 0) return PDQ_OK;
    if (!skinny_gemm(M, N)) {
        GemmArgs g{};
        g.A = xq;
        g.B = wq;
        g.M = (int)M;
        g.N = (int)N;
        g.K = (int)K;
        g.s = a_scale;
        g.z = a_zp;
        g.colsum = w_colsum;
        g.sb = w_scale;
        g.bias = bias;
        g.y = y;
        g.ldy = ldy;
        g.acc_out = acc_out;
        launch_gemm_i8(g, PDQ_BF16, false, static_cast<hipStream_t>(stream), a_zp != 0 ? 1 : 0);
        return launched();
    }
    DecodeArgs d{};
    d.xq = xq;
    d.wq = wq;
    d.M = (int)M;
    d.N = (int)N;
    d.K = (int)K;
    d.s = a_scale;
    d.z = a_zp;
    d.sw = w_scale;
    d.colsum = a_zp != 0 ? w_colsum : nullptr;
    d.bias = bias;
    d.y = y;
    d.ldy = ldy;
    d.acc_out = acc_out;
    launch_decode_gemv(d, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_calibrate_static_sym(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                    float* minmax, float* a_scale, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (!minmax) return PDQ_ERR_NULL;
    if (!aligned(minmax, 4) || !aligned(a_scale, 4)) return PDQ_ERR_ALIGN;
    hipStream_t st = static_cast<hipStream_t>(stream);
    launch_minmax(x, x_dt, M, K, ldx, minmax, st);
    if (a_scale) launch_absmax_finalize(minmax, a_scale, st);
    return launched();
}

pdq_status pdq_quantize_static_sym(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                   float a_scale, int8_t* xq, uint32_t* sat_count, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (!(a_scale > 0.0f) || !isfinite(a_scale)) return PDQ_ERR_UNSUPPORTED;
    if (M > 0 && K > 0 && !xq) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(sat_count, 4)) return PDQ_ERR_ALIGN;
    if (M == 0) return PDQ_OK;
    launch_quant_static(x, x_dt, M, K, ldx, a_scale, 0, xq, sat_count, static_cast<hipStream_t>(stream),
                        true);
    return launched();
}

pdq_status pdq_linear_static_sym(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                 float a_scale, const int8_t* wq, const float* w_scale, const float* bias,
                                 int64_t N, int8_t* xq, uint16_t* y, int64_t ldy, int32_t* acc_out,
                                 uint32_t* sat_count, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (!(a_scale > 0.0f) || !isfinite(a_scale)) return PDQ_ERR_UNSUPPORTED;
    if (N > 0 && !w_scale) return PDQ_ERR_NULL;
    if (M > 0 && K > 0 && !xq) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(w_scale, 4) || !aligned(bias, 4) || !aligned(y, 2) ||
        !aligned(acc_out, 4) || !aligned(sat_count, 4))
        return PDQ_ERR_ALIGN;
    if (N > 0 && decode_fusable(M, K)) {
        DecodeArgs d{};
        d.wq = wq;
        d.M = (int)M;
        d.N = (int)N;
        d.K = (int)K;
        d.s = a_scale;
        d.z = 0;
        d.narrow = 1;
        d.sw = w_scale;
        d.bias = bias;
        d.y = y;
        d.ldy = ldy;
        d.acc_out = acc_out;
        d.x = x;
        d.x_dt = x_dt;
        d.ldx = ldx;
        d.xq_out = xq;
        d.sat = sat_count;
        launch_decode_fused(d, static_cast<hipStream_t>(stream));
        return launched();
    }
    PDQ_TRY(pdq_quantize_static_sym(x, x_dt, M, K, ldx, a_scale, xq, sat_count, stream));
    return pdq_gemm_static(xq, M, K, a_scale, 0, wq, w_scale, nullptr, bias, N, y, ldy, acc_out, stream);
}

pdq_status pdq_calibrate_zeropoint(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                   float* minmax, float* a_scale, int32_t* a_zp, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (!minmax) return PDQ_ERR_NULL;
    if ((a_scale == nullptr) != (a_zp == nullptr)) return PDQ_ERR_NULL;
    if (!aligned(minmax, 4) || !aligned(a_scale, 4) || !aligned(a_zp, 4)) return PDQ_ERR_ALIGN;
    hipStream_t st = static_cast<hipStream_t>(stream);
    launch_minmax(x, x_dt, M, K, ldx, minmax, st);
    if (a_scale) launch_zeropoint_finalize(minmax, a_scale, a_zp, st);
    return launched();
}

pdq_status pdq_quantize_zeropoint(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                  float a_scale, int32_t a_zp, int8_t* xq, uint32_t* sat_count, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (!(a_scale > 0.0f) || !isfinite(a_scale) || a_zp < -127 || a_zp > 127) return PDQ_ERR_UNSUPPORTED;
    if (M > 0 && K > 0 && !xq) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(sat_count, 4)) return PDQ_ERR_ALIGN;
    if (M == 0) return PDQ_OK;
    launch_quant_static(x, x_dt, M, K, ldx, a_scale, a_zp, xq, sat_count, static_cast<hipStream_t>(stream),
                        true);
    return launched();
}

pdq_status pdq_linear_zeropoint(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                                float a_scale, int32_t a_zp, const int8_t* wq, const float* w_scale,
                                const int32_t* w_colsum, const float* bias, int64_t N, int8_t* xq,
                                uint16_t* y, int64_t ldy, int32_t* acc_out, uint32_t* sat_count,
                                void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (!(a_scale > 0.0f) || !isfinite(a_scale) || a_zp < -127 || a_zp > 127) return PDQ_ERR_UNSUPPORTED;
    if (N > 0 && (!w_scale || !w_colsum)) return PDQ_ERR_NULL;
    if (M > 0 && K > 0 && !xq) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(w_scale, 4) || !aligned(w_colsum, 4) || !aligned(bias, 4) ||
        !aligned(y, 2) || !aligned(acc_out, 4) || !aligned(sat_count, 4))
        return PDQ_ERR_ALIGN;
    if (N > 0 && decode_fusable(M, K)) {
        DecodeArgs d{};
        d.wq = wq;
        d.M = (int)M;
        d.N = (int)N;
        d.K = (int)K;
        d.s = a_scale;
        d.z = a_zp;
        d.narrow = 1;
        d.sw = w_scale;
        d.colsum = w_colsum;
        d.bias = bias;
        d.y = y;
        d.ldy = ldy;
        d.acc_out = acc_out;
        d.x = x;
        d.x_dt = x_dt;
        d.ldx = ldx;
        d.xq_out = xq;
        d.sat = sat_count;
        launch_decode_fused(d, static_cast<hipStream_t>(stream));
        return launched();
    }
    PDQ_TRY(pdq_quantize_zeropoint(x, x_dt, M, K, ldx, a_scale, a_zp, xq, sat_count, stream));
    return pdq_gemm_static(xq, M, K, a_scale, a_zp, wq, w_scale, w_colsum, bias, N, y, ldy, acc_out, stream);
}

pdq_status pdq_linear_decode(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx,
                             float a_scale, int32_t a_zp, const int8_t* wq, const float* w_scale,
                             const int32_t* w_colsum, const float* bias, int64_t N, int8_t* xq,
                             uint16_t* y, int64_t ldy, int32_t* acc_out, uint32_t* sat_count,
                             void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    PDQ_TRY(check_operand(wq, 1, N, K, K));
    if (N < 0 || N > kMaxRows || M * N > kMaxOutputs || ldy < N) return PDQ_ERR_SHAPE;
    if (!(a_scale > 0.0f) || !isfinite(a_scale) || a_zp < -128 || a_zp > 127)
        return PDQ_ERR_UNSUPPORTED;
    if (N > 0 && (!w_scale || !w_colsum)) return PDQ_ERR_NULL;
    if (M > 0 && K > 0 && !xq) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(w_scale, 4) || !aligned(w_colsum, 4) || !aligned(bias, 4) ||
        !aligned(y, 2) || !aligned(acc_out, 4) || !aligned(sat_count, 4))
        return PDQ_ERR_ALIGN;
    if (N > 0 && decode_fusable(M, K)) {
        // one launch: the GEMM quantizes the activations itself (and writes xq)
        if (!y) return PDQ_ERR_NULL;
        DecodeArgs d{};
        d.wq = wq;
        d.M = (int)M;
        d.N = (int)N;
        d.K = (int)K;
        d.s = a_scale;
        d.z = a_zp;
        d.sw = w_scale;
        d.colsum = w_colsum;
        d.bias = bias;
        d.y = y;
        d.ldy = ldy;
        d.acc_out = acc_out;
        d.x = x;
        d.x_dt = x_dt;
        d.ldx = ldx;
        d.xq_out = xq;
        d.sat = sat_count;
        launch_decode_fused(d, static_cast<hipStream_t>(stream));
        return launched();
    }
    PDQ_TRY(pdq_quantize_static(x, x_dt, M, K, ldx, a_scale, a_zp, xq, sat_count, stream));
    return pdq_gemm_static(xq, M, K, a_scale, a_zp, wq, w_scale, w_colsum, bias, N, y, ldy, acc_out,
                           stream);
}

size_t pdq_linear_int8_outlier_workspace(int64_t M, int64_t N, int64_t K, int64_t max_outliers) {
    if (M < 0 || N < 0 || K < 0 || max_outliers < 0) return 0;
    const int64_t P = side_pitch(max_outliers);
    const size_t pitch = (size_t)outlier_partial_pitch(K);
    return align256((size_t)outlier_row_blocks(M) * pitch) + align256(pitch) +
           align256((size_t)(M * P * 2)) + align256((size_t)(N * P * 2));
}

pdq_status pdq_linear_int8_outlier(const void* x, pdq_dtype dt, int64_t M, int64_t K, int64_t ldx,
                                   float threshold, const int8_t* wq, const float* w_scale,
                                   const void* w16, int64_t ldw, const float* bias, int64_t N,
                                   void* y, int64_t ldy, int8_t* xq, float* x_scale,
                                   int32_t* outlier_idx, int32_t* n_outlier, int64_t max_outliers,
                                   void* workspace, size_t workspace_bytes, int32_t* acc_out,
                                   void* stream) {
    PDQ_TRY(check_int8_outlier(x, dt, M, K, ldx, threshold, wq, w_scale, w16, ldw, bias, N, y, ldy, xq,
                               x_scale, outlier_idx, n_outlier, max_outliers, acc_out));
    const size_t need = pdq_linear_int8_outlier_workspace(M, N, K, max_outliers);
    if (!workspace || workspace_bytes < need) return PDQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PDQ_ERR_ALIGN;
    run_int8_outlier(x, dt, M, K, ldx, threshold, wq, w_scale, w16, ldw, bias, N, y, ldy, xq, x_scale,
                     outlier_idx, n_outlier, max_outliers, static_cast<char*>(workspace), acc_out,
                     static_cast<hipStream_t>(stream));
    return launched();
}

size_t pdq_noalloc_scratch_bytes(void) { return kScratchBytes; }

pdq_status pdq_linear_int8_outlier_noalloc(const void* x, pdq_dtype dt, int64_t M, int64_t K, int64_t ldx,
                                           float threshold, const int8_t* wq, const float* w_scale,
                                           const void* w16, int64_t ldw, const float* bias, int64_t N,
                                           void* y, int64_t ldy, int8_t* xq, float* x_scale,
                                           int32_t* outlier_idx, int32_t* n_outlier, int64_t max_outliers,
                                           int32_t* acc_out, void* stream) {
    PDQ_TRY(check_int8_outlier(x, dt, M, K, ldx, threshold, wq, w_scale, w16, ldw, bias, N, y, ldy, xq,
                               x_scale, outlier_idx, n_outlier, max_outliers, acc_out));
    if (pdq_linear_int8_outlier_workspace(M, N, K, max_outliers) > kScratchBytes) return PDQ_ERR_WORKSPACE;
    // the argument checks above make no HIP call; from here on the device's
    // own copy of the scratch array is looked up (once per device)
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = nullptr;
    PDQ_TRY(scratch_for_stream(st, &ws));
    run_int8_outlier(x, dt, M, K, ldx, threshold, wq, w_scale, w16, ldw, bias, N, y, ldy, xq, x_scale,
                     outlier_idx, n_outlier, max_outliers, ws, acc_out, st);
    return launched();
}

}  // extern "C"

namespace {

constexpr int64_t kMaxBatch = 65536, kMaxHeads = 256, kMaxSeq = int64_t(1) << 30;
constexpr int64_t kMaxThreads = int64_t(1) << 31;  // of one launch

// The checks that the two cache calls share; fills the kernels' views.
pdq_status check_kv(const pdq_kv_cache* cache, const pdq_kv_batch* batch, int64_t tokens, KvCache* c, KvBatch* b) {
    if (!cache || !batch) return PDQ_ERR_NULL;
    if (cache->pages < 0 || cache->pages > INT32_MAX || cache->heads < 1 || cache->heads > kMaxHeads) return PDQ_ERR_SHAPE;
    if (cache->page != 16 && cache->page != 32 && cache->page != 64 && cache->page != 128 && cache->page != 256)
        return PDQ_ERR_SHAPE;
    if (cache->dim != 64 && cache->dim != 128 && cache->dim != 256) return PDQ_ERR_SHAPE;
    if (tokens < 0 || tokens > kMaxRows || batch->batch < 0 || batch->batch > kMaxBatch) return PDQ_ERR_SHAPE;
    if (batch->max_pages < 0 || (int64_t)batch->max_pages * cache->page > kMaxSeq || batch->ldt < batch->max_pages)
        return PDQ_ERR_SHAPE;
    if (!batch->cu_q && tokens != batch->batch) return PDQ_ERR_SHAPE;
    if (cache->pages > 0 && (!cache->k || !cache->v || !cache->k_scale || !cache->v_scale)) return PDQ_ERR_NULL;
    if (batch->batch > 0 && (!batch->seq_len || (batch->max_pages > 0 && !batch->page_table))) return PDQ_ERR_NULL;
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16) || !aligned(cache->k_scale, 4) ||
        !aligned(cache->v_scale, 4) || !aligned(batch->page_table, 4) || !aligned(batch->seq_len, 4) ||
        !aligned(batch->cu_q, 4))
        return PDQ_ERR_ALIGN;
    *c = KvCache{cache->k, cache->v, cache->k_scale, cache->v_scale, (int)cache->pages, cache->heads, cache->page,
                 cache->dim};
    *b = KvBatch{batch->page_table, batch->ldt, batch->seq_len, batch->cu_q, batch->batch, batch->max_pages,
                 (int)tokens};
    return PDQ_OK;
}

// A [rows, heads, dim] operand of 16-bit values.
pdq_status check_rows(const void* p, int64_t rows, int64_t heads, int64_t dim, int64_t ld) {
    if (rows * heads > kMaxValues / dim || ld < heads * dim || ld > kMaxValues) return PDQ_ERR_SHAPE;
    if (rows > 0 && !p) return PDQ_ERR_NULL;
    if (!aligned(p, 16) || ld % 8 != 0) return PDQ_ERR_ALIGN;
    return PDQ_OK;
}

}  // namespace

extern "C" {

pdq_status pdq_kv_append(const void* k, const void* v, const void* q, pdq_dtype dt, int64_t tokens,
                         int64_t hq, int64_t ldk, int64_t ldv, int64_t ldq, const float* cos, const float* sin,
                         int64_t positions, int64_t rot, int interleaved, const pdq_kv_cache* cache,
                         const pdq_kv_batch* batch, void* q_out, int64_t ldqo, void* stream) {
    if (dt != PDQ_BF16 && dt != PDQ_F16) return PDQ_ERR_DTYPE;
    KvAppendArgs a{};
    PDQ_TRY(check_kv(cache, batch, tokens, &a.c, &a.b));
    PDQ_TRY(check_rows(k, tokens, a.c.heads, a.c.dim, ldk));
    PDQ_TRY(check_rows(v, tokens, a.c.heads, a.c.dim, ldv));
    if (!cos != !sin || (q && !cos) || (q && tokens > 0 && !q_out)) return PDQ_ERR_NULL;
    if (q) {
        if (hq < 1 || hq > kMaxHeads * 64) return PDQ_ERR_SHAPE;
        PDQ_TRY(check_rows(q, tokens, hq, a.c.dim, ldq));
        PDQ_TRY(check_rows(q_out, tokens, hq, a.c.dim, ldqo));
    }
    if (cos) {
        if (positions < 1 || positions > kMaxSeq || rot < 16 || rot > a.c.dim || rot % 16 != 0) return PDQ_ERR_SHAPE;
        if (!aligned(cos, 16) || !aligned(sin, 16)) return PDQ_ERR_ALIGN;
    }
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.ldk = ldk;
    a.ldv = ldv;
    a.ldq = ldq;
    a.ldqo = ldqo;
    a.cos = cos;
    a.sin = sin;
    a.positions = (int)positions;
    a.rot = (int)rot;
    a.interleaved = interleaved != 0;
    a.hq = q ? (int)hq : 1;
    if (kv_append_threads(a) > kMaxThreads) return PDQ_ERR_SHAPE;
    if (tokens == 0 || a.b.batch == 0) return PDQ_OK;
    launch_kv_append(a, dt, static_cast<hipStream_t>(stream));
    return launched();
}

size_t pdq_kv_attention_workspace(int64_t tokens, int64_t batch, int64_t hq, int64_t heads, int64_t dim) {
    if (tokens < 1 || batch < 1 || heads < 1 || heads > kMaxHeads || hq < heads || hq > kMaxHeads * 64 ||
        hq % heads != 0 || dim < 1 || tokens > kMaxRows || batch > kMaxBatch)
        return 0;
    return align256(attention_workspace(tokens, batch, (int)hq, (int)heads, (int)dim));
}

pdq_status pdq_kv_attention(const void* q, pdq_dtype dt, int64_t tokens, int64_t hq, int64_t ldq,
                            const pdq_kv_cache* cache, const pdq_kv_batch* batch, float scale, float softcap,
                            int64_t window, const float* slopes, const int32_t* prefix, void* y, int64_t ldy,
                            float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    if (dt != PDQ_BF16 && dt != PDQ_F16) return PDQ_ERR_DTYPE;
    AttentionArgs a{};
    PDQ_TRY(check_kv(cache, batch, tokens, &a.c, &a.b));
    if (hq < a.c.heads || hq > kMaxHeads * 64 || hq % a.c.heads != 0 || window < 0 || window > INT32_MAX)
        return PDQ_ERR_SHAPE;
    PDQ_TRY(check_rows(q, tokens, hq, a.c.dim, ldq));
    PDQ_TRY(check_rows(y, tokens, hq, a.c.dim, ldy));
    if (!isfinite(scale) || !isfinite(softcap) || softcap < 0.0f) return PDQ_ERR_UNSUPPORTED;
    // the factors that the kernels form of them, which times a zero product would be NaN
    if (!isfinite(1.4426950408889634f * scale) || !isfinite(softcap > 0.0f ? 2.0f * 1.4426950408889634f / softcap * scale : 0.0f))
        return PDQ_ERR_UNSUPPORTED;
    if (!aligned(slopes, 4) || !aligned(prefix, 4) || !aligned(lse, 4)) return PDQ_ERR_ALIGN;
    const size_t need = pdq_kv_attention_workspace(tokens, a.b.batch, hq, a.c.heads, a.c.dim);
    if (need > 0 && (!workspace || workspace_bytes < need)) return PDQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PDQ_ERR_ALIGN;
    a.q = q;
    a.y = y;
    a.lse = lse;
    a.ldq = ldq;
    a.ldy = ldy;
    a.hq = (int)hq;
    a.scale = scale;
    a.softcap = softcap;
    a.window = (int)window;
    a.slopes = slopes;
    a.prefix = prefix;
    a.ws = static_cast<float*>(workspace);
    if (attention_threads(a) > kMaxThreads) return PDQ_ERR_SHAPE;
    if (tokens == 0 || a.b.batch == 0) return PDQ_OK;
    launch_attention(a, dt, static_cast<hipStream_t>(stream));
    return launched();
}

}  // extern "C"

namespace {

constexpr int64_t kMaxExperts = 512, kMaxChoices = 32, kMaxSorted = int64_t(1) << 30;

bool scale_ok(int t) { return t == PDQ_E8M0 || t == PDQ_SCALE_F32; }

// count matrices of N x K: the sizes' limits, of one of them and of all.
pdq_status check_stack(int64_t count, int64_t N, int64_t K) {
    PDQ_TRY(check_mk(N, K, K));
    if (count < 0 || count > kMaxRows) return PDQ_ERR_SHAPE;
    const int64_t padded = (N + 127) / 128 * 128 * (fp8_groups(K) * 128);
    if (count > 0 && padded > kMaxValues / count) return PDQ_ERR_SHAPE;
    return PDQ_OK;
}

// One product: its operands, and as many outputs as a launch's threads take (tiles of 128 x 256 by 256 of them).
pdq_status check_fp8_sizes(int64_t M, int64_t N, int64_t K) {
    PDQ_TRY(check_mk(M, K, K));
    PDQ_TRY(check_stack(1, N, K));
    return M * N > std::min(kMaxOutputs, kMaxThreads * 128) ? PDQ_ERR_SHAPE : PDQ_OK;
}

pdq_status check_fp8_gemm(int64_t M, int64_t K, const uint8_t* wq, const void* w_scale, pdq_scale_type scale_t,
                          const float* bias, int64_t N, const uint8_t* xq, const uint8_t* x_scale, const void* y,
                          pdq_dtype y_dt, int64_t ldy) {
    if (y_dt != PDQ_BF16 && y_dt != PDQ_F16) return PDQ_ERR_DTYPE;
    if (!scale_ok(scale_t)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_fp8_sizes(M, N, K));
    if (ldy < N) return PDQ_ERR_SHAPE;
    if (N > 0 && (!wq || !w_scale)) return PDQ_ERR_NULL;
    if (M > 0 && (!xq || !x_scale)) return PDQ_ERR_NULL;
    if (M > 0 && N > 0 && !y) return PDQ_ERR_NULL;
    if (!aligned(wq, 16) || !aligned(xq, 16) || !aligned(w_scale, 16) || !aligned(x_scale, 4) || !aligned(bias, 4) ||
        !aligned(y, 2))
        return PDQ_ERR_ALIGN;
    return PDQ_OK;
}

Fp8GemmArgs fp8_gemm_args(int64_t M, int64_t K, const uint8_t* wq, const void* w_scale, pdq_scale_type scale_t,
                          const float* bias, int64_t N, const uint8_t* xq, const uint8_t* x_scale, void* y, int64_t ldy) {
    Fp8GemmArgs a{};
    a.x = xq;
    a.xs = x_scale;
    a.w = wq;
    a.ws = w_scale;
    a.ws_f32 = scale_t == PDQ_SCALE_F32;
    a.M = (int)M;
    a.N = (int)N;
    a.groups = (int)fp8_groups(K);
    a.pitch = (int)fp8_scale_pitch(K);
    a.bias = bias;
    a.y = y;
    a.ldy = ldy;
    return a;
}

// The tile of an FP8 product, 0 rows: the kernel for few rows.  The estimates are in microseconds for G groups, from times
// measured on MI355X, every kernel at 416 sizes (65 .. 65536 rows, N 64 .. 28672, K 16 .. 14336, both types of scales; a part of them with
// the weights in the last-level cache): what the rule takes is slower than the best by 2% on average.
// - Few rows: rounds of 256 workgroups (64 rows x 16, 32 or 64 channels), the last one as long as a full one: 600 x 2048 x 11008, 1.3 of
//   them, 40.9 (128 x 128: 49.5), 512 x 4096 x 11008, two, 47.5 (54.0).  Where the blocks of rows that share a weight's channels
//   run on different XCDs, each reads the weight: 400 x 3008 x 11008 50.7 (43.3).
// - 128 x 128: rounds of 512 tiles, two a compute unit, or of 256 for less (1024 x 4096 x 11008 54.9, 2048 x 4096 x 11008 100.8).  The other
//   tiles: rounds of 256.
// - Outputs whose rows are no multiple of 8 leave in single stores: 600 x 1003 x 1360 7.1 / 11.5 / 19.1 / 34.1 (few rows / 128 x 128 / 128 x
//   256 / 256 x 256), 600 x 2048 x 1360 8.2 / 7.7 / 11.1 / 18.4.
// E.g. K 4096: 200 x 4096 14.1 / 19.0 / 28.1 / 38.3, 1024 x 4096 39.1 / 21.0 / 28.6 / 40.5, 2048 x 4096 74.5 / 38.9 / 32.7 / 46.9, 4096 x
// 11008 434 / 178 / 163 / 144; one group, 65536 x 4096: 396 / 179 / 187 / 186.  Binary32 scales (few rows / 128 x 128 / 192 x 256): 512 x 4096
// 23.8 / 21.5 / 42.8, 8192 x 8192 - / 269 / 278, 8192 x 14336 -> 4096 - / 543 / 506; 128 x 256 is never the best there.
Fp8TileShape fp8_tile_shape(int64_t M, int64_t N, int64_t G, bool f32) {
    if (M <= 64) return Fp8TileShape{0, 0};
    auto count = [&](int64_t rows, int64_t channels) { return ((M + rows - 1) / rows) * ((N + channels - 1) / channels); };
    auto ceil256 = [](int64_t n) { return (double)((n + 255) / 256); };
    // rounds of 256 that take `full`, the last one down to `some` the fewer it has
    auto rounds = [&](int64_t n, double some, double full) {
        const int64_t rest = n % 256;
        return (double)(n / 256) * full + (rest ? some + (full - some) * rest / 256 : 0);
    };
    const bool single = N % 8 != 0;

    const int width = fp8_rows_width(M, N);
    const int64_t blocks = (N + 16 * width - 1) / (16 * width), groups = (M + 63) / 64 * blocks;
    const double turns = width == 2 ? std::max(1.0, groups / 128.0 - 1) : ceil256(groups);
    const double a_group = width == 4 ? (f32 ? 0.13 : 0.11) + 0.195 * turns : width == 2 ? 0.08 + 0.16 * turns : 0.02 + 0.14 * turns;
    const double few = groups * 512 > kMaxThreads ? 1e18 : (3 + (f32 ? 1.5 : 1.3) * turns + G * a_group) * (blocks % 8 ? 1.15 : 1.0);

    const int64_t small = count(128, 128), rest = small % 512;
    const double one = f32 ? 3.5 + 0.58 * G : 2.5 + 0.55 * G, two = std::max(5.5 + 0.95 * G, 1.2 * G - 3);
    const double more = std::min(1.4 * one, two);  // a second tile on some compute units
    const double last = rest == 0 ? 0 : rest <= 256 ? one : more + (two - more) * (rest - 256) / 256;
    const double t128 = small * 256 > kMaxThreads ? 1e18 : (double)(small / 512) * two + last + (single ? 3.5 * ceil256(small) : 0);

    const int64_t wide = count(128, 256), most = count(f32 ? 192 : 256, 256);
    const double t128x256 = f32 ? 1e18 : rounds(wide, 4 + 0.85 * G, 4 + 0.93 * G) + (single ? 8 * ceil256(wide) : 0);
    const double full = f32 ? std::max(std::max(8.0 + G, 6 + 1.35 * G), 1.5 * G) : std::max(10 + 0.9 * G, 4 + 1.4 * G);
    const double large = rounds(most, f32 ? 7 + 1.11 * G : 7.5 + 1.02 * G, full) + (single ? (f32 ? 11 : 14) * ceil256(most) : 0);

    const double best = std::min(t128, std::min(t128x256, large));
    if (few <= best) return Fp8TileShape{0, 0};
    if (best == large) return Fp8TileShape{f32 ? 192 : 256, 256};
    return best == t128 ? Fp8TileShape{128, 128} : Fp8TileShape{128, 256};
}

// The parts of the experts' layer's workspace, in bytes.
struct ExpertsSpace {
    size_t x, xs, h, hs, partial;
    size_t all() const { return x + xs + h + hs + partial; }
};
ExpertsSpace experts_space(int64_t tokens, int64_t k, int64_t experts, int64_t hidden, int64_t inner) {
    if (fp8_experts_direct(tokens * k, k, hidden, inner))  // h alone
        return ExpertsSpace{0, 0, 0, 0, align256((size_t)(tokens * k * inner * 4))};
    const int64_t rows = 16 * fp8_blocks(tokens * k, experts);
    return ExpertsSpace{align256((size_t)(rows * fp8_groups(hidden) * kGroup)), align256((size_t)(rows * fp8_scale_pitch(hidden))),
                        align256((size_t)(rows * fp8_groups(inner) * kGroup)), align256((size_t)(rows * fp8_scale_pitch(inner))),
                        align256((size_t)(tokens * k * hidden * 4))};
}
bool experts_sizes_ok(int64_t tokens, int64_t k, int64_t experts, int64_t hidden, int64_t inner) {
    if (tokens < 0 || tokens > kMaxRows || experts < 1 || experts > kMaxExperts || k < 1 || k > std::min(experts, kMaxChoices))
        return false;
    if (tokens * k > kMaxSorted) return false;
    if (hidden < 16 || hidden > kMaxK || hidden % 16 != 0 || inner < 16 || inner > kMaxK || inner % 16 != 0) return false;
    return tokens * k <= kMaxValues / std::max(hidden, inner);
}

}  // namespace

extern "C" {

size_t pdq_fp8_bytes(int64_t rows, int64_t K) {
    if (rows < 0 || K < 0) return 0;
    return (size_t)((rows + kWGroup - 1) / kWGroup) * (size_t)fp8_groups(K) * kGroupBytes;
}

int64_t pdq_fp8_scale_pitch(int64_t K) { return K < 0 ? 0 : fp8_scale_pitch(K); }

pdq_status pdq_quantize_weight_fp8(const void* w, pdq_dtype w_dt, int64_t count, int64_t N, int64_t K, int64_t ldw,
                                   int64_t stride, uint8_t* wq, uint8_t* w_scale, void* stream) {
    if (!dtype_ok(w_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_stack(count, N, K));
    if (ldw < K || ldw > kMaxValues) return PDQ_ERR_SHAPE;
    if (count > 1 && N > 0 && (stride < (N - 1) * ldw + K || stride > kMaxValues)) return PDQ_ERR_SHAPE;
    if (count > 0 && N > 0 && (!w || !wq || !w_scale)) return PDQ_ERR_NULL;
    const int eb = elem_bytes(w_dt);
    if (!aligned(w, 16) || (ldw * eb) % 16 != 0 || (count > 1 && (stride * eb) % 16 != 0) || !aligned(wq, 16))
        return PDQ_ERR_ALIGN;
    if (count == 0 || N == 0) return PDQ_OK;
    launch_fp8_weight(Fp8WeightArgs{w, count, N, K, ldw, stride, wq, w_scale}, w_dt, static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_pack_weight_fp8(const uint8_t* codes, const void* scale, pdq_scale_type scale_t, int64_t count,
                               int64_t N, int64_t K, uint8_t* wq, void* w_scale, void* stream) {
    if (!scale_ok(scale_t)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_stack(count, N, K));
    if (count > 0 && N > 0 && (!codes || !scale || !wq || !w_scale)) return PDQ_ERR_NULL;
    const uintptr_t es = scale_t == PDQ_SCALE_F32 ? 4 : 1;
    if (!aligned(codes, 16) || !aligned(wq, 16) || !aligned(scale, es) || !aligned(w_scale, es)) return PDQ_ERR_ALIGN;
    if (count == 0 || N == 0) return PDQ_OK;
    launch_fp8_pack(Fp8PackArgs{codes, scale, count, N, K, scale_t == PDQ_SCALE_F32, wq, w_scale},
                    static_cast<hipStream_t>(stream));
    return launched();
}

pdq_status pdq_quantize_fp8(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx, uint8_t* xq,
                            uint8_t* x_scale, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    if (M > 0 && (!xq || !x_scale)) return PDQ_ERR_NULL;
    if (!aligned(xq, 16) || !aligned(x_scale, 4)) return PDQ_ERR_ALIGN;
    if (M == 0) return PDQ_OK;
    Fp8QuantArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.M = M;
    a.K = (int)K;
    a.groups = (int)fp8_groups(K);
    a.pitch = (int)fp8_scale_pitch(K);
    a.q = xq;
    a.scale = x_scale;
    launch_fp8_quant(a, x_dt, (M + 15) / 16, static_cast<hipStream_t>(stream));
    return launched();
}

int pdq_gemm_fp8_tile(int64_t M, int64_t N, int64_t K, pdq_scale_type scale_t) {
    if (M < 1 || N < 1 || !scale_ok(scale_t) || check_fp8_sizes(M, N, K) != PDQ_OK) return -1;
    return fp8_tile_shape(M, N, fp8_groups(K), scale_t == PDQ_SCALE_F32).rows;
}

pdq_status pdq_gemm_fp8(const uint8_t* xq, const uint8_t* x_scale, int64_t M, int64_t K, const uint8_t* wq,
                        const void* w_scale, pdq_scale_type scale_t, const float* bias, int64_t N, void* y,
                        pdq_dtype y_dt, int64_t ldy, void* stream) {
    PDQ_TRY(check_fp8_gemm(M, K, wq, w_scale, scale_t, bias, N, xq, x_scale, y, y_dt, ldy));
    if (M == 0 || N == 0) return PDQ_OK;
    const Fp8TileShape tile = fp8_tile_shape(M, N, fp8_groups(K), scale_t == PDQ_SCALE_F32);
    if (tile.rows > 0) {
        Fp8TileArgs t{};
        t.x = xq;
        t.xs = x_scale;
        t.w = wq;
        t.ws = w_scale;
        t.ws_f32 = scale_t == PDQ_SCALE_F32;
        t.M = (int)M;
        t.N = (int)N;
        t.groups = (int)fp8_groups(K);
        t.pitch = (int)fp8_scale_pitch(K);
        t.bias = bias;
        t.y = y;
        t.ldy = ldy;
        launch_fp8_tiles(t, y_dt, tile, static_cast<hipStream_t>(stream));
        return launched();
    }
    launch_fp8_rows(fp8_gemm_args(M, K, wq, w_scale, scale_t, bias, N, xq, x_scale, y, ldy), y_dt,
                    static_cast<hipStream_t>(stream));
    return launched();
}

size_t pdq_linear_fp8_workspace(int64_t M, int64_t K) {
    if (M < 1 || M > kMaxRows || K < 16 || K > kMaxK || K % 16 != 0 || M * K > kMaxValues || fp8_fusable(M, K)) return 0;
    return align256(pdq_fp8_bytes(M, K)) + align256((size_t)(M * fp8_scale_pitch(K)));
}

pdq_status pdq_linear_fp8(const void* x, pdq_dtype x_dt, int64_t M, int64_t K, int64_t ldx, const uint8_t* wq,
                          const void* w_scale, pdq_scale_type scale_t, const float* bias, int64_t N, void* y,
                          pdq_dtype y_dt, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(x_dt)) return PDQ_ERR_DTYPE;
    PDQ_TRY(check_operand(x, elem_bytes(x_dt), M, K, ldx));
    // (the codes' addresses are checked as the workspace's)
    const uint8_t* some = reinterpret_cast<const uint8_t*>(16);
    PDQ_TRY(check_fp8_gemm(M, K, wq, w_scale, scale_t, bias, N, some, some, y, y_dt, ldy));
    const size_t need = pdq_linear_fp8_workspace(M, K);
    if (need > 0 && (!workspace || workspace_bytes < need)) return PDQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PDQ_ERR_ALIGN;
    if (M == 0 || N == 0) return PDQ_OK;
    if (need == 0) {  // one launch
        Fp8GemmArgs a = fp8_gemm_args(M, K, wq, w_scale, scale_t, bias, N, nullptr, nullptr, y, ldy);
        a.raw = x;
        a.raw_dt = x_dt;
        a.K = (int)K;
        a.ldx = ldx;
        launch_fp8_rows(a, y_dt, static_cast<hipStream_t>(stream));
        return launched();
    }
    uint8_t* xq = static_cast<uint8_t*>(workspace);
    uint8_t* xs = xq + align256(pdq_fp8_bytes(M, K));
    PDQ_TRY(pdq_quantize_fp8(x, x_dt, M, K, ldx, xq, xs, stream));
    return pdq_gemm_fp8(xq, xs, M, K, wq, w_scale, scale_t, bias, N, y, y_dt, ldy, stream);
}

size_t pdq_route_workspace(int64_t tokens, int64_t experts) {
    if (tokens < 1 || tokens > kMaxRows || experts < 1 || experts > kMaxExperts) return 0;
    return align256(route_space(tokens, experts));
}

pdq_status pdq_route_experts(const void* logits, pdq_dtype dt, int64_t tokens, int64_t experts, int64_t ldl,
                             const float* bias, const pdq_route_rule* rule, int32_t* ids, float* weights,
                             int32_t* offsets, int32_t* rows, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dt)) return PDQ_ERR_DTYPE;
    if (!rule) return PDQ_ERR_NULL;
    if (tokens < 0 || tokens > kMaxRows || experts < 1 || experts > kMaxExperts || ldl < experts || ldl > kMaxValues)
        return PDQ_ERR_SHAPE;
    if (rule->k < 1 || rule->k > std::min(experts, kMaxChoices) || tokens * rule->k > kMaxSorted) return PDQ_ERR_SHAPE;
    if (rule->groups < 1 || rule->groups > 64 || experts % rule->groups != 0 || rule->top_groups < 1 ||
        rule->top_groups > rule->groups)
        return PDQ_ERR_SHAPE;
    if ((rule->score != PDQ_SOFTMAX && rule->score != PDQ_SIGMOID) || rule->group_score < 1 || rule->group_score > 2 ||
        !isfinite(rule->scale))
        return PDQ_ERR_UNSUPPORTED;
    if (!offsets || (tokens > 0 && (!logits || !ids || !weights || !rows))) return PDQ_ERR_NULL;
    if (!aligned(logits, elem_bytes(dt)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4) ||
        !aligned(offsets, 4) || !aligned(rows, 4))
        return PDQ_ERR_ALIGN;
    if (tokens > 0 && (!workspace || workspace_bytes < pdq_route_workspace(tokens, experts))) return PDQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PDQ_ERR_ALIGN;
    RouteArgs a{};
    a.logits = logits;
    a.dt = dt;
    a.ldl = ldl;
    a.bias = bias;
    a.tokens = (int)tokens;
    a.experts = (int)experts;
    a.k = rule->k;
    a.sigmoid = rule->score == PDQ_SIGMOID;
    a.renormalize = rule->renormalize != 0;
    a.groups = rule->groups;
    a.top_groups = rule->top_groups;
    a.group_score = rule->group_score;
    a.scale = rule->scale;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.rows = rows;
    a.hist = static_cast<int32_t*>(workspace);
    launch_route(a, static_cast<hipStream_t>(stream));
    return launched();
}

size_t pdq_experts_fp8_workspace(int64_t tokens, int64_t k, int64_t experts, int64_t hidden, int64_t inner) {
    if (tokens < 1 || !experts_sizes_ok(tokens, k, experts, hidden, inner)) return 0;
    return experts_space(tokens, k, experts, hidden, inner).all();
}

pdq_status pdq_experts_fp8(const void* x, pdq_dtype dt, int64_t ldx, const pdq_routing* routing,
                           const pdq_experts* experts, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                           void* stream) {
    if (dt != PDQ_BF16 && dt != PDQ_F16) return PDQ_ERR_DTYPE;
    if (!routing || !experts) return PDQ_ERR_NULL;
    if (!scale_ok(experts->scale_t)) return PDQ_ERR_DTYPE;
    const int64_t tokens = routing->tokens, k = routing->k, E = experts->experts, H = experts->hidden, I = experts->inner;
    if (routing->experts != E || !experts_sizes_ok(tokens, k, E, H, I)) return PDQ_ERR_SHAPE;
    PDQ_TRY(check_stack(2 * E, I, H));
    PDQ_TRY(check_stack(E, H, I));
    PDQ_TRY(check_operand(x, 2, tokens, H, ldx));
    if (ldy < H || ldy > kMaxValues) return PDQ_ERR_SHAPE;
    const int64_t blocks = fp8_blocks(tokens * k, E);
    if (blocks * std::max(fp8_groups(I), (H + 63) / 64) * 256 > kMaxThreads) return PDQ_ERR_SHAPE;
    if (!experts->gate_up || !experts->gate_up_scale || !experts->down || !experts->down_scale) return PDQ_ERR_NULL;
    if (!routing->offsets || (tokens > 0 && (!routing->ids || !routing->weights || !routing->rows || !y))) return PDQ_ERR_NULL;
    if (!aligned(experts->gate_up, 16) || !aligned(experts->down, 16) || !aligned(experts->gate_up_scale, 16) ||
        !aligned(experts->down_scale, 16) || !aligned(routing->ids, 4) || !aligned(routing->weights, 4) ||
        !aligned(routing->offsets, 4) || !aligned(routing->rows, 4) || !aligned(y, 8) || ldy % 4 != 0)
        return PDQ_ERR_ALIGN;
    const ExpertsSpace space = experts_space(tokens, k, E, H, I);
    if (tokens > 0 && (!workspace || workspace_bytes < space.all())) return PDQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PDQ_ERR_ALIGN;
    if (tokens == 0) return PDQ_OK;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    Fp8ExpertsArgs a{};
    a.sorted = Fp8Sorted{routing->offsets, routing->rows, (int)E, (int)k, (int)(tokens * k)};
    Fp8QuantArgs q{};
    q.x = x;
    q.ldx = ldx;
    q.M = tokens;
    q.K = (int)H;
    q.groups = (int)fp8_groups(H);
    q.pitch = (int)fp8_scale_pitch(H);
    q.q = ws;
    q.scale = ws + space.x;
    q.sorted = a.sorted;
    a.x = q.q;
    a.xs = q.scale;
    a.h = ws + space.x + space.xs;
    a.hs = a.h + space.h;
    a.partial = reinterpret_cast<float*>(a.hs + space.hs);
    a.gate_up = experts->gate_up;
    a.gate_up_s = experts->gate_up_scale;
    a.down = experts->down;
    a.down_s = experts->down_scale;
    a.ws_f32 = experts->scale_t == PDQ_SCALE_F32;
    a.hidden = (int)H;
    a.inner = (int)I;
    a.ids = routing->ids;
    a.weights = routing->weights;
    a.y = y;
    a.ldy = ldy;
    a.tokens = tokens;
    a.raw = x;
    a.ldx = ldx;
    if (fp8_experts_direct(tokens * k, k, H, I)) {
        launch_fp8_experts_direct(a, dt, static_cast<hipStream_t>(stream));
        return launched();
    }
    launch_fp8_quant(q, dt, blocks, static_cast<hipStream_t>(stream));
    launch_fp8_experts(a, dt, static_cast<hipStream_t>(stream));
    return launched();
}

}  // extern "C"

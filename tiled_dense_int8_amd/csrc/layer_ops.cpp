// C ABI entry points of the 8-bit layer operators: argument checks, choice of
// the kernel, launch.
#include <cmath>

#include "abi_common.h"
#include "quant_rows.h"

namespace tdi8 {
namespace {

int type_bytes(int type) { return type == TDI8_F32 ? 4 : type == TDI8_BF16 || type == TDI8_F16 ? 2 : 0; }

// The bytes of a strided window: rows x cols elements of `size` bytes.
struct Span {
    uintptr_t lo, hi;
};
Span span_of(const void *p, int64_t rows, int64_t cols, int64_t ld, int64_t size) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (!p || rows <= 0 || cols <= 0) return {lo, lo};
    return {lo, lo + static_cast<uintptr_t>(((rows - 1) * ld + cols) * size)};
}
bool meet(const Span &a, const Span &b) { return overlaps(a.lo, a.hi, b.lo, b.hi); }

const RowKernels *row_kernels(int type) {
    static const RowKernels *table = [] {
        static RowKernels k[3];
        register_rows_f32(&k[TDI8_F32]);
        register_rows_bf16(&k[TDI8_BF16]);
        register_rows_f16(&k[TDI8_F16]);
        return k;
    }();
    return &table[type];
}

constexpr int kMostColumns = 1 << 30;
constexpr int kBlock = 128;

// Checks of a row operator; lds is the leading dimension of the scales (1 for s8).
int check_rows(int op, int fmt, int type, const RowArgs &g) {
    const int64_t size = type_bytes(type);
    if (size == 0 || g.rows < 0 || g.cols < 0 || g.cols > kMostColumns) return TDI8_ERR_INVALID_VALUE;
    const int64_t least = g.cols > 1 ? g.cols : 1;
    const int64_t scales = fmt == kFmtS8 ? 1 : (g.cols + kBlock - 1) / kBlock;
    if (g.lda < least || g.ldq < least || (g.b && g.ldb < least) || (g.sum && g.ldsum < least) ||
        g.lds < (scales > 1 ? scales : 1))
        return TDI8_ERR_INVALID_VALUE;
    if (op == kOpNorm && !(g.eps >= 0.0f && std::isfinite(g.eps))) return TDI8_ERR_INVALID_VALUE;
    if (op == kOpNorm && g.sum && !g.b) return TDI8_ERR_INVALID_VALUE;
    if (g.rows == 0 || g.cols == 0) return TDI8_OK;
    if (!g.a || !g.q || !g.scale || (op == kOpNorm ? !g.weight : !g.b)) return TDI8_ERR_NULL_POINTER;
    if (!aligned(g.a, size) || !aligned(g.b, size) || !aligned(g.weight, size) || !aligned(g.sum, size) ||
        !aligned(g.scale, 4))
        return TDI8_ERR_INVALID_VALUE;
    const Span in[3] = {span_of(g.a, g.rows, g.cols, g.lda, size), span_of(g.b, g.rows, g.cols, g.ldb, size),
                        span_of(g.weight, 1, g.cols, g.cols, size)};
    const Span out[3] = {span_of(g.q, g.rows, g.cols, g.ldq, 1), span_of(g.scale, g.rows, scales, g.lds, 4),
                         span_of(g.sum, g.rows, g.cols, g.ldsum, size)};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 3; ++i) {
            const bool in_place = o == 2 && ((i == 0 && g.sum == g.a && g.ldsum == g.lda) ||
                                             (i == 1 && g.sum == g.b && g.ldsum == g.ldb));
            if (!in_place && meet(out[o], in[i])) return TDI8_ERR_ALIASING;
        }
        for (int i = 0; i < o; ++i)
            if (meet(out[o], out[i])) return TDI8_ERR_ALIASING;
    }
    return TDI8_OK;
}

int rows_entry(int op, int fmt, int type, RowArgs g, hipStream_t stream) {
    int st = check_rows(op, fmt, type, g);
    if (st != TDI8_OK) return st;
    if (g.rows == 0 || g.cols == 0) return TDI8_OK;
    int units = 0;
    st = device_units(&units);
    if (st != TDI8_OK) return st;
    // the smallest shape that keeps the row in registers, else the one that
    // reads it twice; f8 activations need only whole blocks of 128 columns
    // and take a row by blocks of at most kActShape
    int shape = g.cols < 8 ? 0 : 1;
    auto width = [](int s) { return kRowShape[s].threads * kRowShape[s].vectors * 8; };
    const bool apart = op == kOpAct && fmt == kFmtF8;
    while (shape > 0 && shape + 1 < kRowShapes && width(shape) < g.cols && !(apart && shape == kActShape)) ++shape;
    unsigned parts = apart && shape > 0 ? (g.cols + width(shape) - 1) / width(shape) : 1;
    if (parts > 65535) {  // the grid's limit
        shape = kRowShapes - 1;
        parts = 1;
    }
    const int per = rows_per_block(kRowShape[shape].threads);
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(g.rows) + per - 1) / per);
    void *args[] = {&g};
    const hipError_t e = hipLaunchKernel(row_kernels(type)->kernel[shape][op][fmt], dim3(blocks, parts),
                                         dim3(kRowShape[shape].threads * per), args, 0, stream);
    return e == hipSuccess ? TDI8_OK : hip_fail(e);
}

int norm_entry(int fmt, int type, int T, int H, const void *x, int ldx, const void *residual, int ldr,
               const void *weight, float eps, void *sum, int ldsum, void *q, int ldq, float *scale, int lds,
               hipStream_t stream) {
    RowArgs g{};
    g.a = x;
    g.b = residual;
    g.weight = weight;
    g.sum = sum;
    g.q = q;
    g.scale = scale;
    g.lda = ldx;
    g.ldb = ldr;
    g.ldsum = ldsum;
    g.ldq = ldq;
    g.lds = lds;
    g.rows = T;
    g.cols = H;
    g.eps = eps;
    return rows_entry(kOpNorm, fmt, type, g, stream);
}

int act_entry(int fmt, int type, int T, int N, const void *gate, int ldg, const void *up, int ldu, void *q,
              int ldq, float *scale, int lds, hipStream_t stream) {
    RowArgs g{};
    g.a = gate;
    g.b = up;
    g.q = q;
    g.scale = scale;
    g.lda = ldg;
    g.ldb = ldu;
    g.ldq = ldq;
    g.lds = lds;
    g.rows = T;
    g.cols = N;
    if (ldu < (N > 1 ? N : 1)) return TDI8_ERR_INVALID_VALUE;
    return rows_entry(kOpAct, fmt, type, g, stream);
}

}  // namespace
}  // namespace tdi8

using namespace tdi8;

extern "C" {

int rmsnorm_quant_s8(int type, int T, int H, const void *x, int ldx, const void *residual, int ldr,
                     const void *weight, float eps, void *sum, int ldsum, int8_t *q, int ldq, float *scale,
                     hipStream_t stream) {
    return norm_entry(kFmtS8, type, T, H, x, ldx, residual, ldr, weight, eps, sum, ldsum, q, ldq, scale, 1, stream);
}

int rmsnorm_quant_f8(int type, int T, int H, const void *x, int ldx, const void *residual, int ldr,
                     const void *weight, float eps, void *sum, int ldsum, uint8_t *q, int ldq, float *scale,
                     int lds, hipStream_t stream) {
    return norm_entry(kFmtF8, type, T, H, x, ldx, residual, ldr, weight, eps, sum, ldsum, q, ldq, scale, lds,
                      stream);
}

int swiglu_quant_s8(int type, int T, int N, const void *gate, int ldg, const void *up, int ldu, int8_t *q,
                    int ldq, float *scale, hipStream_t stream) {
    return act_entry(kFmtS8, type, T, N, gate, ldg, up, ldu, q, ldq, scale, 1, stream);
}

int swiglu_quant_f8(int type, int T, int N, const void *gate, int ldg, const void *up, int ldu, uint8_t *q,
                    int ldq, float *scale, int lds, hipStream_t stream) {
    return act_entry(kFmtF8, type, T, N, gate, ldg, up, ldu, q, ldq, scale, lds, stream);
}

}  // extern "C"

// C ABI entry points of the 8-bit layer operators: argument checks, choice of
// the kernel, launch.
#include <algorithm>
#include <climits>
#include <cmath>

#include "abi_common.h"
#include "product_table.h"
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
    const int threads = kRowShape[shape].threads * rows_per_block(kRowShape[shape].threads);
    const int per = rows_per_block(kRowShape[shape].threads);
    // a grid holds fewer than 2^32 threads: more rows take more launches
    const int64_t most = static_cast<int64_t>(INT_MAX / threads) * per;
    const int64_t size = type_bytes(type), rows = g.rows;
    const int64_t scales = fmt == kFmtS8 ? 1 : g.lds;
    const RowArgs all = g;
    for (int64_t first = 0; first < rows; first += most) {
        auto at = [&](const void *p, int64_t ld) {
            return p ? static_cast<const char *>(p) + first * ld * size : nullptr;
        };
        g.a = at(all.a, all.lda);
        g.b = at(all.b, all.ldb);
        g.sum = const_cast<char *>(at(all.sum, all.ldsum));
        g.q = static_cast<char *>(all.q) + first * all.ldq;
        g.scale = all.scale + first * scales;
        g.rows = static_cast<int>(std::min(rows - first, most));
        const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(g.rows) + per - 1) / per);
        void *args[] = {&g};
        const hipError_t e = hipLaunchKernel(row_kernels(type)->kernel[shape][op][fmt], dim3(blocks, parts),
                                             dim3(threads), args, 0, stream);
        if (e != hipSuccess) return hip_fail(e);
    }
    return TDI8_OK;
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

const ProductKernels *product_kernels(bool f8, int type) {
    static const ProductKernels *table = [] {
        static ProductKernels k[3];
        register_products_s8(&k[kProductS8]);
        register_products_f8(&k[kProductF8]);
        register_products_f8wide(&k[kProductF8Wide]);
        return k;
    }();
    return &table[product_type(f8, type)];
}

// LDS tile kernels of an operand type, in the order of lds_tiles.
struct TileKernels {
    const void *kernel[kLdsTiles];
};
const TileKernels &tile_kernels(bool f8, int type) {
    static const TileKernels *table = [] {
        static TileKernels t[3];
        register_grouped_tiles(t[kProductS8].kernel);
        register_f8_tiles(t[kProductF8].kernel);
        register_f8wide_tiles(t[kProductF8Wide].kernel);
        return t;
    }();
    return table[product_type(f8, type)];
}

// Checks of a scaled product; kb: scales of a row of A (1, or K's blocks of 128).
int check_product(bool f8, const ProductArgs &g) {
    const int64_t size = type_bytes(g.type);
    if (size == 0 || g.M < 0 || g.N < 0 || g.K < 0 || g.G < 0 || g.a_rows < 0 || g.M > kMostColumns ||
        g.N > kMostColumns || g.K > kMostColumns || g.G > kMostColumns)
        return TDI8_ERR_INVALID_VALUE;
    const int64_t kb = (static_cast<int64_t>(g.K) + kBlock - 1) / kBlock;
    const int64_t kmin = g.K > 1 ? g.K : 1;
    if (g.lda < kmin || g.ldb < kmin || g.ldc < (g.N > 1 ? g.N : 1)) return TDI8_ERR_INVALID_VALUE;
    if (f8 && (g.ldas < (kb > 1 ? kb : 1) || g.ldbs < (kb > 1 ? kb : 1))) return TDI8_ERR_INVALID_VALUE;
    if (!f8 && g.K > kMostK8) return TDI8_ERR_INVALID_VALUE;
    if (!g.offsets && g.G > 1) return TDI8_ERR_NULL_POINTER;
    if (!g.rows && g.a_rows < g.M) return TDI8_ERR_INVALID_VALUE;
    if (g.M == 0 || g.N == 0 || g.G == 0) return TDI8_OK;
    if (g.a_rows == 0) return TDI8_ERR_INVALID_VALUE;
    const int64_t b_bytes = (g.N - 1) * g.ldb + g.K;
    if (g.G > 1 && g.group_b < b_bytes) return TDI8_ERR_INVALID_VALUE;
    if (!g.C || (!f8 && (!g.a_scale || !g.b_scale))) return TDI8_ERR_NULL_POINTER;
    if (g.K > 0 && (!g.A || !g.B || !g.a_scale || !g.b_scale)) return TDI8_ERR_NULL_POINTER;
    if (!aligned(g.C, size) || !aligned(g.a_scale, 4) || !aligned(g.b_scale, 4) || !aligned(g.rows, 4) ||
        !aligned(g.offsets, 4))
        return TDI8_ERR_INVALID_VALUE;
    const int64_t nb = (static_cast<int64_t>(g.N) + kBlock - 1) / kBlock;
    const Span c = span_of(g.C, g.M, g.N, g.ldc, size);
    const Span in[6] = {
        span_of(g.A, g.a_rows, g.K, g.lda, 1),
        g.K > 0 ? span_of(g.B, g.G, b_bytes, g.group_b, 1) : Span{0, 0},
        f8 ? span_of(g.a_scale, g.M, kb, g.ldas, 4) : span_of(g.a_scale, 1, g.a_rows, 1, 4),
        f8 ? span_of(g.b_scale, nb, kb, g.ldbs, 4) : span_of(g.b_scale, g.G, g.N, g.N, 4),
        span_of(g.rows, 1, g.M, 1, 4),
        span_of(g.offsets, 1, static_cast<int64_t>(g.G) + 1, 1, 4),
    };
    for (const Span &s : in)
        if (meet(c, s)) return TDI8_ERR_ALIASING;
    return TDI8_OK;
}

int product_entry(bool f8, ProductArgs g, hipStream_t stream) {
    int st = check_product(f8, g);
    if (st != TDI8_OK) return st;
    if (g.M == 0 || g.N == 0 || g.G == 0) return TDI8_OK;
    int units = 0;
    st = device_units(&units);
    if (st != TDI8_OK) return st;
    const bool al = aligned(g.A, 16) && aligned(g.B, 16) && g.lda % 16 == 0 && g.ldb % 16 == 0 && g.K % 16 == 0 &&
                    (g.G == 1 || g.group_b % 16 == 0);
    const bool near = !f8 || (256 * std::max(g.lda, g.ldb) + g.K < INT_MAX && 4 * (256 * g.ldas + g.K) < INT_MAX);
    ProductChoice c{};
    if (!choose_product(f8, g.type, g.G, g.M, g.N, g.K, al, near, units, &c)) return TDI8_ERR_INVALID_VALUE;
    g.tiles_m = c.tiles_m;
    g.tiles_n = c.tiles_n;
    // an empty sum is zero, whatever its scales: no row counts as inside A
    if (g.K == 0) g.a_rows = 0;
    const ProductKernels &pk = *product_kernels(f8, g.type);
    const void *kernel = c.form == TDI8_SCALED_STREAM             ? pk.stream[c.index]
                         : c.form == TDI8_SCALED_STREAM_UNALIGNED ? (c.index == kGroupStream ? pk.unaligned_group
                                                                                             : pk.unaligned[c.index])
                         : c.form == TDI8_SCALED_LDS              ? tile_kernels(f8, g.type).kernel[c.index]
                                                                  : pk.staged;
    void *args[] = {&g};
    const hipError_t e = hipLaunchKernel(kernel, dim3(static_cast<unsigned>(c.blocks)),
                                         dim3(static_cast<unsigned>(c.threads)), args, 0, stream);
    return e == hipSuccess ? TDI8_OK : hip_fail(e);
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

int gemm_s8s8_grouped(int type, int G, int M, int N, int K, const int8_t *A, int lda, int a_rows,
                      const float *a_scale, const int32_t *rows, const int32_t *offsets, const int8_t *B, int ldb,
                      int64_t group_b, const float *b_scale, void *C, int ldc, hipStream_t stream) {
    ProductArgs g{};
    g.A = A;
    g.B = B;
    g.C = C;
    g.a_scale = a_scale;
    g.b_scale = b_scale;
    g.rows = rows;
    g.offsets = offsets;
    g.lda = lda;
    g.ldb = ldb;
    g.ldc = ldc;
    g.group_b = group_b;
    g.M = M;
    g.N = N;
    g.K = K;
    g.G = G;
    g.a_rows = a_rows;
    g.type = type;
    return product_entry(false, g, stream);
}

int gemm_f8f8_block128(int type, int M, int N, int K, const uint8_t *A, int lda, const float *a_scale, int ldas,
                       const uint8_t *B, int ldb, const float *b_scale, int ldbs, void *C, int ldc,
                       hipStream_t stream) {
    ProductArgs g{};
    g.A = reinterpret_cast<const int8_t *>(A);
    g.B = reinterpret_cast<const int8_t *>(B);
    g.C = C;
    g.a_scale = a_scale;
    g.b_scale = b_scale;
    g.lda = lda;
    g.ldb = ldb;
    g.ldc = ldc;
    g.ldas = ldas;
    g.ldbs = ldbs;
    g.M = M;
    g.N = N;
    g.K = K;
    g.G = 1;
    g.a_rows = M;
    g.type = type;
    return product_entry(true, g, stream);
}

}  // extern "C"

// Arguments of the kernels that turn rows of activations into 8-bit operands
// with scales (quant_rows_kernel.h), and their table by type, row shape,
// operator and format.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace tdi8 {

struct RowArgs {
    const void *a, *b;     // x and the residual (or null); gate and up
    const void *weight;    // norm only
    void *sum;             // norm: where a + b goes, or null
    void *q;               // 8-bit rows
    float *scale;          // one per row, or one per row and block of 128 columns
    int64_t lda, ldb, ldsum, ldq, lds;
    int rows, cols;
    float eps;
};

// Row shapes: threads per row times vectors of 8 columns that a thread keeps
// in registers.  The first (vectors < 0) takes rows shorter than 8 columns,
// the last (0) keeps none and reads the row twice.
enum { kRowShapes = 9 };
struct RowShape {
    int threads, vectors;
};
constexpr RowShape kRowShape[kRowShapes] = {{64, -1}, {64, 1},  {256, 1}, {256, 2}, {256, 3},
                                            {256, 4}, {512, 3}, {512, 4}, {1024, 0}};
// f8 activations, which need no whole row, take a longer one by blocks of this
// shape (8192 x 11008 bf16: 102 us; by {256, 2} 106, by {256, 1} 118, one block
// of 1024 threads per row 163).
constexpr int kActShape = 4;  // {256, 3}
// Rows that one block computes: the one-wave shape puts four in a block.
constexpr int rows_per_block(int threads) { return threads == 64 ? 4 : 1; }

enum { kOpNorm = 0, kOpAct = 1 };
enum { kFmtS8 = 0, kFmtF8 = 1 };

struct RowKernels {
    const void *kernel[kRowShapes][2][2];  // [shape][operator][format]
};
void register_rows_f32(RowKernels *k);
void register_rows_bf16(RowKernels *k);
void register_rows_f16(RowKernels *k);

}  // namespace tdi8

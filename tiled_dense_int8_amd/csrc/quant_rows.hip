// Instantiates quant_rows_kernel for one type (TDI8_ROWS_TYPE, set on the
// compiler command line: F32, Bf16 or F16) and registers its entry points.
#include "quant_rows_kernel.h"

#ifndef TDI8_ROWS_TYPE
#error "TDI8_ROWS_TYPE must name a type and TDI8_ROWS_REGISTER its registration function"
#endif

namespace tdi8 {

template <int S, int OP, int FMT>
static const void *row_entry() {
    return reinterpret_cast<const void *>(
        &quant_rows_kernel<TDI8_ROWS_TYPE, kRowShape[S].threads, kRowShape[S].vectors, OP, FMT>);
}

template <int S>
static void register_shape(RowKernels *k) {
    k->kernel[S][kOpNorm][kFmtS8] = row_entry<S, kOpNorm, kFmtS8>();
    k->kernel[S][kOpNorm][kFmtF8] = row_entry<S, kOpNorm, kFmtF8>();
    k->kernel[S][kOpAct][kFmtS8] = row_entry<S, kOpAct, kFmtS8>();
    k->kernel[S][kOpAct][kFmtF8] = row_entry<S, kOpAct, kFmtF8>();
    if constexpr (S + 1 < kRowShapes) register_shape<S + 1>(k);
}

void TDI8_ROWS_REGISTER(RowKernels *k) { register_shape<0>(k); }

}  // namespace tdi8

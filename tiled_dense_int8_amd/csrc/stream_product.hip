// Instantiates the stream kernels of one operand type (TDI8_PRODUCT_TYPE, set on
// the compiler command line: S8, F8 or F8Wide) and registers the type's kernels.
#include "product_table.h"
#include "staged_product.h"

#ifndef TDI8_PRODUCT_TYPE
#error "TDI8_PRODUCT_TYPE must name an operand type and TDI8_PRODUCT_REGISTER its registration function"
#endif

namespace tdi8 {

template <int T>
static void register_stream(ProductKernels *k) {
    constexpr StreamTile t = kStreamTile[T];
    k->stream[T][0] = reinterpret_cast<const void *>(
        &stream_product_kernel<TDI8_PRODUCT_TYPE, t.bm / 16, t.bn / 16, t.waves, t.batch, false>);
    k->stream[T][1] = reinterpret_cast<const void *>(
        &stream_product_kernel<TDI8_PRODUCT_TYPE, t.bm / 16, t.bn / 16, t.waves, t.batch, true>);
    if constexpr (T + 1 < kStreamTiles) register_stream<T + 1>(k);
}

void TDI8_PRODUCT_REGISTER(ProductKernels *k) {
    register_stream<0>(k);
    k->staged = reinterpret_cast<const void *>(&staged_product_kernel<TDI8_PRODUCT_TYPE, 2, 4, 2, 2>);
}

}  // namespace tdi8

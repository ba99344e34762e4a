// Instantiates the stream kernels and the kernels for unaligned operands of one
// operand type (TDI8_PRODUCT_TYPE, set on the compiler command line: S8, F8 or
// F8Wide) and registers them.
#include "product_table.h"
#include "staged_product.h"
#include "stream_product.h"
#include "unaligned_stream.h"

#ifndef TDI8_PRODUCT_TYPE
#error "TDI8_PRODUCT_TYPE must name an operand type and TDI8_PRODUCT_REGISTER its registration function"
#endif

namespace tdi8 {

template <int T>
static void register_stream(ProductKernels *k) {
    constexpr Tile t = kStreamTile[T];
    k->stream[T] = reinterpret_cast<const void *>(&stream_product_kernel<TDI8_PRODUCT_TYPE, t.bm, t.bn, t.threads / 64>);
    if constexpr (T + 1 < kStreamTiles) register_stream<T + 1>(k);
}
template <int T>
static void register_unaligned(ProductKernels *k) {
    constexpr UnalignedStreamTile t = kUnalignedStreamTile[T];
    k->unaligned_stream[T] = reinterpret_cast<const void *>(
        &unaligned_stream_kernel<TDI8_PRODUCT_TYPE, t.bm / 16, t.bn / 16, t.waves, t.batch>);
    if constexpr (T + 1 < kUnalignedStreamTiles) register_unaligned<T + 1>(k);
}

void TDI8_PRODUCT_REGISTER(ProductKernels *k) {
    register_stream<0>(k);
    register_unaligned<0>(k);
    constexpr int MT = kStagedRows / 32, NT = kStagedColumns / 64;
    static_assert(kStagedThreads == 2 * 4 * 64, "two waves by four");
    k->staged = reinterpret_cast<const void *>(&staged_product_kernel<TDI8_PRODUCT_TYPE, 2, 4, MT, NT>);
}

}  // namespace tdi8

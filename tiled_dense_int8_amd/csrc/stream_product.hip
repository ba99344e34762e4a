// Instantiates the stream kernels and the kernels for unaligned operands of one
// operand type (TDI8_PRODUCT_TYPE, set on the compiler command line: S8, F8 or
// F8Wide) and registers them.
#include "product_table.h"
#include "staged_product.h"
#include "stream_product.h"

#ifndef TDI8_PRODUCT_TYPE
#error "TDI8_PRODUCT_TYPE must name an operand type and TDI8_PRODUCT_REGISTER its registration function"
#endif

namespace tdi8 {

template <int T>
static void register_stream(ProductKernels *k) {
    constexpr Tile t = kStreamTile[T];
    k->stream[T] = reinterpret_cast<const void *>(
        &stream_product_kernel<TDI8_PRODUCT_TYPE, t.bm, t.bn, t.threads / 64, true>);
    if constexpr (T + 1 < kStreamTiles) register_stream<T + 1>(k);
}
template <int T>
static void register_unaligned(ProductKernels *k) {
    constexpr Tile t = kUnalignedTile[T];
    k->unaligned[T] = reinterpret_cast<const void *>(
        &stream_product_kernel<TDI8_PRODUCT_TYPE, t.bm, t.bn, t.threads / 64, false>);
    if constexpr (T + 1 < kUnalignedStreams) register_unaligned<T + 1>(k);
}

void TDI8_PRODUCT_REGISTER(ProductKernels *k) {
    register_stream<0>(k);
    register_unaligned<0>(k);
    constexpr Tile t = kStreamTile[kGroupStream], s = kStagedTile[0];
    k->unaligned_group = reinterpret_cast<const void *>(
        &stream_product_kernel<TDI8_PRODUCT_TYPE, t.bm, t.bn, t.threads / 64, false>);
    static_assert(s.threads == 2 * 4 * 64, "two waves by four");
    k->staged = reinterpret_cast<const void *>(&staged_product_kernel<TDI8_PRODUCT_TYPE, 2, 4, s.bm / 32, s.bn / 64>);
}

}  // namespace tdi8

// Kernels of the scaled products, by operand type and tile.
#pragma once

#include "scaled_product.h"

namespace tdi8 {

// Row tiles of the stream kernels: 16, 32 and 64 rows.
enum { kStreamTiles = 3 };
struct StreamTile {
    int bm, bn, waves;
};
constexpr StreamTile kStreamTile[kStreamTiles] = {{16, 16, 4}, {32, 32, 4}, {64, 64, 4}};

// Tiles of the kernels that stage both operands in LDS, smallest first.
enum { kLdsTiles = 3 };
struct LdsTile {
    int bm, bn, threads;
};
constexpr LdsTile kGroupedTile[kLdsTiles] = {{64, 128, 512}, {128, 128, 256}, {256, 256, 512}};

struct ProductKernels {
    const void *stream[kStreamTiles][2];  // [tile][aligned]
};
void register_grouped_tiles(const void **k);  // kLdsTiles kernels
void register_products_s8(ProductKernels *k);
void register_products_f8(ProductKernels *k);
void register_products_f8wide(ProductKernels *k);

}  // namespace tdi8

// Kernels of the scaled products, by operand type and tile.
#pragma once

#include "scaled_product.h"

#ifndef TB
#define TB 128, 256, 512
#endif
namespace tdi8 {

// Row tiles of the stream kernels: 16, 32 and 64 rows.
#ifdef MANY
enum { kStreamTiles = 14 };
#else
enum { kStreamTiles = 3 };
#endif
struct StreamTile {
    int bm, bn, waves, batch;
};
#ifdef MANY
constexpr StreamTile kStreamTile[kStreamTiles] = {{16,16,4,4}, {16,16,4,8}, {16,16,8,4}, {16,16,16,2}, {32,16,8,2}, {32,16,8,4}, {32,32,4,2}, {32,32,8,2}, {32,32,4,4}, {64,16,8,2}, {64,32,4,1}, {64,32,8,1}, {64,32,8,2}, {64,64,4,1}};
#else
constexpr StreamTile kStreamTile[kStreamTiles] = {{16, 16, 4, 4}, {32, 32, 4, 2}, {64, 64, 4, 1}};
#endif

// Tiles of the kernels that stage both operands in LDS, smallest first.
enum { kLdsTiles = 3 };
struct LdsTile {
    int bm, bn, threads;
};
constexpr LdsTile kGroupedTile[kLdsTiles] = {{64, 128, 512}, {TB}, {256, 256, 512}};

constexpr LdsTile kF8Tile[kLdsTiles] = {{64, 128, 256}, {128, 128, 256}, {256, 256, 512}};
constexpr LdsTile kF8WideTile[kLdsTiles] = {{64, 128, 256}, {128, 128, 256}, {128, 128, 512}};

struct ProductKernels {
    const void *stream[kStreamTiles][2];  // [tile][aligned]
};
void register_grouped_tiles(const void **k);  // kLdsTiles kernels each
void register_f8_tiles(const void **k);
void register_f8wide_tiles(const void **k);
void register_products_s8(ProductKernels *k);
void register_products_f8(ProductKernels *k);
void register_products_f8wide(ProductKernels *k);

}  // namespace tdi8

// Kernels of the scaled products, by operand type and tile.
#pragma once

#include "scaled_product.h"

namespace tdi8 {

// Stream kernels (stream_product.h): block tile, waves sharing K, chunks that
// a wave loads at once.
enum { kStreamTiles = 6 };
struct StreamTile {
    int bm, bn, waves, batch;
};
constexpr StreamTile kStreamTile[kStreamTiles] = {
    {16, 16, 4, 4}, {16, 16, 8, 4}, {16, 32, 4, 2}, {32, 16, 8, 2}, {32, 32, 4, 2}, {64, 32, 8, 1}};

// Tiles of the kernels that stage both operands in LDS, and what they were
// measured to take: a round of `per_cu` blocks on every compute unit costs
// fixed + per_4096 * K / 4096 microseconds.
struct LdsTile {
    int bm, bn, threads;
    int per_cu;
    float fixed, per_4096;
};
enum { kLdsTiles = 4 };
constexpr LdsTile kGroupedTile[kLdsTiles] = {
    {64, 128, 512, 1, 2.5f, 14.0f}, {128, 256, 512, 1, 8.0f, 31.0f}, {256, 256, 512, 1, 12.0f, 58.0f}, {}};
constexpr LdsTile kF8Tile[kLdsTiles] = {{64, 128, 256, 1, 6.0f, 16.0f},
                                        {128, 128, 256, 1, 7.0f, 24.0f},
                                        {128, 128, 256, 2, 9.0f, 34.0f},
                                        {256, 256, 512, 1, 12.0f, 58.0f}};
constexpr LdsTile kF8WideTile[kLdsTiles] = {{64, 128, 256, 1, 7.0f, 20.0f},
                                            {128, 128, 256, 1, 8.0f, 34.0f},
                                            {128, 128, 256, 2, 10.0f, 55.0f},
                                            {}};
// Tile of the kernel for unaligned operands (staged_product.h).
constexpr LdsTile kStagedTile = {64, 128, 512, 1, 0.0f, 0.0f};

struct ProductKernels {
    const void *stream[kStreamTiles][2];  // [tile][aligned]
    const void *staged;
};
void register_products_s8(ProductKernels *k);
void register_products_f8(ProductKernels *k);
void register_products_f8wide(ProductKernels *k);
// The LDS tile kernels of each type, as in its table.
void register_grouped_tiles(const void **k);
void register_f8_tiles(const void **k);
void register_f8wide_tiles(const void **k);

}  // namespace tdi8

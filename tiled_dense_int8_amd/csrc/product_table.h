// Kernels of the scaled products, by operand type and tile.
#pragma once

#include "scaled_product.h"

namespace tdi8 {

// Tiles of a kernel, and what a product of them was measured to take: start
// microseconds, and for each round of `per_cu` blocks on every compute unit
// fixed + per_4096 * K / 4096.
struct Tile {
    int bm, bn, threads;
    int per_cu;
    float start, fixed, per_4096;
};

// The kernels that stage both operands in LDS.
enum { kLdsTiles = 4 };
constexpr Tile kGroupedTile[kLdsTiles] = {{64, 128, 512, 1, 0.0f, 2.5f, 14.0f},
                                          {128, 256, 512, 1, 0.0f, 8.0f, 31.0f},
                                          {256, 256, 512, 1, 0.0f, 12.0f, 58.0f},
                                          {}};
constexpr Tile kF8Tile[kLdsTiles] = {{64, 128, 256, 1, 0.0f, 6.0f, 16.0f},
                                     {128, 128, 256, 1, 0.0f, 7.0f, 24.0f},
                                     {128, 128, 256, 2, 0.0f, 9.0f, 34.0f},
                                     {256, 256, 512, 1, 0.0f, 12.0f, 58.0f}};
constexpr Tile kF8WideTile[kLdsTiles] = {{64, 128, 256, 1, 0.0f, 7.0f, 20.0f},
                                         {128, 128, 256, 1, 0.0f, 8.0f, 34.0f},
                                         {128, 128, 256, 2, 0.0f, 10.0f, 55.0f},
                                         {}};

// The stream kernels (stream_product.h); the types differ by less than the
// steps from tile to tile.  The last one is for groups of few rows and chosen
// by a rule of its own.
enum { kStreamTiles = 7, kGroupStream = 6 };
constexpr Tile kStreamTile[kStreamTiles] = {{8, 16, 512, 1, 3.0f, 0.1f, 1.75f},  {16, 16, 512, 1, 3.0f, 0.1f, 1.75f},
                                            {32, 16, 512, 1, 2.9f, 0.2f, 2.45f}, {32, 32, 512, 1, 2.7f, 0.4f, 3.5f},
                                            {32, 64, 512, 1, 1.5f, 1.9f, 5.3f},  {64, 64, 512, 1, 1.5f, 2.6f, 8.4f},
                                            {16, 32, 256, 1, 0.0f, 0.0f, 0.0f}};

// The kernels for unaligned operands: the streams of these tiles (64 x 64 has
// too few registers for that), and tiles staged through registers
// (staged_product.h; the same kernel with one block on a compute unit or two).
enum { kUnalignedStreams = 5, kStagedTiles = 2 };
constexpr Tile kUnalignedTile[kUnalignedStreams] = {{8, 16, 512, 1, 3.0f, 0.2f, 3.3f},
                                                    {16, 16, 512, 1, 3.0f, 0.2f, 4.0f},
                                                    {32, 16, 512, 1, 2.9f, 0.6f, 5.4f},
                                                    {32, 32, 512, 1, 2.7f, 1.4f, 7.6f},
                                                    {32, 64, 512, 1, 0.0f, 4.5f, 11.0f}};
constexpr Tile kStagedTile[kStagedTiles] = {{64, 128, 512, 1, 0.0f, 2.2f, 46.0f}, {64, 128, 512, 2, 0.0f, 3.2f, 54.0f}};

struct ProductKernels {
    const void *stream[kStreamTiles];
    const void *unaligned[kUnalignedStreams], *unaligned_group;
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

// Kernels of the scaled products, by operand type and tile, and the choice
// between them.
#pragma once

#include "../../include/tdi8.h"
#include "scaled_product.h"

namespace tdi8 {

// Tiles of a kernel, and what a product of them was measured to take: start
// microseconds, and for each round of `per_cu` blocks on every compute unit
// fixed + per_4096 * K / 4096.  They rank the tiles of one product; they do not
// foretell its time, having no term for bytes from HBM (8 groups of 32 rows,
// 28672 x 4096 int8: 115 us by the table, 182 for reading B) nor for what long
// sums gain (4096 x 4096 x 4095 e4m3, staged: 229 us by the table, 172 measured).
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

// Operand types of the kernels.  e4m3 products take the matrix instruction's
// own sums for bf16 results only: they can be off by half a step of fp16
// (operand_types.h).  With fp16 and fp32 results e4m3 is widened (4096^3 127
// us to fp16, 71 to bf16; 256 x 4096 x 4096 14.1 and 11.6, 16 rows 5.4 and 5.2).
enum { kProductS8 = 0, kProductF8 = 1, kProductF8Wide = 2 };
inline int product_type(bool f8, int type) {
    return !f8 ? kProductS8 : type == TDI8_BF16 ? kProductF8 : kProductF8Wide;
}
// The LDS tiles of an operand type (those with threads).
inline const Tile *lds_tiles(bool f8, int type) {
    const Tile *tiles[] = {kGroupedTile, kF8Tile, kF8WideTile};
    return tiles[product_type(f8, type)];
}

// Sizes stay this far from the end of int, so that a kernel may round one up
// to its tile; a sum of kMostK8 products of int8 cannot wrap an int32.
constexpr int kMostColumns = 1 << 30;
constexpr int kMostK8 = 131071;

// How a scaled product runs: a form (tdi8_scaled_form) and its entry in that
// form's table, the tile, the row tiles (a bound, whatever the groups' sizes),
// the column tiles and the blocks of the grid.
struct ProductChoice {
    int form, index;
    int bm, bn, threads;
    int tiles_m, tiles_n;
    int64_t blocks;
};
// al: operands on 16 bytes; near: they fit the buffer addresses of the LDS
// tiles.  M, N, G > 0.  False if no tile's grid can be launched (2^31 threads).
bool choose_product(bool f8, int type, int64_t G, int64_t M, int64_t N, int64_t K, bool al, bool near, int units,
                    ProductChoice *out);

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

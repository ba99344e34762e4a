// The choice of a scaled product's kernel, on described hardware: nothing here
// touches a device.
#include <algorithm>
#include <climits>

#include "product_table.h"

namespace tdi8 {

bool choose_product(bool f8, int type, int64_t G, int64_t M, int64_t N, int64_t K, bool al, bool near, int units,
                    ProductChoice *out) {
    // The choice goes by the sizes alone: how the rows fall to the groups is
    // known to the device only.
    const int64_t groups = G < M ? G : M;  // that can have rows
    const int64_t rows = (M + groups - 1) / groups;
    // row tiles of height bm: half a tile of each group is lost on average
    auto expected = [&](int bm, int bn) {
        const int64_t m = groups == 1 ? (M + bm - 1) / bm : std::max<int64_t>(groups, M / bm + groups / 2);
        return m * ((N + bn - 1) / bn);
    };
    // Takes a tile if one grid holds its blocks: every group that has rows ends
    // in at most one partial tile.
    auto take = [&](int form, int index, const Tile &t) {
        const int64_t tm = (M + groups * (t.bm - 1)) / t.bm;
        const int64_t tn = (N + t.bn - 1) / t.bn;
        if (tm > INT_MAX || tm * tn > INT_MAX / t.threads - 8) return false;
        *out = {form, index, t.bm, t.bn, t.threads, static_cast<int>(tm), static_cast<int>(tn),
                (tm * tn + 7) / 8 * 8};
        return true;
    };
    const int64_t lds = expected(64, 128);
    // Groups of few rows: most row tiles hold few, so that B is read once
    // (int8: 256 groups of 2 rows on average, 1024 x 2048: 86 us, by LDS
    // tiles 118; 64 of 2, 2048 x 4096: 85 and 78; 8 of 16, 1024 x 4096: 10.4
    // and 18.8; 8 of 8, 4096 x 4096, where many have two row tiles: 33 and 27.6).
    if (groups > 1 && (rows <= 2 || (rows <= 32 && lds < units)) &&
        take(al ? TDI8_SCALED_STREAM : TDI8_SCALED_STREAM_UNALIGNED, kGroupStream, kStreamTile[kGroupStream]))
        return true;
    // the least of the tiles' measured costs; equal ones to the first
    float best = 0.0f;
    bool taken = false;
    auto weigh = [&](int form, int index, const Tile &t) {
        const int64_t round = static_cast<int64_t>(units) * t.per_cu;
        const int64_t rounds = (expected(t.bm, t.bn) + round - 1) / round;
        const float cost = t.start + rounds * (t.fixed + t.per_4096 * K / 4096.0f);
        if ((taken && cost >= best) || !take(form, index, t)) return;
        best = cost;
        taken = true;
    };
    // Streams while the LDS tiles leave compute units idle (512 x 4096 x
    // 4096 e4m3, 256 of those: 25 us against 22) or where B is all there is
    // to read (8 x 32768 x 4096: 25 against 28.6); no tile of twice the rows.
    const Tile *streams = al ? kStreamTile : kUnalignedTile;
    if (lds < units || rows <= 8)
        for (int i = 0; i < (al ? +kGroupStream : +kUnalignedStreams); ++i)
            if (streams[i].bm < 2 * rows || i == 0)
                weigh(al ? TDI8_SCALED_STREAM : TDI8_SCALED_STREAM_UNALIGNED, i, streams[i]);
    if (al && near) {
        const Tile *tile = lds_tiles(f8, type);
        for (int i = 0; i < kLdsTiles && tile[i].threads; ++i) weigh(TDI8_SCALED_LDS, i, tile[i]);
    } else {
        for (int i = 0; i < kStagedTiles; ++i) weigh(TDI8_SCALED_STAGED, i, kStagedTile[i]);
    }
    return taken;
}

}  // namespace tdi8

using namespace tdi8;

extern "C" int scaled_product_plan(int f8, int type, int G, int M, int N, int K, int is_aligned, int num_cu,
                                   tdi8_scaled_plan *out) {
    if (!out) return TDI8_ERR_NULL_POINTER;
    *out = tdi8_scaled_plan{};
    if (type < TDI8_F32 || type > TDI8_F16 || G < 0 || M < 0 || N < 0 || K < 0 || num_cu < 1 || (f8 && G > 1) ||
        G > kMostColumns || M > kMostColumns || N > kMostColumns || K > (f8 ? kMostColumns : kMostK8))
        return TDI8_ERR_INVALID_VALUE;
    if (G == 0 || M == 0 || N == 0) return TDI8_OK;
    ProductChoice c{};
    if (!choose_product(f8 != 0, type, G, M, N, K, is_aligned != 0, true, num_cu, &c)) return TDI8_ERR_INVALID_VALUE;
    out->form = c.form;
    out->block_m = c.bm;
    out->block_n = c.bn;
    out->threads = c.threads;
    out->blocks = c.blocks;
    return TDI8_OK;
}

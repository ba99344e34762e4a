// Products of 8-bit operands with their scales: int8 grouped by expert and
// e4m3 with a scale for each block of 128.  Arguments, the search for a
// block's rows, and the rounded store that the kernels share.
#pragma once

#include "device_common.h"

namespace tdi8 {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;

struct ProductArgs {
    const int8_t *A, *B;  // int8 or e4m3 bytes, K contiguous
    void *C;
    const float *a_scale, *b_scale;
    const int32_t *rows;     // A's row of each C row, or null: its own
    const int32_t *offsets;  // G + 1 ends of the groups' rows, or null: one group of all
    int64_t lda, ldb, ldc;
    int64_t group_b;         // bytes from one group's B to the next
    int64_t ldas, ldbs;      // e4m3: leading dimensions of the scales
    int M, N, K, G;          // M: rows of C
    int a_rows;              // rows of A (entries of `rows` outside give rows of zeros)
    int type;                // tdi8_type of C
    int tiles_m, tiles_n;    // tiles of the grid: tiles_m bounds the groups' row tiles
};

// The rows [m0, m0 + BM) within one group, [begin, end).
struct RowTile {
    int group, m0, begin, end;
    int turn;  // the K tile to start with (mod their number), where that is free
};

// Row tile `tile` of the groups' tiles in order (ceil(rows / BM) for each
// group), and how many there are.  Every wave searches by itself: 64 offsets a
// step, a prefix sum over the lanes.  Offsets are clamped to [0, M] and to
// rising order within each group, so that no value of theirs leads outside C;
// groups that overlap all the same could count past any bound, so the sums
// stop at kMostTiles (at most M + G <= 2^31 tiles of at least a row are asked
// for, of which disjoint groups have at most 2^30).
constexpr uint32_t kMostTiles = 1u << 30;
__device__ __forceinline__ bool find_rows(const ProductArgs &g, int bm, int tile, RowTile &out, int *count) {
    if (!g.offsets) {
        const int tiles = (g.M + bm - 1) / bm;
        if (count) *count = tiles;
        out = {0, tile * bm, 0, g.M, 0};
        return tile >= 0 && tile < tiles;
    }
    const int lane = threadIdx.x & 63;
    uint32_t before = 0;
    bool found = tile < 0;
    for (int base = 0; base < g.G; base += 64) {
        const int e = base + lane;
        int lo = 0, hi = 0;
        if (e < g.G) {
            lo = min(max(g.offsets[e], 0), g.M);
            hi = min(max(g.offsets[e + 1], lo), g.M);
        }
        const uint32_t tiles = static_cast<uint32_t>(hi - lo + bm - 1) / bm;
        uint32_t sum = tiles;
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const uint32_t o = static_cast<uint32_t>(__shfl_up(static_cast<int>(sum), s));
            if (lane >= s) sum = min(sum + o, kMostTiles);
        }
        const uint32_t total = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(sum), 63));
        if (!found && static_cast<uint32_t>(tile) < before + total) {
            const int l = __builtin_ctzll(__ballot(before + sum > static_cast<uint32_t>(tile)));
            const int first = static_cast<int>(before) + __builtin_amdgcn_readlane(static_cast<int>(sum - tiles), l);
            out.group = base + l;
            out.begin = __builtin_amdgcn_readlane(lo, l);
            out.m0 = out.begin + (tile - first) * bm;
            out.end = __builtin_amdgcn_readlane(hi, l);
            if (!count) return true;
            found = true;
        }
        before = min(before + total, kMostTiles);
    }
    if (count) *count = static_cast<int>(before);
    return found && tile >= 0;
}

// Position of block `bid` among `total` that are dealt out so that each XCD
// (blocks go to the 8 XCDs in turn) takes one run of consecutive positions;
// total or more if it has none.  Launched in multiples of 8.
__device__ __forceinline__ int64_t xcd_run(int64_t bid, int64_t total) {
    const int64_t per = (total + 7) >> 3;
    const int64_t at = bid >> 3;
    return at < per ? (bid & 7) * per + at : total;
}

// A's row of C row m: its own or rows[m], or -1 for an entry outside A.
__device__ __forceinline__ int a_row(const ProductArgs &g, int m) {
    const int r = g.rows ? g.rows[m] : m;
    return static_cast<unsigned>(r) < static_cast<unsigned>(g.a_rows) ? r : -1;
}

// Four consecutive values of row m from column n on, rounded to C's type
// (once, to nearest even); columns past N are left out.  STREAM: with the
// non-temporal hint, where a wave's stores cover whole lines.
template <bool STREAM = false>
__device__ __forceinline__ void store_row4(const ProductArgs &g, int64_t m, int n, f32x4 v) {
    const int64_t at = m * g.ldc + n;
    const int left = g.N - n;
    if (g.type == 0) {
        float *p = static_cast<float *>(g.C) + at;
        typedef f32x4 f32x4_a4 __attribute__((aligned(4)));
        if (left >= 4) {
            if (STREAM)
                __builtin_nontemporal_store(v, reinterpret_cast<f32x4_a4 *>(p));
            else
                __builtin_memcpy(p, &v, 16);
        } else {
#pragma unroll
            for (int e = 0; e < 3; ++e)
                if (e < left) p[e] = v[e];
        }
        return;
    }
    uint32_t w[2];
    if (g.type == 1) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 a = {static_cast<__bf16>(v[0]), static_cast<__bf16>(v[1])};
        const bf16x2 b = {static_cast<__bf16>(v[2]), static_cast<__bf16>(v[3])};
        w[0] = __builtin_bit_cast(uint32_t, a);
        w[1] = __builtin_bit_cast(uint32_t, b);
    } else {
        typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
        const f16x2 a = {static_cast<_Float16>(v[0]), static_cast<_Float16>(v[1])};
        const f16x2 b = {static_cast<_Float16>(v[2]), static_cast<_Float16>(v[3])};
        w[0] = __builtin_bit_cast(uint32_t, a);
        w[1] = __builtin_bit_cast(uint32_t, b);
    }
    uint16_t *p = static_cast<uint16_t *>(g.C) + at;
    typedef uint32_t u32x2_a4 __attribute__((ext_vector_type(2), aligned(4)));
    if (left >= 4) {
        // (at 2-byte alignment the hinted store would be split)
        if (STREAM && (reinterpret_cast<uintptr_t>(p) & 3) == 0)
            __builtin_nontemporal_store(u32x2_a4{w[0], w[1]}, reinterpret_cast<u32x2_a4 *>(p));
        else
            __builtin_memcpy(p, w, 8);
    } else {
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (e < left) p[e] = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
}

// Scales of four results of a row of an int8 product, from column n on.  Read
// before the sums are made: at the end the row's index, its scale and the store
// would wait for each other (8 groups of 1000 rows, 1501 x 777: 14.6 us against
// 13.2; 16 of 1024, 512 x 2048: 10.5 and 9.6).
struct Scales4 {
    int row;  // of A, or -1: zeros
    float a;
    f32x4 b;
};
__device__ __forceinline__ Scales4 load_scales4(const ProductArgs &g, const RowTile &rt, int m, int n) {
    Scales4 s;
    s.row = a_row(g, min(m, rt.end - 1));
    s.a = g.a_scale[max(s.row, 0)];
    const float *sb = g.b_scale + static_cast<int64_t>(rt.group) * g.N;
#pragma unroll
    for (int e = 0; e < 4; ++e) s.b[e] = sb[min(n + e, g.N - 1)];
    return s;
}
__device__ __forceinline__ void store_scaled4(const ProductArgs &g, int m, int n, i32x4 sum, const Scales4 &s) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = s.row < 0 ? 0.0f : static_cast<float>(sum[e]) * (s.a * s.b[e]);
    store_row4(g, m, n, v);
}

}  // namespace tdi8

// Product of e4m3 operands with a scale for each block of 128, for more rows
// than the stream kernels take: both operands staged in LDS.
//
// K tile = scale block = 128.  One v_mfma_f32_16x16x128_f8f6f4 makes a 16 x 16
// tile's part of a whole scale block; since the block scales are no powers of
// two it starts from zero, and acc += part * (a_scale * b_scale) in fp32
// follows: 4 multiply-adds a lane for 32 cycles of the matrix core, which run
// beside it (fp32 and fp16 results take F8Wide's four bf16 instructions instead).  A
// lane's part belongs to one row of A (B is the instruction's first operand)
// and a wave's columns to one block of 128, so the scale is one register per
// 16 rows.
//
// Staging.  A and B tiles go to LDS by 16-byte DMA loads with the 16-byte
// chunks of a row permuted (row16_swizzle), so that an operand read touches
// every bank once; the tile's a_scale column goes with them by 4-byte DMA.
// They are buffer loads: one 32-bit offset per lane and a scalar K offset
// (64-bit addresses would take 16 more registers than a wave has), and what
// lies outside the operand, rows past M or N and chunks past K, gets an offset
// past the buffer's end, which reads as zero.
//
// Schedule of a K tile (STAGES stages, one barrier).  Rows 16 i .. 16 i + 15 of
// the wave's part are one step; steps 0 .. MT - 3 read the A operand two steps
// ahead.  Then every operand of the tile is in registers: the loads of the
// next tile have landed (issued STAGES - 1 tiles ago), a barrier publishes
// them and frees this tile's stage, which is refilled at once.  The last two steps
// go column by column, and each B operand's registers take the next tile's as
// soon as both steps are done with it, so the next tile starts with operands
// in place.  Scaled additions follow three instructions behind the matrix
// instruction whose part they add (kLag), across steps and tiles.
//
// Measured on MI355X: 4096^3 to bf16 72 to 77 us (1.8 PFLOP/s), 8192^3 500 to
// 550 us (2.1 PFLOP/s; the range is that of the chip's clock from one machine
// to the next; a plain e4m3 product of that size without scales reaches 2.6),
// to fp32 4096^3 127 to 135 us.  At 8192^3 the matrix cores are busy 47% of
// the cycles at 2.1 GHz, the vector units 37%, LDS reads 22%: none is full, and
// each of the two waves of a SIMD waits 31% of its time ((128 + 64) rows read
// for 128 x 64 results a wave; wider wave tiles need more accumulators than a
// wave has registers that multiply-adds can address).  Tiles: 256 x 256 of two
// stages for many rows; 128 x 128 twice on a compute unit, or with four
// stages once; 64 x 128 with four (product_table.h has their costs).
#pragma once

#include "operand_types.h"

namespace tdi8 {

template <class E, int WM, int WN, int MT, int NT, int STAGES>
__global__ void __launch_bounds__(WM * WN * 64, 2) block_scale_kernel(ProductArgs g) {
    constexpr int NW = WM * WN;
    constexpr int BM = WM * MT * 16, BN = WN * NT * 16;
    constexpr int BK = 128, CPR = BK / 16;
    constexpr int LA = BM * CPR / 64 / NW, LB = BN * CPR / 64 / NW;  // DMA loads per wave and tile
    constexpr int SCALES = (BM + BN) * BK;                           // offset of the a_scale column in a stage
    constexpr int STAGE = SCALES + BM * 4;
    static_assert(BM * CPR % (64 * NW) == 0 && BN * CPR % (64 * NW) == 0 && NW % 2 == 0, "loads split evenly");
    static_assert(BM % 64 == 0 && BM / 64 <= NW, "one scale load per wave");
    static_assert(128 % (NT * 16) == 0 && BN % 128 == 0, "a wave's columns lie in one block of 128");
    static_assert(STAGES >= 2 && (STAGES & (STAGES - 1)) == 0, "a power of two stages");
    static_assert((STAGES - 1) * (LA + LB + 1) < 64, "the wait counter holds 63");
    static_assert(MT % 4 == 0, "the operand ring starts over with every tile");
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) int8_t lds[STAGES * STAGE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r16 = lane & 15, q = lane >> 4;

    // Four row tiles by all column tiles, in runs of one XCD (rc_pipelined_kernel.h).
    const int64_t total = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
    const int64_t l = xcd_run(blockIdx.x, total);
    if (l >= total) return;
    const int64_t gsize = 4ll * g.tiles_n;
    const int first = static_cast<int>(l / gsize) * 4;
    const int grows = min(g.tiles_m - first, 4);
    const int within = static_cast<int>(l % gsize);
    const int m0 = (first + within % grows) * BM;
    const int n0 = (within / grows) * BN;
    const int nk = (g.K + BK - 1) / BK;
    // With one row tile each block reads its part of B alone, and starts at a
    // K tile of its own (rc_pipelined_kernel.h, the grouped source).
    const int turn = g.tiles_m == 1 && nk > 0 ? 5 * static_cast<int>(blockIdx.x >> 3) % nk : 0;
    auto turned = [&](int kt) { return kt + turn < nk ? kt + turn : kt + turn - nk; };

    // Buffers over the tile's rows.  A row past M or N starts past the end of
    // its buffer (lda >= K), and so does kOut.
    constexpr uint32_t kOut = 0x80000000u;
    const int rows_a = min(BM, g.M - m0), rows_b = min(BN, g.N - n0);
    const int lda = static_cast<int>(g.lda), ldb = static_cast<int>(g.ldb);
    const __amdgpu_buffer_rsrc_t buf_a = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t *>(g.A + m0 * g.lda), 0, (rows_a - 1) * lda + g.K, 0x00027000);
    const __amdgpu_buffer_rsrc_t buf_b = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<int8_t *>(g.B + n0 * g.ldb), 0, (rows_b - 1) * ldb + g.K, 0x00027000);
    const __amdgpu_buffer_rsrc_t buf_s = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float *>(g.a_scale + m0 * g.ldas), 0, ((rows_a - 1) * static_cast<int>(g.ldas) + nk) * 4,
        0x00027000);
    // Load i of this wave fills LDS rows 8 (i NW + wave) .. + 7; NW is even, so
    // the chunk permutation is the same for every i.
    const int lrow = wave * 8 + (lane >> 3);
    const int lchunk = (lane & 7) ^ row16_swizzle((wave & 1) * 8 + (lane >> 3));
    const uint32_t off_a = lrow * lda + 16 * lchunk;
    const uint32_t off_b = lrow * ldb + 16 * lchunk;
    // (every wave loads 64 rows' scales, the same ones more than once: a branch
    // here would let the compiler sink the scaled additions behind it)
    const int swave = wave % (BM / 64);
    const uint32_t off_s = (swave * 64 + lane) * static_cast<int>(g.ldas) * 4;
    constexpr int LOADS = LA + LB + 1;
    auto issue = [&](int kt) {
        int8_t *dst = lds + (kt & (STAGES - 1)) * STAGE;
        const int kk = turned(kt);
        const int k = kk * BK;
        const uint32_t past = k + 16 * lchunk >= g.K ? kOut : 0u;  // chunks of a last, partial K tile
#pragma unroll
        for (int i = 0; i < LA; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buf_a, (lds_void_t *)(dst + (i * NW + wave) * 1024), 16,
                                                     static_cast<int>((off_a + i * (NW * 8) * lda) | past), k, 0, 0);
#pragma unroll
        for (int i = 0; i < LB; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buf_b, (lds_void_t *)(dst + BM * BK + (i * NW + wave) * 1024), 16,
                                                     static_cast<int>((off_b + i * (NW * 8) * ldb) | past), k, 0, 0);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buf_s, (lds_void_t *)(dst + SCALES + swave * 256), 4,
                                                 static_cast<int>(off_s), kk * 4, 0, 0);
    };
    // This wave's scales of B: one block of 128 columns, read as scalars.
    typedef const __attribute__((address_space(4))) float *scalar_t;
    const scalar_t scale_b = (scalar_t)(g.b_scale + ((n0 + wn * (NT * 16)) / 128 < (g.N + 127) / 128
                                                         ? (n0 + wn * (NT * 16)) / 128 * g.ldbs
                                                         : 0));

    // LDS offsets of the operand pieces q and 4 + q of row r16.
    const int sw = row16_swizzle(r16);
    const int lo_a = (wm * (MT * 16) + r16) * BK + 16 * (q ^ sw);
    const int lo_b = BM * BK + (wn * (NT * 16) + r16) * BK + 16 * (q ^ sw);
    const int ls = SCALES + (wm * (MT * 16) + r16) * 4;
    auto piece = [&](const int8_t *p) { return *reinterpret_cast<const i32x4 *>(p); };

    f32x4 acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    constexpr int RING = 4;  // A operands in registers: read two steps ahead
    constexpr int kLag = 3;  // scaled additions behind
    i32x4 ra[RING][2];
    float rs[RING];
    Operand<E> ob[NT];
    float s[RING];           // a_scale * b_scale of the last steps
    f32x4 part[kLag + 1];
    Operand<E> oa[RING];
    auto read_a = [&](int kt, int i) {
        const int8_t *p = lds + (kt & (STAGES - 1)) * STAGE;
        ra[i % RING][0] = piece(p + lo_a + i * (16 * BK));
        ra[i % RING][1] = piece(p + (lo_a ^ 64) + i * (16 * BK));
        rs[i % RING] = *reinterpret_cast<const float *>(p + ls + i * 64);
    };
    auto read_b = [&](int kt, int j) {
        const int8_t *p = lds + (kt & (STAGES - 1)) * STAGE;
        ob[j].set(piece(p + lo_b + j * (16 * BK)), piece(p + (lo_b ^ 64) + j * (16 * BK)));
    };
    // Matrix instruction x of a tile works on step step_of(x), column col_of(x):
    // row by row, the last two steps column by column.
    constexpr int X = MT * NT;
    constexpr int TAIL = (MT - 2) * NT;  // first instruction of the last two steps
    auto step_of = [](int x) constexpr { return x < TAIL ? x / NT : MT - 2 + (x - TAIL) % 2; };
    auto col_of = [](int x) constexpr { return x < TAIL ? x % NT : (x - TAIL) / 2; };
    auto add = [&](int x) {  // of instruction x, x < 0: of the tile before
        const int y = (x + X) % X;
        const int i = step_of(y), j = col_of(y);
        const f32x4 p = part[y % (kLag + 1)];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(p[e], s[i % RING], acc[i][j][e]);
    };
    static_assert(2 * NT >= kLag + 1 && X % (kLag + 1) == 0, "parts keep their registers from tile to tile");

    if (nk > 0) {
        const int ahead = nk < STAGES ? nk : STAGES;
#pragma unroll
        for (int t = 0; t < STAGES; ++t)
            if (t < ahead) issue(t);
#pragma unroll
        for (int x = 0; x <= kLag; ++x) part[x] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < RING; ++i) s[i] = 0.0f;
        // tile 0 has landed when only the later ones' loads are out
        if (ahead == STAGES) {
            TDI8_WAIT_VMCNT((STAGES - 1) * LOADS);
        } else {
            TDI8_WAIT_VMCNT(0);
        }
        block_barrier();
        read_a(0, 0);
        read_a(0, 1);
#pragma unroll
        for (int j = 0; j < NT; ++j) read_b(0, j);
        float sb = scale_b[turn];

        // LOAD: refill the freed stage with tile kt + STAGES; NEXT: tile kt + 1
        // exists; INFLIGHT: the loads of tiles kt + 2 .. kt + STAGES - 1 may
        // stay out while tile kt + 1's are waited for.
        auto tile = [&](int kt, auto load_tag, auto next_tag, auto inflight_tag) {
            constexpr bool LOAD = decltype(load_tag)::value, NEXT = decltype(next_tag)::value;
            constexpr bool INFLIGHT = decltype(inflight_tag)::value;
            const float sb_next = NEXT ? scale_b[turned(kt + 1)] : 0.0f;
            static_for<X>([&](auto xt) {
                constexpr int x = decltype(xt)::value;
                constexpr int i = step_of(x), j = col_of(x);
                if constexpr (x == TAIL && NEXT) {
                    // every operand of this tile is in registers
                    if constexpr (INFLIGHT) {
                        TDI8_WAIT_VMCNT((STAGES - 2) * LOADS);
                    } else {
                        TDI8_WAIT_VMCNT(0);
                    }
                    TDI8_WAIT_LGKM0();
                    block_barrier();
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (LOAD) issue(kt + STAGES);
                }
                if constexpr (x < TAIL && j == 0) read_a(kt, i + 2);
                if constexpr (j == 0) oa[i % RING].set(ra[i % RING][0], ra[i % RING][1]);
                part[x % (kLag + 1)] = Operand<E>::mma(ob[j], oa[i % RING]);
                add(x - kLag);
                // The scales of a step, before its first addition and, for the
                // last two, after the last ones of the tile before.
                if constexpr (x < TAIL && j == 0) s[i % RING] = rs[i % RING] * sb;
                if constexpr (x == TAIL + kLag - 1) {
                    s[RING - 2] = rs[RING - 2] * sb;
                    s[RING - 1] = rs[RING - 1] * sb;
                }
                if constexpr (NEXT && x >= TAIL && (x - TAIL) % 2 == 1) {
                    read_b(kt + 1, j);
                    if constexpr (j < 2) read_a(kt + 1, j);
                }
                __builtin_amdgcn_sched_barrier(0);
            });
            sb = sb_next;
        };
        using T1 = std::true_type;
        using T0 = std::false_type;
        int kt = 0;
        for (; kt + STAGES < nk; ++kt) tile(kt, T1{}, T1{}, T1{});
        if (kt + STAGES == nk && kt + 1 < nk) {
            tile(kt, T0{}, T1{}, T1{});
            ++kt;
        }
        for (; kt + 1 < nk; ++kt) tile(kt, T0{}, T1{}, T0{});
        tile(kt, T0{}, T0{}, T0{});
        static_for<kLag>([&](auto xt) { add(X - kLag + decltype(xt)::value); });
    }

    // C through LDS in passes of 64 rows, whole rows of the tile to a wave's
    // stores (rows padded so that an instruction's writes spread over the banks).
    constexpr int RS = BN + 4, RP = 64;
    static_assert(RP * RS * 4 <= STAGES * STAGE, "a pass fits the stages");
    float *cl = reinterpret_cast<float *>(lds);
    for (int p0 = 0; p0 < BM; p0 += RP) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int rb = wm * (MT * 16) + i * 16;
            if (rb < p0 || rb >= p0 + RP) continue;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                *reinterpret_cast<f32x4 *>(cl + (rb - p0 + r16) * RS + wn * (NT * 16) + j * 16 + 4 * q) = acc[i][j];
        }
        __syncthreads();
        for (int x = threadIdx.x; x < RP * (BN / 4); x += NW * 64) {
            const int r = x / (BN / 4), c = x - r * (BN / 4);
            const int m = m0 + p0 + r, n = n0 + 4 * c;
            if (m < g.M && n < g.N)
                store_row4<true>(g, m, n, *reinterpret_cast<const f32x4 *>(cl + r * RS + 4 * c));
        }
    }
#endif
}

}  // namespace tdi8

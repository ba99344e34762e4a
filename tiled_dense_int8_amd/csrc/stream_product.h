// Products of few rows: every wave streams its share of K.
//
// Block: BM rows of one group, BN columns, all of K, which its W waves share by
// chunks of 128 (wave w takes chunks w, w + W, ...).  A wave moves a chunk of
// its BM + BN rows into LDS of its own by 16-byte LDS DMA, eight whole 128-byte
// lines an instruction, reads it back as operands (operand_types.h), and sends
// the next chunk's loads before it multiplies.  No wave waits for another
// before the end, where the partial tiles are summed in the order of the waves
// (a result does not depend on which came first).  Rows past the end repeat the
// last one; of BM = 8 rows each is read by two lanes.
//
// Operands off 16-byte alignment (K, a pointer or a leading dimension): a chunk
// of a row lies within nine aligned pieces, which go to LDS as they are (every
// piece read holds a byte of the row); a lane shifts each pair of pieces that
// it reads into place.  Unaligned loads into registers run at about a third of
// the rate of aligned ones (21 of 58 bytes per cycle and compute unit from L2):
// 16 x 4096 x 4095 e4m3 18.2 us by those, 8.0 by shifted pieces, 100 x 1000 x
// 1001 8.9 and 4.6.
//
// With few rows the product is a read of B, bound by HBM: 16 x 65536 x 4096
// e4m3 51.4 us, 5.2 TB/s; 16 x 4096 x 4096 5.9 us, of which 3 are a launch's.
// Through the middle (64 to 512 rows) a block's (BM + BN) K bytes from L2 bound
// it, about 31 bytes a cycle and compute unit; the larger tiles read less, the
// smaller fill the chip, and the choice weighs the two by their measured costs
// (product_table.h; 256 x 4096 x 4096 e4m3: 13.9 us at 64 x 64, 19.9 at
// 32 x 32, 22 with the LDS tiles; 64 x 4096 x 4096: 14.3, 8.1 and 21.8).
// Two or four chunks of LDS a wave instead of one: 16 x 4096 x 4096 5.9 and
// 6.0 us, 64 x 4096 x 4096 9.2, so what lies beside the other blocks of the
// compute unit counts for more.  Loads into registers, 64 bytes of 16 rows an
// instruction, ask for every line twice: 7.5 and 12.4 us.
#pragma once

#include "operand_types.h"

namespace tdi8 {

template <class E, int BM, int BN, int W, bool ALIGNED>
__global__ void __launch_bounds__(W * 64) stream_product_kernel(ProductArgs g) {
    constexpr int MT = (BM + 15) / 16, NT = BN / 16;
    constexpr int PITCH = ALIGNED ? kChunk : kChunk + 16;  // of a row in LDS
    constexpr int LOADS = ((BM + BN) * PITCH + 1023) / 1024;
    constexpr int SCALES = LOADS * 1024;
    constexpr int STAGE = SCALES + (E::kBlockScales ? 256 : 0);
    static_assert(16 * MT * BN * 4 <= STAGE && W * STAGE <= 160 * 1024, "LDS");
    static_assert(BM <= 64, "one load takes a chunk's scales");
#if defined(__HIP_DEVICE_COMPILE__)
    using Acc = typename E::Acc;
    __shared__ __attribute__((aligned(1024))) int8_t lds[W * STAGE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, q = lane >> 4;

    const int64_t total = static_cast<int64_t>(g.tiles_m) * g.tiles_n;
    const int64_t at = xcd_run(blockIdx.x, total);
    if (at >= total) return;
    // row tiles of one column tile follow each other: they share B
    const int tn = static_cast<int>(at / g.tiles_m);
    RowTile rt{};
    if (!find_rows(g, BM, static_cast<int>(at - static_cast<int64_t>(tn) * g.tiles_m), rt, nullptr)) return;
    const int n0 = tn * BN;

    // rows past the group repeat its last one; rows outside A are zeroed at the end
    auto row_a = [&](int r) { return g.A + max(a_row(g, min(rt.m0 + r, rt.end - 1)), 0) * g.lda; };
    auto row_b = [&](int r) {
        return g.B + rt.group * g.group_b + static_cast<int64_t>(min(n0 + r, g.N - 1)) * g.ldb;
    };
    // Load i fills the 1024 bytes i of a stage: A's rows and then B's.  Aligned,
    // eight rows with their pieces permuted; otherwise the nine aligned pieces
    // that hold a row's 128 bytes, for src, its bytes.
    const int8_t *src[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int x = 64 * i + lane;
        const int row = x / (PITCH / 16), piece = x % (PITCH / 16);
        const int r = row < BM ? row : row - BM;
        src[i] = (row < BM ? row_a(r) : row_b(r)) + wave * kChunk + 16 * (ALIGNED ? piece ^ row16_swizzle(r & 15) : piece);
    }
    const float *ssrc = nullptr, *psb = nullptr;
    if constexpr (E::kBlockScales) {
        ssrc = g.a_scale + min(rt.m0 + lane % BM, rt.end - 1) * g.ldas + wave;
        psb = g.b_scale + (n0 / kChunk) * g.ldbs + wave;  // 128 is a multiple of BN
    }
    int8_t *const mine = lds + wave * STAGE;
    const int whole = g.K / kChunk;
    const int some = ALIGNED ? whole : (g.K + kChunk - 1) / kChunk;  // chunks that take the loop
    const int n = some > wave ? (some - wave + W - 1) / W : 0;
    // bytes of chunk c of this wave
    auto bytes = [&](int c) { return min(g.K - (wave + c * W) * kChunk, kChunk); };
    // A block that reads its part of B alone starts at a chunk of its own: rows
    // a power of two apart lie in one memory channel, which all blocks would
    // want at once (1 x 32768 x 4096 e4m3 27.7 -> 23.7 us, 8 groups of 2 rows,
    // 11008 x 4096 int8 75 -> 65; 2 groups, 4096 x 4096, whose B the cache still
    // holds, 8.0 -> 9.1).  Blocks that share B stay in step.
    const int turn = n > 0 && rt.end - rt.begin <= BM ? static_cast<int>(blockIdx.x >> 3) % n : 0;
    auto turned = [&](int c) { return c + turn < n ? c + turn : c + turn - n; };
    auto issue = [&](int c) {
        c = turned(c);
        if constexpr (E::kBlockScales)
            __builtin_amdgcn_global_load_lds(ssrc + c * W, (lds_void_t *)(mine + SCALES), 4, 0, 0);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int8_t *p = src[i] + c * (W * kChunk);
            if constexpr (!ALIGNED) {
                // the piece's first byte lies `over` behind the row's last of
                // this chunk: load the last piece instead
                const int s = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15);
                const int over = 16 * ((64 * i + lane) % (PITCH / 16)) - s - bytes(c);
                p -= s + (over >= 0 ? (over & ~15) + 16 : 0);
            }
            __builtin_amdgcn_global_load_lds(p, (lds_void_t *)(mine + 1024 * i), 16, 0, 0);
        }
    };

    Acc acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Acc{};
    const int ra = r16 % BM;
    const int lo_a = ra * PITCH + 16 * (ALIGNED ? q ^ row16_swizzle(ra) : q);
    const int lo_b = (BM + r16) * PITCH + 16 * (ALIGNED ? q ^ row16_swizzle(r16) : q);
    int shift_a[MT], shift_b[NT];  // of the rows from 16 bytes
    if constexpr (!ALIGNED) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
            shift_a[i] = static_cast<int>(reinterpret_cast<uintptr_t>(row_a(16 * i + ra)) & 15);
#pragma unroll
        for (int j = 0; j < NT; ++j)
            shift_b[j] = static_cast<int>(reinterpret_cast<uintptr_t>(row_b(16 * j + r16)) & 15);
    }
    // Pieces q and q + 4 of the row at p.
    auto read = [&](const int8_t *p, int shift, i32x4 (&v)[2]) {
        if constexpr (ALIGNED) {
            v[0] = load16(p);
            v[1] = load16(mine + ((p - mine) ^ 64));
        } else {
            v[0] = funnel16(load16(p), load16(p + 16), shift);
            v[1] = funnel16(load16(p + 64), load16(p + 80), shift);
        }
    };
    if (n > 0) issue(0);
    constexpr int ITEMS = (BM * (BN / 4) + W * 64 - 1) / (W * 64);  // of four results a thread
    Scales4 scales[ITEMS];
    if constexpr (!E::kBlockScales) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int x = threadIdx.x + i * (W * 64);
            scales[i] = load_scales4(g, rt, rt.m0 + x / (BN / 4), n0 + x % (BN / 4) * 4);
        }
    }
    for (int c = 0; c < n; ++c) {
        const float scale_b = E::kBlockScales ? psb[turned(c) * W] : 0.0f;
        TDI8_WAIT_VMCNT(0);
        asm volatile("" ::: "memory");
        i32x4 a[MT][2], b[NT][2];
        float s[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            read(mine + i * (16 * PITCH) + lo_a, shift_a[i], a[i]);
            s[i] = E::kBlockScales ? *reinterpret_cast<const float *>(mine + SCALES + 64 * i + 4 * ra) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) read(mine + j * (16 * PITCH) + lo_b, shift_b[j], b[j]);
        if (c + 1 < n) {
            TDI8_WAIT_LGKM0();  // the chunk is in registers
            asm volatile("" ::: "memory");
            issue(c + 1);
        }
        if (!ALIGNED && bytes(turned(c)) < kChunk) {  // the last, partial chunk: zeros behind the rows' ends
            const int left = bytes(turned(c)) - 16 * q;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                a[i][0] = keep16(a[i][0], left);
                a[i][1] = keep16(a[i][1], left - 64);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                b[j][0] = keep16(b[j][0], left);
                b[j][1] = keep16(b[j][1], left - 64);
            }
        }
        Operand<E> ob[NT], oa;
#pragma unroll
        for (int j = 0; j < NT; ++j) ob[j].set(b[j][0], b[j][1]);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            oa.set(a[i][0], a[i][1]);
#pragma unroll
            for (int j = 0; j < NT; ++j) Operand<E>::add(ob[j], oa, s[i] * scale_b, acc[i][j]);
        }
    }
    if (ALIGNED && whole * kChunk < g.K && whole % W == wave) {  // the last, partial chunk
        const int k = whole * kChunk + 16 * q;
        auto load = [&](const int8_t *p, int h) { return load16_masked(p + k + h, clamp16(g.K - k - h)); };
        Operand<E> ob[NT], oa;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int8_t *p = row_b(16 * j + r16);
            ob[j].set(load(p, 0), load(p, 64));
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int8_t *p = row_a(16 * i + r16);
            oa.set(load(p, 0), load(p, 64));
            float s = 0.0f;
            if constexpr (E::kBlockScales)
                s = g.a_scale[min(rt.m0 + 16 * i + r16, rt.end - 1) * g.ldas + whole] * psb[whole - wave];
#pragma unroll
            for (int j = 0; j < NT; ++j) Operand<E>::add(ob[j], oa, s, acc[i][j]);
        }
    }

    // partial tiles: a lane writes four consecutive columns of its row
    constexpr int PART = STAGE / 16;  // from one wave's to the next
    Acc *part = reinterpret_cast<Acc *>(lds);
    auto at_part = [](int r, int c4) { return r * (BN / 4) + (c4 ^ (r & (BN / 4 - 1))); };
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            part[wave * PART + at_part(16 * i + r16, 4 * j + q)] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int x = threadIdx.x + i * (W * 64);
        const int r = x / (BN / 4), c4 = x - r * (BN / 4);
        const int m = rt.m0 + r, nn = n0 + 4 * c4;
        if (x >= BM * (BN / 4) || m >= rt.end || nn >= g.N) continue;
        Acc sum = part[at_part(r, c4)];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += part[w * PART + at_part(r, c4)];
        if constexpr (E::kBlockScales)
            store_row4(g, m, nn, sum);
        else
            store_scaled4(g, m, nn, sum, scales[i]);
    }
#endif
}

}  // namespace tdi8

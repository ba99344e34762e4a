// Products of operands off 16-byte alignment (K, a pointer or a leading
// dimension) with more rows than the stream kernels take: both operands go
// through registers into LDS.
//
// An unaligned 16-byte load runs at about a third of the rate of an aligned
// one (21 of 58 bytes per cycle and compute unit from L2), so what counts is
// how few of them a tile needs: a BM x BN tile loads BM + BN rows once, where
// the stream kernels' tiles are smaller (1000 x 3000 x 777 e4m3: 24 us there).
//
// Two LDS stages, K tiles of 128.  A K tile's loads go out while the tile
// before is multiplied, wait in registers and are written to the stage that
// was freed by the last barrier; one barrier per K tile.  Rows past the end
// repeat the last one (their results are not stored); in a last, partial K
// tile the bytes past K are zero.  Scales and the 16 x 16 parts are those of
// the stream kernels; chunks lie permuted by row16_swizzle.
//
// 64 x 128 by eight waves: 13.7 us at 1000 x 3000 x 777 e4m3 to bf16 and
// 27.4 us (585 TFLOP/s) at 2000 x 2000 x 2001, where four waves took 15.2 and
// 29.4 us, 128 x 128 by four 18.7 and 34.0, and loads two tiles ahead 14.8
// and 27.9.  Aligned pieces shifted into place on their way to LDS, as the
// stream kernels do on reading: 15.4 and 29.5.
#pragma once

#include "operand_types.h"

namespace tdi8 {

template <class E, int WM, int WN, int MT, int NT>
__global__ void __launch_bounds__(WM * WN * 64, 2) staged_product_kernel(ProductArgs g) {
    constexpr int THREADS = WM * WN * 64;
    constexpr int BM = WM * MT * 16, BN = WN * NT * 16;
    constexpr int BK = kChunk, CPR = BK / 16;
    constexpr int LOADS = (BM + BN) * CPR / THREADS;
    constexpr int SCALES = (BM + BN) * BK;
    constexpr int STAGE = SCALES + (E::kBlockScales ? BM * 4 : 0);
    constexpr int RS = BN + 4, ITEMS = BM * (BN / 4) / THREADS;  // of four results a thread
    static_assert(BM * (BN / 4) % THREADS == 0 && BM * RS * 4 <= 2 * STAGE, "C fits the stages");
    static_assert((BM + BN) * CPR % THREADS == 0 && BM <= THREADS, "loads split evenly");
    static_assert(128 % (NT * 16) == 0 && BN % 128 == 0, "a wave's columns lie in one block of 128");
#if defined(__HIP_DEVICE_COMPILE__)
    using Acc = typename E::Acc;
    __shared__ __attribute__((aligned(1024))) int8_t lds[2 * STAGE];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int r16 = lane & 15, q = lane >> 4;

    RowTile rt{};
    int tiles = 0;
    find_rows(g, BM, -1, rt, &tiles);
    const int64_t total = static_cast<int64_t>(tiles) * g.tiles_n;
    const int64_t l = xcd_run(blockIdx.x, total);
    if (l >= total) return;
    const int64_t gsize = 4ll * g.tiles_n;
    const int first = static_cast<int>(l / gsize) * 4;
    const int grows = min(tiles - first, 4);
    const int within = static_cast<int>(l % gsize);
    if (!find_rows(g, BM, first + within % grows, rt, nullptr)) return;
    const int n0 = within / grows * BN;
    const int nk = (g.K + BK - 1) / BK;

    // Load i of this thread: chunk `lc` of row lr + i * THREADS / 8 of A, then B.
    const int lr = threadIdx.x / CPR, lc = threadIdx.x % CPR;
    const int8_t *src[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int r = lr + i * (THREADS / CPR);
        if (r < BM)
            src[i] = g.A + max(a_row(g, min(rt.m0 + r, rt.end - 1)), 0) * g.lda + 16 * lc;
        else
            src[i] = g.B + rt.group * g.group_b + min(n0 + r - BM, g.N - 1) * g.ldb + 16 * lc;
    }
    const float *ssrc = E::kBlockScales
                            ? g.a_scale + max(a_row(g, min(rt.m0 + static_cast<int>(threadIdx.x), rt.end - 1)), 0) * g.ldas
                            : nullptr;
    const float *sb = E::kBlockScales
                          ? g.b_scale + min((n0 + wn * (NT * 16)) / 128, (g.N + 127) / 128 - 1) * g.ldbs
                          : nullptr;
    i32x4 st[LOADS];
    float sst = 0.0f;
    auto fetch = [&](int kt) {
        const int k = kt * BK;
        if (k + BK <= g.K) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) st[i] = load16_unaligned(src[i] + k);
        } else {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) st[i] = load16_masked(src[i] + k, clamp16(g.K - k - 16 * lc));
        }
        if (E::kBlockScales && threadIdx.x < BM) sst = ssrc[kt];
    };
    auto stash = [&](int kt) {
        int8_t *p = lds + (kt & 1) * STAGE;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int r = lr + i * (THREADS / CPR);
            *reinterpret_cast<i32x4 *>(p + r * BK + 16 * (lc ^ row16_swizzle(r & 15))) = st[i];
        }
        if (E::kBlockScales && threadIdx.x < BM) *reinterpret_cast<float *>(p + SCALES + threadIdx.x * 4) = sst;
    };

    Acc acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Acc{};
    const int sw = row16_swizzle(r16);
    auto read = [&](Operand<E> &o, const int8_t *p, int r) {
        o.set(load16(p + r * BK + 16 * (q ^ sw)), load16(p + r * BK + 16 * ((q + 4) ^ sw)));
    };
    if (nk > 0) fetch(0);
    Scales4 scales[ITEMS];
    if constexpr (!E::kBlockScales) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int x = threadIdx.x + i * THREADS;
            scales[i] = load_scales4(g, rt, rt.m0 + x / (BN / 4), n0 + x % (BN / 4) * 4);
        }
    }
    for (int kt = 0; kt < nk; ++kt) {
        stash(kt);
        const float scale_b = E::kBlockScales ? sb[kt] : 0.0f;
        TDI8_WAIT_LGKM0();
        block_barrier();
        if (kt + 1 < nk) fetch(kt + 1);
        const int8_t *p = lds + (kt & 1) * STAGE;
        Operand<E> b[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) read(b[j], p, BM + wn * (NT * 16) + j * 16 + r16);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int r = wm * (MT * 16) + i * 16 + r16;
            Operand<E> a;
            read(a, p, r);
            const float s = E::kBlockScales ? *reinterpret_cast<const float *>(p + SCALES + 4 * r) * scale_b : 0.0f;
#pragma unroll
            for (int j = 0; j < NT; ++j) Operand<E>::add(b[j], a, s, acc[i][j]);
        }
    }

    // C through LDS
    Acc *cl = reinterpret_cast<Acc *>(lds);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            cl[((wm * (MT * 16) + i * 16 + r16) * RS + wn * (NT * 16) + j * 16) / 4 + q] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int x = threadIdx.x + i * THREADS;
        const int r = x / (BN / 4), c = x - r * (BN / 4);
        const int m = rt.m0 + r, n = n0 + 4 * c;
        if (m >= rt.end || n >= g.N) continue;
        const Acc v = cl[r * RS / 4 + c];
        if constexpr (E::kBlockScales)
            store_row4(g, m, n, v);
        else
            store_scaled4(g, m, n, v, scales[i]);
    }
#endif
}

}  // namespace tdi8

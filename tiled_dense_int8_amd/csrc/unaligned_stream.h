// Products of few rows with operands off 16-byte alignment (K, a pointer or a
// leading dimension): the stream of stream_product.h with loads into registers.
//
// Block: 16 MT rows of one group, 16 NT columns, all of K, which its W waves
// share by chunks of 128 (wave w takes chunks w, w + W, ...).  The waves'
// partial tiles are summed in LDS in the order of the waves.
//
// The LDS loads of stream_product.h take 16 aligned bytes (or 4 a lane, at a
// quarter of the rate).  A register load covers 64 bytes of 16 rows at once, so
// that every line is asked for twice; with aligned operands that made
// 16 x 4096 x 4096 e4m3 7.5 us against 5.9 and 64 x 4096 x 4096 12.4 against 8.1.
#pragma once

#include "operand_types.h"

namespace tdi8 {

template <class E, int MT, int NT, int W, int U>
__global__ void __launch_bounds__(W * 64) unaligned_stream_kernel(ProductArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int BM = 16 * MT, BN = 16 * NT;
    constexpr int RS = BN + 4;  // row stride of a partial tile in LDS
    using Acc = typename E::Acc;
    __shared__ __attribute__((aligned(16))) Acc part[W * BM * RS / 4];
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

    const int8_t *pa[MT], *pb[NT];
    const float *psa[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int m = min(rt.m0 + 16 * i + r16, rt.end - 1);  // rows past the group repeat its last one
        const int r = max(a_row(g, m), 0);                    // rows outside A are zeroed at the end
        pa[i] = g.A + r * g.lda;
        psa[i] = g.a_scale + (E::kBlockScales ? r * g.ldas : 0);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j)
        pb[j] = g.B + rt.group * g.group_b + static_cast<int64_t>(min(n0 + 16 * j + r16, g.N - 1)) * g.ldb;
    const float *psb = E::kBlockScales ? g.b_scale + (n0 / kChunk) * g.ldbs : nullptr;  // 128 is a multiple of BN

    Acc acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = Acc{};

    constexpr int ITEMS = (BM * (BN / 4) + W * 64 - 1) / (W * 64);  // of four results a thread
    Scales4 scales[ITEMS];
    if constexpr (!E::kBlockScales) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const int x = threadIdx.x + i * (W * 64);
            scales[i] = load_scales4(g, rt, rt.m0 + x / (BN / 4), n0 + x % (BN / 4) * 4);
        }
    }
    auto load = [&](const int8_t *p, int k, auto whole) -> i32x4 {
        if constexpr (decltype(whole)::value)
            return load16_unaligned(p + k);
        else
            return load16_masked(p + k, clamp16(g.K - k));
    };
    const int whole = g.K / kChunk;
    // U chunks a time, all of their loads before the first product: a wave has
    // U (MT + NT) KiB on the way at once.
    auto chunks = [&](int kc, auto count, auto whole) {
        constexpr int C = decltype(count)::value;
        i32x4 a[C][MT][2], b[C][NT][2];
        float s[C][MT];
#pragma unroll
        for (int u = 0; u < C; ++u) {
            const int k = (kc + u * W) * kChunk + 16 * q;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                b[u][j][0] = load(pb[j], k, whole);
                b[u][j][1] = load(pb[j], k + 64, whole);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                a[u][i][0] = load(pa[i], k, whole);
                a[u][i][1] = load(pa[i], k + 64, whole);
                s[u][i] = E::kBlockScales ? psa[i][kc + u * W] * psb[kc + u * W] : 0.0f;
            }
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < C; ++u) {
            Operand<E> ob[NT], oa;
#pragma unroll
            for (int j = 0; j < NT; ++j) ob[j].set(b[u][j][0], b[u][j][1]);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                oa.set(a[u][i][0], a[u][i][1]);
#pragma unroll
                for (int j = 0; j < NT; ++j) Operand<E>::add(ob[j], oa, s[u][i], acc[i][j]);
            }
        }
    };
    using One = std::integral_constant<int, 1>;
    int kc = wave;
    if constexpr (U > 1)
        for (; kc + (U - 1) * W < whole; kc += U * W) chunks(kc, std::integral_constant<int, U>{}, std::true_type{});
    for (; kc < whole; kc += W) chunks(kc, One{}, std::true_type{});
    if (whole * kChunk < g.K && whole % W == wave) chunks(whole, One{}, std::false_type{});

    // partial tiles: a lane writes four consecutive columns of its row
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
            part[((wave * BM + 16 * i + r16) * RS + 16 * j) / 4 + q] = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int x = threadIdx.x + i * (W * 64);
        const int r = x / (BN / 4), c = x - r * (BN / 4);
        const int m = rt.m0 + r, n = n0 + 4 * c;
        if (x >= BM * (BN / 4) || m >= rt.end || n >= g.N) continue;
        Acc sum = part[r * RS / 4 + c];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += part[(w * BM + r) * RS / 4 + c];
        if constexpr (E::kBlockScales)
            store_row4(g, m, n, sum);
        else
            store_scaled4(g, m, n, sum, scales[i]);
    }
#endif
}

}  // namespace tdi8

// Products of few rows, and of operands that the tile kernels cannot load
// (rows or K off 16-byte alignment): every wave streams its share of K
// straight from memory into registers.
//
// Block: 16 MT rows of one group, 16 NT columns, all of K, which its W waves
// share by chunks of 128 (wave w takes chunks w, w + W, ...).  With few rows
// the product is a stream over B, read once: there are N / (16 NT) blocks per
// group, enough to keep every compute unit's loads in flight, and no byte of
// B passes through LDS, since no two waves want the same one.
//
// Operands.  Lane l = 16 q + r holds, of row r of A and of column r of B, the
// 16-byte pieces q and 4 + q of the chunk (one load instruction covers 64
// contiguous bytes of 16 rows); both operands permute K alike, so the sum is
// that of the chunk.  s8: two v_mfma_i32_16x16x64_i8 a chunk.  e4m3: one
// v_mfma_f32_16x16x128_f8f6f4, whose 128 products of K are exactly a scale
// block, then acc += scale * part in fp32 (for fp32 results see F8Wide).  B is
// the first operand and A the second, so a lane ends with four consecutive
// columns of one row.
//
// The waves' partial tiles are summed in LDS in the order of the waves, so a
// result does not depend on which came first.
#pragma once

#include "scaled_product.h"

namespace tdi8 {

struct S8 {
    using Acc = i32x4;
    static constexpr bool kBlockScales = false;
    static __device__ __forceinline__ void chunk(const i32x4 (&a)[2], const i32x4 (&b)[2], float, Acc &acc) {
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[0], a[0], acc, 0, 0, 0);
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[1], a[1], acc, 0, 0, 0);
    }
};
// The e4m3 instructions add the 16 products of a 16-byte piece after cutting
// each to a multiple of 2^-13 of the largest one's power of two (measured:
// 2^5 + 2^-8 is exact within a piece, 2^6 + 2^-8 gives 2^6; between pieces
// sums are fp32).  On normal operands a result is off by 1.5 * 10^-5 of the
// results' size, far below half a step of the 16-bit types (2^-9, 2^-12).
struct F8 {
    using Acc = f32x4;
    static constexpr bool kBlockScales = true;
    static __device__ __forceinline__ i32x8 join(const i32x4 (&v)[2]) {
        return i32x8{v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]};
    }
    static __device__ __forceinline__ void chunk(const i32x4 (&a)[2], const i32x4 (&b)[2], float scale, Acc &acc) {
        // scale arguments of 0 select the instruction without block exponents
        const f32x4 part = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(b), join(a), f32x4{0, 0, 0, 0}, 0, 0,
                                                                            0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(part[e], scale, acc[e]);
    }
};

// For fp32 results: e4m3 widened to bf16 (exact), whose products are added in
// fp32: v_mfma_f32_16x16x32_bf16, four a chunk, at half the rate.
struct F8Wide {
    using Acc = f32x4;
    static constexpr bool kBlockScales = true;
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ bf16x8 widen(int32_t lo, int32_t hi) {
        const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
        const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
        const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
        const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
        return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
    }
    static __device__ __forceinline__ void chunk(const i32x4 (&a)[2], const i32x4 (&b)[2], float scale, Acc &acc) {
        f32x4 part = {0, 0, 0, 0};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const i32x4 x = b[h >> 1], y = a[h >> 1];
            const int o = 2 * (h & 1);
            part = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(x[o], x[o + 1]), widen(y[o], y[o + 1]), part, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(part[e], scale, acc[e]);
    }
};

constexpr int kChunk = 128;

// ALIGNED: A, B, lda, ldb, group_b and K are multiples of 16.
template <class E, int MT, int NT, int W, int U, bool ALIGNED>
__global__ void __launch_bounds__(W * 64) stream_product_kernel(ProductArgs g) {
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

    auto load = [&](const int8_t *p, int k, auto whole) -> i32x4 {
        if constexpr (decltype(whole)::value)
            return ALIGNED ? load16(p + k) : load16_unaligned(p + k);
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
        for (int u = 0; u < C; ++u)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int j = 0; j < NT; ++j) E::chunk(a[u][i], b[u][j], s[u][i], acc[i][j]);
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
    for (int x = threadIdx.x; x < BM * (BN / 4); x += W * 64) {
        const int r = x / (BN / 4), c = x - r * (BN / 4);
        const int m = rt.m0 + r, n = n0 + 4 * c;
        if (m >= rt.end || n >= g.N) continue;
        Acc sum = part[r * RS / 4 + c];
#pragma unroll
        for (int w = 1; w < W; ++w) sum += part[(w * BM + r) * RS / 4 + c];
        if constexpr (E::kBlockScales)
            store_row4(g, m, n, sum);
        else
            store_scaled4(g, rt.group, rt.end, m, n, sum);
    }
#endif
}

}  // namespace tdi8

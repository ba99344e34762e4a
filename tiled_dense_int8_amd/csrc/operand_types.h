// Operand types of the scaled products: how a lane's pieces of a chunk of 128
// values of K are multiplied.
//
// Lane l = 16 q + r holds, of row r of A and of column r of B, the 16-byte
// pieces q and 4 + q of the chunk; both operands permute K alike, so the sum is
// that of the chunk.  s8: two v_mfma_i32_16x16x64_i8.  e4m3: one
// v_mfma_f32_16x16x128_f8f6f4, whose 128 products of K are exactly a scale
// block, then acc += scale * part in fp32 (for fp32 results see F8Wide).  B is
// the first operand and A the second, so a lane ends with four consecutive
// columns of one row.
#pragma once

#include "scaled_product.h"

namespace tdi8 {

constexpr int kChunk = 128;

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

}  // namespace tdi8

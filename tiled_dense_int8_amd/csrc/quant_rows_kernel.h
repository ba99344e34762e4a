// Rows of activations to 8-bit operands with scales: RMS norm with the
// residual's addition, and the gated activation.
//
//   norm  h = rnd_T(x + r)  (r optional; h is stored as the new residual)
//         v = h w,  y = v / sqrt(mean(h^2) + eps)
//   act   v = y = g / (1 + e^-g) * u
//   s8    per row: scale = max|y| / 127,  q = rne(127 v / max|v|)
//   f8    per row and block of 128 columns: scale = max|y| / 448,
//         q = e4m3(448 v / max|v|)
//
// The norm's root cancels out of q, so q needs the row's (block's) largest
// |v| only and the root goes into the scale.  s8 is exact: q is the integer
// nearest to the real quotient (ties to even).  The quotient is first taken
// in fp32, whose error is below kNear (counted at to_s8); where it lies that
// near a border between two integers it is taken again in fp64.  Without
// this, values next to a border would round by the last bit of a sum or an
// exponential, and two orders of the same computation would give different
// bytes.  f8 rounds the fp32 quotient (v and the largest |v| are off by at
// most 10 * 2^-24 each, its two operations by 2^-24: below 2^-19, a step is
// 2^-3).  The sum of squares is held in fp64: finite inputs cannot overflow
// it, and it then says whether a row holds an infinity or NaN.
//
// A row (f8: block) that holds an infinity or NaN has q = 0 and scale = NaN,
// so that products with it come out NaN; one of zeros has q = 0 and scale = 0.
//
// Bound by memory: 3 T-sized streams and 1 byte per element (norm with a
// residual), read and written once.  A row stays in registers between its
// reduction and its quotients (up to 16384 columns; longer rows are read
// twice, the second time mostly from the cache), each thread holding vectors
// of 8 columns, so a block of 128 columns is 16 neighbouring lanes and its
// maximum needs no shared memory.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "quant_rows.h"

namespace tdi8 {

struct F32 {
    using Raw = float;
    static __device__ __forceinline__ float to_float(float v) { return v; }
    static __device__ __forceinline__ float round(float v) { return v; }
};
struct Bf16 {
    using Raw = uint16_t;
    static __device__ __forceinline__ float to_float(uint16_t v) { return __uint_as_float(uint32_t{v} << 16); }
    // nearest, ties to even; NaN stays NaN
    static __device__ __forceinline__ uint16_t round(float v) {
        const uint32_t u = __float_as_uint(v);
        if ((u & 0x7fffffffu) > 0x7f800000u) return static_cast<uint16_t>((u >> 16) | 0x40u);
        return static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
    }
};
struct F16 {
    using Raw = uint16_t;
    static __device__ __forceinline__ float to_float(uint16_t v) {
        return static_cast<float>(__builtin_bit_cast(_Float16, v));
    }
    static __device__ __forceinline__ uint16_t round(float v) {
        return __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    }
};

template <class T>
struct Vec8 {
    typename T::Raw e[8];
};

// Eight elements at p (any alignment of p that its type allows; global memory
// takes unaligned wide loads), or the first n of them and zeros.
template <class T>
__device__ __forceinline__ Vec8<T> load8(const typename T::Raw *p, int n) {
    Vec8<T> v;
    if (n >= 8) {
        __builtin_memcpy(&v, p, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.e[i] = i < n ? p[i] : typename T::Raw(0);
    }
    return v;
}
template <class T>
__device__ __forceinline__ void store8(typename T::Raw *p, const Vec8<T> &v, int n) {
    if (n >= 8) {
        __builtin_memcpy(p, &v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v.e[i];
    }
}

// Largest magnitude by its bits: unlike a floating maximum it keeps NaN, and
// infinities and NaN compare above every finite value.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint64_t abs_bits(double v) {
    return __builtin_bit_cast(uint64_t, v) & 0x7fffffffffffffffull;
}
constexpr uint64_t kInf64 = 0x7ff0000000000000ull;

// fp32 arithmetic on v is used where the largest |v| lies in [2^-60, 2^100):
// below, products and exponentials may have lost bits to underflow that
// matter next to it; above, or where it is no number, some may have
// overflowed.  Other rows (blocks) take the fp64 path.
constexpr uint32_t kLeast32 = (127u - 60u) << 23;
constexpr uint32_t kMost32 = (127u + 100u) << 23;
__device__ __forceinline__ bool plain_range(uint32_t bits) { return bits >= kLeast32 && bits < kMost32; }

template <int OP>
__device__ __forceinline__ double value64(float a, float b) {
    if constexpr (OP == kOpNorm) {
        return static_cast<double>(a) * static_cast<double>(b);
    } else {
        if (a == 0.0f || b == 0.0f) return 0.0 * (static_cast<double>(a) + static_cast<double>(b));
        const double g = static_cast<double>(a);
        return g / (1.0 + exp(-g)) * static_cast<double>(b);
    }
}

// The same in fp32.  act: relative error at most 10 * 2^-24 in the range
// above: e^-g = 2^hi (1 + lo ln 2) with hi + lo = -g log2 e to twice the
// precision (2^hi and the reciprocal are off by 2^-23 each, the other six
// operations by 2^-24).  Below g = -80 the exponential may overflow; the
// value is then at most 80 e^-80 |u|, nothing next to 2^-60 unless |u| is
// huge: such a value is reported as out of range.
template <int OP>
__device__ __forceinline__ float value32(float a, float b) {
    if constexpr (OP == kOpNorm) {
        return a * b;
    } else {
        constexpr float kLog2e = 1.44269502162933349609375f;   // fp32 nearest to log2 e
        constexpr float kLog2eLo = 1.92596299112661746887e-8f;  // log2 e - kLog2e
        const float hi = a * -kLog2e;
        const float lo = __builtin_fmaf(a, -kLog2e, -hi) - a * kLog2eLo;
        float e = __builtin_amdgcn_exp2f(hi);
        e = hi < 120.0f ? __builtin_fmaf(e, lo * 0.693147182f, e) : e;
        float v = a * __builtin_amdgcn_rcpf(1.0f + e) * b;
        if (a < -80.0f) v = fabsf(b) > 1048576.0f ? __builtin_inff() : 0.0f;
        return v + ((a - a) + (b - b));  // NaN where a or b is no finite number
    }
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), s)));
    return v;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) {
        const uint64_t o = __shfl_xor(static_cast<unsigned long long>(v), s);
        v = o > v ? o : v;
    }
    return v;
}
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    return v;
}
// Maximum over the 16 lanes that share a block of 128 columns.
template <class U>
__device__ __forceinline__ U block128_max(U v) {
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) {
        U o;
        if constexpr (sizeof(U) == 4)
            o = static_cast<U>(__shfl_xor(static_cast<int>(v), s));
        else
            o = static_cast<U>(__shfl_xor(static_cast<unsigned long long>(v), s));
        v = o > v ? o : v;
    }
    return v;
}

// Scale of a row or block whose largest |v| is m: 0 for zeros (also where
// eps = 0 leaves the root of a row of zeros infinite).
__device__ __forceinline__ float scale_of(double m, double inv, double top, bool number) {
    return !number ? __builtin_nanf("") : m == 0.0 ? 0.0f : static_cast<float>(m * inv / top);
}

// How near a border the fp32 quotient counts as undecided.  Error of t = v k:
// k = 127 / max|v| rounded once, the product once, v by at most 10 * 2^-24:
// 12 * 2^-24 * 127 < 2^-13.
constexpr float kNear = 0x1p-13f;

template <class T, int THREADS, int NV, int OP, int FMT>
__global__ void __launch_bounds__(THREADS == 64 ? 256 : THREADS) quant_rows_kernel(RowArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
    using Raw = typename T::Raw;
    constexpr int WAVES = THREADS / 64;
    constexpr int KEEP = NV > 0 ? NV : 1;
    __shared__ double sh_sum[WAVES];
    __shared__ uint32_t sh_max[WAVES];
    __shared__ uint64_t sh_max64[WAVES];
    const int t = THREADS == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int wave = t >> 6;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block(THREADS) +
                        (THREADS == 64 ? threadIdx.x >> 6 : 0);
    if (row >= g.rows) return;  // whole waves of the one-wave shape, which has no barrier
    const Raw *pa = static_cast<const Raw *>(g.a) + row * g.lda;
    const Raw *pb = g.b ? static_cast<const Raw *>(g.b) + row * g.ldb : nullptr;
    const Raw *pw = static_cast<const Raw *>(g.weight);
    Raw *psum = g.sum ? static_cast<Raw *>(g.sum) + row * g.ldsum : nullptr;
    uint8_t *pq = static_cast<uint8_t *>(g.q) + row * g.ldq;
    const int nv = NV > 0 ? NV : (g.cols + THREADS * 8 - 1) / (THREADS * 8);

    // norm: h and w; act: gate and up.  `again`: the second reading of a row
    // that is not kept, by when a + b may have replaced a or b in place.
    auto fetch = [&](int v, Vec8<T> &a, Vec8<T> &b, bool again) -> int {
        const int c = (v * THREADS + t) * 8;
        const int n = g.cols - c;
        if (n <= 0) {
            a = Vec8<T>{};
            b = Vec8<T>{};
            return n;
        }
        if constexpr (OP == kOpAct) {
            a = load8<T>(pa + c, n);
            b = load8<T>(pb + c, n);
        } else {
            b = load8<T>(pw + c, n);
            if (again && psum) {
                a = load8<T>(psum + c, n);
            } else {
                a = load8<T>(pa + c, n);
                if (pb) {
                    const Vec8<T> r = load8<T>(pb + c, n);
#pragma unroll
                    for (int i = 0; i < 8; ++i) a.e[i] = T::round(T::to_float(a.e[i]) + T::to_float(r.e[i]));
                }
                if (psum) store8<T>(psum + c, a, n);
            }
        }
        return n;
    };
    auto values = [&](const Vec8<T> &a, const Vec8<T> &b, float *v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = value32<OP>(T::to_float(a.e[i]), T::to_float(b.e[i]));
    };
    auto value_at = [&](const Vec8<T> &a, const Vec8<T> &b, int i) {
        return value64<OP>(T::to_float(a.e[i]), T::to_float(b.e[i]));
    };
    auto max_at64 = [&](const Vec8<T> &a, const Vec8<T> &b) {
        uint64_t m = 0;
        for (int i = 0; i < 8; ++i) {
            const uint64_t o = abs_bits(value_at(a, b, i));
            m = o > m ? o : m;
        }
        return m;
    };

    Vec8<T> ka[KEEP], kb[KEEP];
    double sum = 0.0;
    uint32_t most = 0;
    auto first = [&](int v, Vec8<T> &a, Vec8<T> &b) {
        fetch(v, a, b, false);
        float f[8];
        if constexpr (FMT == kFmtS8) {
            values(a, b, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) most = max(most, abs_bits(f[i]));
        }
        if constexpr (OP == kOpNorm) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double h = static_cast<double>(T::to_float(a.e[i]));
                sum = __builtin_fma(h, h, sum);
            }
        }
    };
    if constexpr (NV > 0) {
#pragma unroll
        for (int v = 0; v < NV; ++v) first(v, ka[v], kb[v]);
    } else {
        for (int v = 0; v < nv; ++v) first(v, ka[0], kb[0]);
    }

    // Over the row: the sum of squares and the largest |v|.
    if constexpr (OP == kOpNorm) sum = wave_sum(sum);
    if constexpr (FMT == kFmtS8) most = wave_max(most);
    if constexpr (WAVES > 1 && (OP == kOpNorm || FMT == kFmtS8)) {
        if ((t & 63) == 0) {
            sh_sum[wave] = sum;
            sh_max[wave] = most;
        }
        __syncthreads();
        sum = 0.0;
        most = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            sum += sh_sum[w];
            most = max(most, sh_max[w]);
        }
    }
    const double inv = OP == kOpNorm ? 1.0 / sqrt(sum / g.cols + static_cast<double>(g.eps)) : 1.0;

    // For each vector of the row: f(v, a, b).
    auto each = [&](auto &&f) {
        if constexpr (NV > 0) {
#pragma unroll
            for (int v = 0; v < NV; ++v) f(v, ka[v], kb[v]);
        } else {
            for (int v = 0; v < nv; ++v) {
                fetch(v, ka[0], kb[0], true);
                f(v, ka[0], kb[0]);
            }
        }
    };

    if constexpr (FMT == kFmtS8) {
        const bool plain = plain_range(most);
        // The largest |v| in fp64: among the values that may be it (an fp32
        // value is off by less than 2^-20), or among all.  Products of 16-bit
        // types are exact in fp32.
        uint64_t m64 = 0;
        if (plain && OP == kOpNorm && sizeof(Raw) == 2) {
            m64 = abs_bits(static_cast<double>(__uint_as_float(most)));
        } else {
            const uint32_t from = plain ? abs_bits(__uint_as_float(most) * (1.0f - 0x1p-19f)) : 0u;
            each([&](int, const Vec8<T> &a, const Vec8<T> &b) {
                if (plain) {
                    float f[8];
                    values(a, b, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (abs_bits(f[i]) >= from) {
                            const uint64_t o = abs_bits(value_at(a, b, i));
                            m64 = o > m64 ? o : m64;
                        }
                } else {
                    const uint64_t o = max_at64(a, b);
                    m64 = o > m64 ? o : m64;
                }
            });
            m64 = wave_max(m64);
            if constexpr (WAVES > 1) {
                if ((t & 63) == 0) sh_max64[wave] = m64;
                __syncthreads();
                m64 = 0;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) m64 = sh_max64[w] > m64 ? sh_max64[w] : m64;
            }
        }
        const double m = __builtin_bit_cast(double, m64);
        const bool number = m64 < kInf64;
        if (t == 0) g.scale[row] = scale_of(m, inv, 127.0, number);
        const float k = plain ? static_cast<float>(127.0 / m) : 0.0f;
        each([&](int v, const Vec8<T> &a, const Vec8<T> &b) {
            const int c = (v * THREADS + t) * 8;
            const int n = g.cols - c;
            if (n <= 0) return;
            int q[8];
            if (plain) {
                float f[8];
                values(a, b, f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = f[i] * k;
                    const float r = rintf(x);
                    q[i] = static_cast<int>(r);
                    if (fabsf(x - r) > 0.5f - kNear)
                        q[i] = static_cast<int>(rint(value_at(a, b, i) * 127.0 / m));
                }
            } else {
                for (int i = 0; i < 8; ++i)
                    q[i] = number && m64 != 0 ? static_cast<int>(rint(value_at(a, b, i) * 127.0 / m)) : 0;
            }
            uint32_t w2[2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                w2[h] = (q[4 * h] & 0xff) | (q[4 * h + 1] & 0xff) << 8 | (q[4 * h + 2] & 0xff) << 16 |
                        static_cast<uint32_t>(q[4 * h + 3]) << 24;
            if (n >= 8) {
                __builtin_memcpy(pq + c, w2, 8);
            } else {
                for (int i = 0; i < n; ++i) pq[c + i] = static_cast<uint8_t>(w2[i >> 2] >> (8 * (i & 3)));
            }
        });
    } else {
        each([&](int v, const Vec8<T> &a, const Vec8<T> &b) {
            const int c = (v * THREADS + t) * 8;
            const int n = g.cols - c;
            float f[8];
            values(a, b, f);
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) bits = max(bits, abs_bits(f[i]));
            bits = block128_max(bits);  // lanes past the row hold zeros
            double m;
            bool number = true;
            if (plain_range(bits)) {
                const float mf = __uint_as_float(bits);
                const float k = 448.0f / mf;
                m = mf;
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= k;
            } else {
                // the 16 lanes of a block come here together
                const uint64_t m64 = block128_max(max_at64(a, b));
                m = __builtin_bit_cast(double, m64);
                number = m64 < kInf64;
                for (int i = 0; i < 8; ++i)
                    f[i] = number && m64 != 0 ? static_cast<float>(value_at(a, b, i) * 448.0 / m) : 0.0f;
            }
            if (n <= 0) return;
            if ((t & 15) == 0) g.scale[row * g.lds + (c >> 7)] = scale_of(m, inv, 448.0, number);
            int w2[2] = {0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w2[h] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h], f[4 * h + 1], 0, false);
                w2[h] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2], f[4 * h + 3], w2[h], true);
            }
            if (n >= 8) {
                __builtin_memcpy(pq + c, w2, 8);
            } else {
                for (int i = 0; i < n; ++i)
                    pq[c + i] = static_cast<uint8_t>(static_cast<uint32_t>(w2[i >> 2]) >> (8 * (i & 3)));
            }
        });
    }
#endif
}

}  // namespace tdi8

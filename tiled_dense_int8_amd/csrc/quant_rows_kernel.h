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
// |v| only and the root goes into the scale.  q is exact: the integer nearest
// to the real quotient, or the e4m3 value nearest to the real quotient rounded
// to fp32, ties to even.  The quotient is first taken in fp32 with a known
// error (kNear, kOff); where it lies that near a border between two values it
// is taken again in fp64.  Without this, values next to a border would round by
// the last bit of a sum or an exponential, and two orders of the same
// computation would give different bytes.  The sum of squares is held in fp64:
// finite inputs cannot overflow it, and it then says whether a row holds an
// infinity or NaN.
//
// A row (f8: block) that holds an infinity or NaN has q = 0 and scale = NaN,
// so that products with it come out NaN; one of zeros has q = 0 and scale = 0.
// The other f8 blocks of a norm's row that holds one are values over the row's
// root: zeros over an infinity, NaN over NaN.
//
// Bound by memory: 3 T-sized streams and 1 byte per element (norm with a
// residual), read and written once.  A row stays in registers between its
// reduction and its quotients (up to 16384 columns; longer rows are read
// twice, the second time mostly from the cache), each thread holding vectors
// of 8 columns, so a block of 128 columns is 16 neighbouring lanes and its
// maximum needs no shared memory.
//
// Measured on MI355X (bytes read and written once over the time; a device
// copy of 1 GiB runs at 5.2 TB/s): norm of 16384 x 8192 bf16 with a residual
// 162 us (5.8 TB/s) s8, 163 us f8; 4096 x 16384 89 us (5.3 TB/s); 2048 x 20000,
// read twice, 84 us (3.4 TB/s) s8, 73 us f8.  act of 8192 x 11008 bf16 118 us
// (3.8 TB/s) s8, 100 us (4.5 TB/s) f8: there the vector units count, active in
// 69% (s8) and 89% (f8) of the cycles.  Both execute the same number of
// instructions within 3%; s8's waves wait longer (57% of their cycles against 37%), for
// the row's two reductions across a block of 512 threads, which f8 has not.  A
// single row of 4096 columns takes 3 us, most of it the launch.
#pragma once

#include "quant_rows.h"

namespace tdi8 {

// Eight elements as 32-bit words: one each for F32, two elements in each for
// the 16-bit types.
// kHalf: products of two magnitudes stay below 2^32, and halves are normal fp32 numbers.
struct F32 {
    static constexpr bool kHalf = false;
    static constexpr int kBytes = 4;
    typedef uint32_t Words __attribute__((ext_vector_type(8)));
    static __device__ __forceinline__ float get(const Words &w, int i) { return __uint_as_float(w[i]); }
    static __device__ __forceinline__ void set2(Words &w, int i, float a, float b) {
        w[i] = __float_as_uint(a);
        w[i + 1] = __float_as_uint(b);
    }
};
struct Bf16 {
    static constexpr bool kHalf = false;
    static constexpr int kBytes = 2;
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    static __device__ __forceinline__ float get(const Words &w, int i) {
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    // nearest, ties to even (v_cvt_pk_bf16_f32)
    static __device__ __forceinline__ void set2(Words &w, int i, float a, float b) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
        w[i >> 1] = __builtin_bit_cast(uint32_t, v);
    }
};
struct F16 {
    static constexpr bool kHalf = true;
    static constexpr int kBytes = 2;
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    static __device__ __forceinline__ float get(const Words &w, int i) {
        const uint32_t pair = w[i >> 1];
        return static_cast<float>(__builtin_bit_cast(f16x2, pair)[i & 1]);
    }
    static __device__ __forceinline__ void set2(Words &w, int i, float a, float b) {
        w[i >> 1] = __builtin_bit_cast(uint32_t, f16x2{static_cast<_Float16>(a), static_cast<_Float16>(b)});
    }
};

template <class T>
struct Vec8 {
    static constexpr int kWords = 2 * T::kBytes;
    typename T::Words w;
    __device__ __forceinline__ float get(int i) const { return T::get(w, i); }
    // Element i of a run-time index, for paths that few rows take: a loop
    // over it keeps them short.
    __device__ __forceinline__ float pick(int i) const {
        float v = get(0);
#pragma unroll
        for (int j = 1; j < 8; ++j) v = i == j ? get(j) : v;
        return v;
    }
};

// The elements moved down by one, zero at the top.
template <class T>
__device__ __forceinline__ void shift_down(Vec8<T> &v) {
    constexpr int W = Vec8<T>::kWords;
#pragma unroll
    for (int j = 0; j + 1 < W; ++j) v.w[j] = T::kBytes == 4 ? v.w[j + 1] : v.w[j] >> 16 | v.w[j + 1] << 16;
    v.w[W - 1] = T::kBytes == 4 ? 0u : v.w[W - 1] >> 16;
}

// Eight elements at p, at any alignment that their type allows (global memory
// takes unaligned wide loads).
template <class T>
__device__ __forceinline__ void load8(Vec8<T> &v, const char *p) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int h = 0; h < Vec8<T>::kWords / 4; ++h) {
        u32x4 x;
        __builtin_memcpy(&x, p + 16 * h, 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) v.w[4 * h + j] = x[j];
    }
}
// The first n < 8 elements at p and zeros, for rows shorter than 8.
template <class T>
__device__ __forceinline__ void load_few(Vec8<T> &v, const char *p, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t e = 0;
        if (i < n) {
            if constexpr (T::kBytes == 4)
                e = reinterpret_cast<const uint32_t *>(p)[i];
            else
                e = reinterpret_cast<const uint16_t *>(p)[i];
        }
        if constexpr (T::kBytes == 4)
            v.w[i] = e;
        else
            v.w[i >> 1] = i & 1 ? v.w[i >> 1] | e << 16 : e;
    }
}
// Eight elements to p, or the first n.
template <class T>
__device__ __forceinline__ void store8(char *p, Vec8<T> v, int n) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if (n >= 8) {
#pragma unroll
        for (int h = 0; h < Vec8<T>::kWords / 4; ++h) {
            const u32x4 x = {v.w[4 * h], v.w[4 * h + 1], v.w[4 * h + 2], v.w[4 * h + 3]};
            __builtin_memcpy(p + 16 * h, &x, 16);
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
            if constexpr (T::kBytes == 4)
                reinterpret_cast<uint32_t *>(p)[i] = v.w[0];
            else
                reinterpret_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(v.w[0]);
            shift_down(v);
        }
    }
}
// Eight bytes at p, or the first n.
__device__ __forceinline__ void store8_bytes(uint8_t *p, uint32_t lo, uint32_t hi, int n) {
    uint64_t v = static_cast<uint64_t>(hi) << 32 | lo;
    if (n >= 8) {
        __builtin_memcpy(p, &v, 8);
    } else {
#pragma unroll 1
        for (int i = 0; i < n; ++i, v >>= 8) p[i] = static_cast<uint8_t>(v);
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
// operations by 2^-24).  Below g = -80 it takes e^80, so that the exponential
// cannot overflow; the value is then below 2 * 10^-35 |g u| instead of next to
// nothing.  While |g u| is at most 2^32 that is 10^-7 of a row's 2^-60 and 4 *
// 10^-5 of the f8 quotient's scale, against a border to the least e4m3 value
// at 2^-10.  A gate so small that half of it is no normal number is off by
// 2^-150; times |u| up to 2^40 that is 2^-50 of 2^-60.  values32 sees to both
// limits.  NaN and infinities come out as NaN or an infinity.
template <int OP>
__device__ __forceinline__ float value32(float a, float b) {
    if constexpr (OP == kOpNorm) {
        return a * b;
    } else {
        constexpr float kLog2e = 1.44269502162933349609375f;   // fp32 nearest to log2 e
        constexpr float kLog2eLo = 1.92596299112661746887e-8f;  // log2 e - kLog2e
        const float g = fmaxf(a, -80.0f);
        const float hi = g * -kLog2e;
        const float lo = __builtin_fmaf(g, -kLog2eLo, __builtin_fmaf(g, -kLog2e, -hi));
        const float e2 = __builtin_amdgcn_exp2f(hi);
        const float e = __builtin_fmaf(e2, lo * 0.693147182f, e2);
        return a * __builtin_amdgcn_rcpf(1.0f + e) * b;
    }
}
// Eight of them; one is an infinity where the fp32 form may not hold, which
// sends the row (block) to the fp64 path: where the largest |g| times the
// largest |u| of the eight passes 2^32, or the latter 2^40 (2^-8 times it 2^32).
template <class T, int OP>
__device__ __forceinline__ void values32(const Vec8<T> &a, const Vec8<T> &b, float *v) {
    float am = 0x1p-8f, bm = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = a.get(i), y = b.get(i);
        v[i] = value32<OP>(x, y);
        am = fmaxf(am, fabsf(x));
        bm = fmaxf(bm, fabsf(y));
    }
    if constexpr (OP == kOpAct && !T::kHalf) v[0] = am * bm > 0x1p32f ? __builtin_inff() : v[0];
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

// s8: how near a border the fp32 quotient counts as undecided, above its error.
// t = v k is rounded with its border test in one step (fused), so it is off by
// 127 times the relative errors of v (at most 10 * 2^-24, 2^-24, 0 for the
// activation, the norm of fp32, the norm of 16-bit types), of the maximum's
// fp32 form (2^-24, exact for 16-bit products) and of k (2^-24):
// 12, 3 and 1 times 127 * 2^-24.
template <class T, int OP>
constexpr float kNear = OP == kOpAct ? 0x1p-13f : T::kBytes == 4 ? 0x1p-15f : 0x1p-16f;
// Relative error of the fp32 quotient v k of f8, k = 448 / max|v|: v and the
// maximum by the errors above (twice 10, 1, 0), k and the product by 2^-24
// each, its two sides kOff apart by another two: 24, 6 and 4 times 2^-24 at
// most, the last with an exact maximum (k, its side and the product: 3).
template <class T, int OP>
constexpr float kOff = OP == kOpAct ? 0x1p-19f : T::kBytes == 4 ? 0x1p-21f : 0x1p-22f;

// Four fp32 values as e4m3 bytes, nearest, ties to even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}
// x as an e4m3 byte, by way of fp32: the same byte as a conversion of the fp32
// quotient gives (a quotient within 2^-25 of a border counts as on it).
__device__ __forceinline__ uint32_t e4m3_of(double x) {
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(static_cast<float>(x), 0.0f, 0, false)) & 0xffu;
}

// fp32 values from 2^22 up to 2^23 in magnitude plus this have their integer
// part, rounded to nearest even, in the low mantissa bits.
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23

template <class T, int THREADS, int NV, int OP, int FMT>
__global__ void __launch_bounds__(THREADS == 64 ? 256 : THREADS) quant_rows_kernel(RowArgs g) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int SIZE = T::kBytes;
    constexpr int WAVES = THREADS / 64;
    constexpr bool FEW = NV < 0;  // rows shorter than 8: one wave each, its first thread holds them
    constexpr int KEEP = NV > 0 ? NV : 1;
    __shared__ double sh_sum[WAVES];
    __shared__ uint32_t sh_max[WAVES];
    __shared__ uint64_t sh_max64[WAVES];
    const int t = THREADS == 64 ? threadIdx.x & 63 : threadIdx.x;
    const int wave = t >> 6;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rows_per_block(THREADS) +
                        (THREADS == 64 ? threadIdx.x >> 6 : 0);
    if (row >= g.rows) return;  // whole waves of the one-wave shape, which has no barrier
    const char *pa = static_cast<const char *>(g.a) + row * g.lda * SIZE;
    const char *pb = g.b ? static_cast<const char *>(g.b) + row * g.ldb * SIZE : nullptr;
    const char *pw = static_cast<const char *>(g.weight);
    char *psum = g.sum ? static_cast<char *>(g.sum) + row * g.ldsum * SIZE : nullptr;
    uint8_t *pq = static_cast<uint8_t *>(g.q) + row * g.ldq;
    // f8 activations need no whole row: blockIdx.y takes one block's share of columns
    const int col0 = OP == kOpAct && FMT == kFmtF8 && NV > 0 ? blockIdx.y * (THREADS * KEEP * 8) : 0;
    const int nv = FEW ? 1 : NV > 0 ? NV : (g.cols + THREADS * 8 - 1) / (THREADS * 8);

    // Vector v of the row as it lies: norm x, weight and residual; act gate
    // and up.  `again`: the second reading of a row that is not kept, when
    // x + residual may have replaced either in place.  Without a branch on
    // where the row ends, so that a thread's loads are all in flight at once:
    // a vector that passes the end reads the row's last eight elements, and
    // settle() moves the ones it owns into place.  (The others may just be
    // replaced by their sum in place; they are dropped.)
    auto load = [&](int v, Vec8<T> &a, Vec8<T> &b, Vec8<T> &r, bool again) {
        const int c = col0 + (v * THREADS + t) * 8;
        const char *from = again && psum ? psum : pa;
        if constexpr (FEW) {
            const int n = t == 0 ? g.cols : 0;
            load_few(a, from, n);
            load_few(b, OP == kOpAct ? pb : pw, n);
            if (OP == kOpNorm && pb) load_few(r, pb, n);
            return;
        }
        const int64_t at = static_cast<int64_t>(min(c, g.cols - 8)) * SIZE;
        load8(a, from + at);
        if constexpr (OP == kOpAct) {
            load8(b, pb + at);
        } else {
            if (pb && !(again && psum)) load8(r, pb + at);
            load8(b, pw + at);
        }
    };
    // The vector's own elements in place, zeros past the row; norm: h = x +
    // residual for x.
    auto settle = [&](int v, Vec8<T> &a, Vec8<T> &b, const Vec8<T> &r, bool again) {
        const int c = col0 + (v * THREADS + t) * 8;
        const int n = g.cols - c;
        const bool sums = OP == kOpNorm && pb && !(again && psum);
        if (sums) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) T::set2(a.w, i, a.get(i) + r.get(i), a.get(i + 1) + r.get(i + 1));
        }
        if (!FEW && n < 8) {
#pragma unroll 1
            for (int i = n > 0 ? n : 0; i < 8; ++i) {
                shift_down(a);
                shift_down(b);
            }
        }
        if (sums && psum && n > 0) store8<T>(psum + static_cast<int64_t>(c) * SIZE, a, n);
    };
    auto values = [&](const Vec8<T> &a, const Vec8<T> &b, float *v) { values32<T, OP>(a, b, v); };
    // f8 activations: whether this wave has any of vector v's columns (8192 x
    // 6000: 85 us without, 57; the longer rows of s8 ran 4% slower with it).
    auto has = [&](int v) {
        return OP != kOpAct || FMT != kFmtF8 || col0 + (v * THREADS + __builtin_amdgcn_readfirstlane(wave) * 64) * 8 < g.cols;
    };
    auto value_at = [&](const Vec8<T> &a, const Vec8<T> &b, int i) { return value64<OP>(a.pick(i), b.pick(i)); };
    auto max_at64 = [&](const Vec8<T> &a, const Vec8<T> &b) {
        uint64_t m = 0;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
            const uint64_t o = abs_bits(value_at(a, b, i));
            m = o > m ? o : m;
        }
        return m;
    };
    // For each vector of the row: f(v, values, operands), operands(a, b)
    // giving what the values are made of, for the few that need 64 bits.  The
    // norm's operands are kept and its products made again; the activation's
    // values are kept (an exponential each), and its operands too, but for
    // long s8 rows, which read them again when asked (8192 x 11008: 136 us
    // with them in registers, 119 without; 8192 x 4096: 40 and 44).
    constexpr bool KEEP_VALUES = NV > 0 && OP == kOpAct;
    constexpr bool READ_AGAIN = KEEP_VALUES && FMT == kFmtS8 && NV > 2;
    Vec8<T> ka[KEEP], kb[KEEP], kr[KEEP];
    float kv[KEEP_VALUES ? KEEP : 1][8];
    auto each = [&](auto &&f) {
        if constexpr (KEEP_VALUES) {
#pragma unroll
            for (int v = 0; v < KEEP; ++v) {
                if (!has(v)) continue;
                f(v, kv[v], [&](Vec8<T> &a, Vec8<T> &b) {
                    if constexpr (READ_AGAIN) {
                        Vec8<T> none;
                        load(v, a, b, none, true);
                        settle(v, a, b, none, true);
                    } else {
                        a = ka[v];
                        b = kb[v];
                    }
                });
            }
        } else if constexpr (NV != 0) {
#pragma unroll
            for (int v = 0; v < KEEP; ++v) {
                // hides that the products are those of the first pass, which
                // the compiler would otherwise keep in registers
#pragma unroll
                for (int j = 0; j < Vec8<T>::kWords; ++j) {
                    uint32_t word = ka[v].w[j];
                    asm volatile("" : "+v"(word));
                    ka[v].w[j] = word;
                }
                values(ka[v], kb[v], kv[0]);
                f(v, kv[0], [&](Vec8<T> &a, Vec8<T> &b) {
                    a = ka[v];
                    b = kb[v];
                });
            }
        } else {
            for (int v = 0; v < nv; ++v) {
                load(v, ka[0], kb[0], kr[0], true);
                settle(v, ka[0], kb[0], kr[0], true);
                values(ka[0], kb[0], kv[0]);
                f(v, kv[0], [&](Vec8<T> &a, Vec8<T> &b) {
                    a = ka[0];
                    b = kb[0];
                });
            }
        }
    };

    // Over the row: the sum of squares and the largest |v|.
    double sum = 0.0;
    uint32_t most = 0;
    auto first = [&](const Vec8<T> &a, const Vec8<T> &b, float *f) {
        if constexpr (FMT == kFmtS8 || KEEP_VALUES) values(a, b, f);
        if constexpr (FMT == kFmtS8) {
#pragma unroll
            for (int i = 0; i < 8; ++i) most = max(most, abs_bits(f[i]));
        }
        if constexpr (OP == kOpNorm) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double h = static_cast<double>(a.get(i));
                sum = __builtin_fma(h, h, sum);
            }
        }
    };
    if constexpr (NV != 0) {
#pragma unroll
        for (int v = 0; v < KEEP; ++v) load(v, ka[v], kb[v], kr[v], false);
#pragma unroll
        for (int v = 0; v < KEEP; ++v) {
            if (KEEP_VALUES && !has(v)) continue;
            settle(v, ka[v], kb[v], kr[v], false);
            first(ka[v], kb[v], kv[KEEP_VALUES ? v : 0]);
        }
    } else if constexpr (OP == kOpNorm || FMT == kFmtS8) {
        for (int v = 0; v < nv; ++v) {
            load(v, ka[0], kb[0], kr[0], false);
            settle(v, ka[0], kb[0], kr[0], false);
            first(ka[0], kb[0], kv[0]);
        }
    }
    [[maybe_unused]] const uint32_t mine = most;  // this thread's part
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
    auto root = [&]() {
        return OP == kOpNorm ? 1.0 / sqrt(sum / g.cols + static_cast<double>(g.eps)) : 1.0;
    };

    if constexpr (FMT == kFmtS8) {
        const bool plain = plain_range(most);
        // The largest |v| in fp64: among the values that may be it (an fp32
        // value is off by less than 2^-20), or among all.  Products of 16-bit
        // types are exact in fp32.
        uint64_t m64 = 0;
        if (plain && OP == kOpNorm && SIZE == 2) {
            m64 = abs_bits(static_cast<double>(__uint_as_float(most)));
        } else {
            const uint32_t from = plain ? abs_bits(__uint_as_float(most) * (1.0f - 0x1p-19f)) : 0u;
            if (mine >= from) {
                each([&](int, const float *f, auto &&operands) {
                    uint32_t which = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) which |= abs_bits(f[i]) >= from ? 1u << i : 0u;
                    if (which == 0) return;
                    Vec8<T> a, b;
                    operands(a, b);
                    for (; which != 0; which &= which - 1) {
                        const int i = __builtin_ctz(which);
                        const uint64_t o = abs_bits(value64<OP>(a.pick(i), b.pick(i)));
                        m64 = o > m64 ? o : m64;
                    }
                });
            }
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
        const float k = plain ? 127.0f / static_cast<float>(m) : 0.0f;
        each([&](int v, const float *f, auto &&operands) {
            const int c = col0 + (v * THREADS + t) * 8;
            const int n = g.cols - c;
            if (n <= 0) return;
            uint32_t w2[2] = {0, 0};
            float near = 1.0f;
            if (plain) {
                uint32_t y[8];
                near = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float r = __builtin_fmaf(f[i], k, kRound);
                    y[i] = __float_as_uint(r);
                    near = fmaxf(near, fabsf(__builtin_fmaf(f[i], k, kRound - r)));
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    w2[h] = __builtin_amdgcn_perm(
                        __builtin_amdgcn_perm(y[4 * h + 3], y[4 * h + 2], 0x0c0c0400u),
                        __builtin_amdgcn_perm(y[4 * h + 1], y[4 * h], 0x0c0c0400u), 0x05040100u);
            }
            if (near > 0.5f - kNear<T, OP>) {
                Vec8<T> a, b;
                operands(a, b);
                uint64_t q = static_cast<uint64_t>(w2[1]) << 32 | w2[0];
                auto undecided = [&](float x) {
                    const float r = __builtin_fmaf(x, k, kRound);
                    return !plain || fabsf(__builtin_fmaf(x, k, kRound - r)) > 0.5f - kNear<T, OP>;
                };
                auto decide = [&](int i, float x, float y) {
                    const int qi = number && m64 != 0 ? static_cast<int>(rint(value64<OP>(x, y) * 127.0 / m)) : 0;
                    q = (q & ~(0xffull << (8 * i))) | static_cast<uint64_t>(static_cast<uint8_t>(qi)) << (8 * i);
                };
                if constexpr (OP == kOpNorm && NV > 2) {
                    // one index for all lanes and each product made again:
                    // fewest registers for long rows; short ones take the
                    // other, faster form (1000 x 2999 fp32: 8.3 and 7.0 us)
#pragma unroll 1
                    for (int i = 0; i < 8; ++i) {
                        const float x = a.pick(i), y = b.pick(i);
                        if (undecided(value32<OP>(x, y))) decide(i, x, y);
                    }
                } else {
                    uint32_t which = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) which |= undecided(f[i]) ? 1u << i : 0u;
                    for (; which != 0; which &= which - 1) {
                        const int i = __builtin_ctz(which);
                        decide(i, a.pick(i), b.pick(i));
                    }
                }
                w2[0] = static_cast<uint32_t>(q);
                w2[1] = static_cast<uint32_t>(q >> 32);
            }
            store8_bytes(pq + c, w2[0], w2[1], n);
        });
        if (t == 0) g.scale[row] = scale_of(m, root(), 127.0, number);
    } else {
        const double inv = root();
        const bool rooted = OP != kOpNorm || sum < __builtin_inf();
        each([&](int v, const float *f, auto &&operands) {
            const int c = col0 + (v * THREADS + t) * 8;
            const int n = g.cols - c;
            uint32_t bits = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) bits = max(bits, abs_bits(f[i]));
            const uint32_t own = bits;
            bits = block128_max(bits);  // lanes past the row hold zeros
            const bool plain = plain_range(bits);
            double m = __uint_as_float(bits);
            bool number = true;
            uint32_t w2[2] = {0, 0}, diff[2] = {~0u, ~0u};
            if (plain) {
                // The quotients a little low and a little high: where both
                // round to the same bytes those are right.
                const float k = 448.0f / __uint_as_float(bits);
                const float low = k * (1.0f - kOff<T, OP>), high = k * (1.0f + kOff<T, OP>);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    w2[h] = e4m3x4(f[4 * h] * low, f[4 * h + 1] * low, f[4 * h + 2] * low, f[4 * h + 3] * low);
                    diff[h] = w2[h] ^ e4m3x4(f[4 * h] * high, f[4 * h + 1] * high, f[4 * h + 2] * high,
                                             f[4 * h + 3] * high);
                }
            }
            // Others are decided in fp64, by all 16 lanes of the block together.
            const uint64_t undecided = __ballot((diff[0] | diff[1]) != 0);
            if ((undecided >> (t & 48) & 0xffff) != 0) {
                Vec8<T> a, b;
                operands(a, b);
                if (!(plain && OP == kOpNorm && SIZE == 2)) {
                    // the largest |v|, as for s8
                    const uint32_t from = plain ? abs_bits(__uint_as_float(bits) * (1.0f - 0x1p-19f)) : 0u;
                    uint64_t m64 = 0;
                    if (own >= from) {
                        uint32_t which = plain ? 0u : 0xffu;
#pragma unroll
                        for (int i = 0; i < 8; ++i) which |= abs_bits(f[i]) >= from ? 1u << i : 0u;
                        for (; which != 0; which &= which - 1) {
                            const int i = __builtin_ctz(which);
                            const uint64_t o = abs_bits(value64<OP>(a.pick(i), b.pick(i)));
                            m64 = o > m64 ? o : m64;
                        }
                    }
                    m64 = block128_max(m64);
                    m = __builtin_bit_cast(double, m64);
                    number = m64 < kInf64;
                }
                uint64_t q = static_cast<uint64_t>(w2[1]) << 32 | w2[0];
                const uint64_t d = static_cast<uint64_t>(diff[1]) << 32 | diff[0];
#pragma unroll 1
                for (int i = 0; i < 8; ++i) {
                    if ((d >> (8 * i) & 0xff) == 0) continue;
                    const uint32_t byte = number && m != 0.0 ? e4m3_of(value64<OP>(a.pick(i), b.pick(i)) * 448.0 / m) : 0u;
                    q = (q & ~(0xffull << (8 * i))) | static_cast<uint64_t>(byte) << (8 * i);
                }
                w2[0] = static_cast<uint32_t>(q);
                w2[1] = static_cast<uint32_t>(q >> 32);
            }
            if (n <= 0) return;
            if (!rooted) {
                w2[0] = w2[1] = 0;
                number = number && sum == sum;
            }
            if ((t & 15) == 0) g.scale[row * g.lds + (c >> 7)] = scale_of(m, inv, 448.0, number);
            store8_bytes(pq + c, w2[0], w2[1], n);
        });
    }
#endif
}

}  // namespace tdi8

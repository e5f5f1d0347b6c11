// What the norm's kernels share: chunks of 16 bytes of a row, sums over the lanes
// that hold a row, 1 / sqrt(mean + eps), and the whole numbers of the 8-bit form.
#pragma once

#include "i8.hpp"

namespace sgemm {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// A value rounded to FP32 before it is rounded to a type. (The compiler would otherwise take some
// products and their conversion to half in one instruction, with one rounding, and others not.)
__device__ __forceinline__ float as_f32(float v) {
    asm("" : "+v"(v));
    return v;
}

// N elements of a row (16 bytes, if not said otherwise) at an address aligned to its element only, as FP32.
template <class T, int N_ = 16 / (int)sizeof(T)>
struct Chunk {
    static constexpr int N = N_;
    typedef T Vec __attribute__((ext_vector_type(N)));
    typedef Vec VecU __attribute__((aligned(sizeof(T))));
    float v[N];

    // Elements at .. at + N - 1 of a row of n; zeros past its end.
    __device__ __forceinline__ void load(const T* row, int at, int n) {
        if (at + N <= n) {
            const Vec x = *(const VecU*)(row + at);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = (float)x[e];
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = at + e < n ? (float)row[at + e] : 0.0f;
        }
    }
    __device__ __forceinline__ void store(T* row, int at, int n) const {
        if (at + N <= n) {
            Vec x;
#pragma unroll
            for (int e = 0; e < N; ++e) x[e] = (T)v[e];
            *(VecU*)(row + at) = x;
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (at + e < n) row[at + e] = (T)v[e];
        }
    }
};

// The same 16 bytes as they are stored, for rows that stay in registers. Where a chunk would reach past the row's
// end, the row's last 16 bytes are taken instead (`place_of`): their first elements are another lane's too, so sums
// leave them out (`first`), while both lanes store the same results there. No load or store is then apart from
// the others. Rows of less than 16 bytes (SHORT) are one lane's, element by element.
template <class T>
struct Raw {
    static constexpr int N = 16 / (int)sizeof(T);
    typedef T Vec __attribute__((ext_vector_type(N)));
    typedef Vec VecU __attribute__((aligned(sizeof(T))));
    Vec v;

    template <bool SHORT>
    __device__ __forceinline__ static uint32_t place_of(int at, int n) {
        return SHORT ? 0 : (uint32_t)(at < n - N ? at : n - N);
    }
    // The first element of the chunk at `place`, meant to be at `at`, that is this lane's. (Computed
    // anew for each row: the compiler would otherwise keep one mask for each element of a chunk.)
    __device__ __forceinline__ static int first(int at, uint32_t place) {
        int k = at - (int)place;
        asm volatile("" : "+v"(k));
        return k;
    }
    template <bool SHORT>
    __device__ __forceinline__ void load(const T* row, uint32_t place, int n) {
        if constexpr (!SHORT) {
            v = *(const VecU*)(row + place);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const T y = row[e < n ? e : n - 1];
                v[e] = e < n ? y : (T)0.0f;
            }
        }
    }
    template <bool SHORT>
    __device__ __forceinline__ void store(T* row, uint32_t place, int n) const {
        if constexpr (!SHORT) {
            *(VecU*)(row + place) = v;
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (e < n) row[e] = v[e];
        }
    }
    // The compiler keeps what it has converted to FP32 for the next pass, and converts several chunks
    // ahead, for twice the registers; past this it converts again, behind what was stored before.
    __device__ __forceinline__ void forget() {
        i32x4 x = __builtin_bit_cast(i32x4, v);
        asm volatile("" : "+v"(x)::"memory");
        v = __builtin_bit_cast(Vec, x);
    }
    // Whether any element is not zero (of either sign).
    __device__ __forceinline__ uint32_t any() const {
        typedef uint32_t U __attribute__((ext_vector_type(4)));
        const U u = __builtin_bit_cast(U, v) & (sizeof(T) == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu);
        return u.x | u.y | u.z | u.w;
    }
};

// Whole numbers of a chunk as bytes.
template <int N>
struct Bytes {
    typedef int W __attribute__((ext_vector_type(N / 4)));
    typedef W Wu __attribute__((aligned(1)));
    __device__ __forceinline__ static void store(int8_t* p, const int (&q)[N]) {
        W w;
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = (q[4 * i] & 255) | (q[4 * i + 1] & 255) << 8 | (q[4 * i + 2] & 255) << 16 | q[4 * i + 3] << 24;
        *(Wu*)p = w;
    }
};
// To a row of int8, as far as it goes.
template <int N>
__device__ __forceinline__ void store_levels(int8_t* row, int at, int n, const int (&q)[N]) {
    if constexpr (N >= 4)
        if (at + N <= n) return Bytes<N>::store(row + at, q);
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (at + e < n) row[at + e] = (int8_t)q[e];
}

struct Plus {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Or {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a | b; }
};
struct Max {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
    __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};

// A value of another lane of 16: data-parallel moves of its words.
template <int CTRL, class V>
__device__ __forceinline__ V moved(V v) {
    constexpr int WORDS = sizeof(V) / 4;
    typedef int W __attribute__((ext_vector_type(WORDS == 1 ? 2 : WORDS)));
    if constexpr (WORDS == 1)
        return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
    else {
        W w = __builtin_bit_cast(W, v);
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = __builtin_amdgcn_update_dpp(0, w[i], CTRL, 0xF, 0xF, true);
        return __builtin_bit_cast(V, w);
    }
}
// f of the values of lanes 16 (32) apart, by the exchange of rows (halves) between two registers.
template <int APART, class V, class Fn>
__device__ __forceinline__ V across(V v, Fn f) {
    constexpr int WORDS = sizeof(V) / 4;
    uint32_t w[WORDS], x[WORDS], y[WORDS];
    __builtin_memcpy(w, &v, sizeof(V));
#pragma unroll
    for (int i = 0; i < WORDS; ++i) {
        if constexpr (APART == 16) {
            const auto r = __builtin_amdgcn_permlane16_swap(w[i], w[i], false, false);
            x[i] = r[0];
            y[i] = r[1];
        } else {
            const auto r = __builtin_amdgcn_permlane32_swap(w[i], w[i], false, false);
            x[i] = r[0];
            y[i] = r[1];
        }
    }
    V a, b;
    __builtin_memcpy(&a, x, sizeof(V));
    __builtin_memcpy(&b, y, sizeof(V));
    return f(a, b);
}

// f over the LANES lanes of a row, the same in all of them (LANES <= 64: parts of a
// wave; beyond, whole waves of one workgroup through `red`, a word for each).
template <int LANES, class V, class Fn>
__device__ __forceinline__ V over_row(V v, Fn f, V* red) {
    static_assert(LANES == 16 || LANES % 64 == 0, "rows of 16 lanes, or whole waves");
    v = f(v, moved<0xB1>(v));    // quad_perm 1,0,3,2
    v = f(v, moved<0x4E>(v));    // quad_perm 2,3,0,1
    v = f(v, moved<0x141>(v));   // row_half_mirror
    v = f(v, moved<0x140>(v));   // row_mirror
    if constexpr (LANES >= 64) {
        v = across<16>(v, f);
        v = across<32>(v, f);
    }
    if constexpr (LANES > 64) {
        constexpr int WAVES = LANES / 64;
        __syncthreads();   // the words of an earlier call have been read
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) v = f(v, red[w]);
    }
    return v;
}

// Squares whose FP32 sum says nothing: beyond its range, or so small that single
// squares have lost their bits (2^-149 each) and eps does not make up for them.
__device__ __forceinline__ bool sum_lost(float ss, float eps) {
    return !(ss <= 3.0e38f) || (ss < 1.0e-30f && eps < 1.0e-20f);
}
// 1 / sqrt(ss / n + eps). A mean of no elements is 0. The reciprocal root of the hardware is off by
// one step; a Newton step takes that away where the mean is an ordinary number.
__device__ __forceinline__ float rstd_of(float ss, int n, float eps) {
    const float v = n > 0 ? ss / (float)n + eps : eps;
    const float r = __builtin_amdgcn_rsqf(v);
    if (!(v >= 1.0e-30f && v <= 1.0e30f)) return (float)(1.0 / sqrt((double)v));
    return __builtin_fmaf(__builtin_fmaf(-v * r, r, 1.0f), 0.5f * r, r);
}
// The same of squares summed times 2^(-2 shift).
__device__ __forceinline__ float rstd_scaled(float ss, int shift, int n, float eps) {
    return (float)(1.0 / sqrt(ldexp((double)ss / n, 2 * shift) + (double)eps));
}

// round(127 v / top), halves to even. The product with 127 / top is off by at
// most 127 x 3 half steps, 0.00003 in FP32, so its nearest whole number is the quotient's unless
// it lies that close to a half f + 1/2; there the sign of 254 v - (2 f + 1) top decides, in
// 64 bits: exactly for FP32 v and top (32 bits each product), and to 2^-52 for v and top that are
// products of two FP32 numbers themselves.
__device__ __forceinline__ double settled(double v, double top, double x) {
    const double f = floor(x), d = __builtin_fma(254.0, v, -(2.0 * f + 1.0) * top);
    const double even = rint(f + 0.5), up = f + 1.0;
    return d > 0.0 ? up : d < 0.0 ? f : even;
}
__device__ __forceinline__ bool near_half(float x, float n) { return fabsf(x - n) > 0.4999f; }
__device__ __forceinline__ bool near_half(double x, double n) { return fabs(x - n) > 0.4999999999; }
// A chunk's whole numbers. One branch for all of its elements, which a wave of 512 elements takes one
// time in ten (FP32).
template <int N, class V>
__device__ __forceinline__ void levels(const V (&v)[N], V inv, V top, int (&q)[N]) {
    V n[N];
    bool close = false;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const V x = v[e] * inv;
        n[e] = __builtin_rint(x);
        close = close || near_half(x, n[e]);
    }
    if (__builtin_amdgcn_ballot_w64(close) != 0) {
        asm volatile("");   // (not to be computed ahead of the branch)
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const V x = v[e] * inv;
            if (near_half(x, n[e])) n[e] = (V)settled((double)v[e], (double)top, (double)x);
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) q[e] = (int)n[e];
}
// Whether the FP32 form serves: 127 / top is an ordinary number, and FP32 products next to
// top have lost no bits.
__device__ __forceinline__ bool ordinary(float top) { return top >= 1.0e-30f && top <= 3.0e38f; }

}  // namespace sgemm

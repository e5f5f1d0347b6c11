// What the norm's kernels share: chunks of 16 bytes of a row, sums over the lanes
// that hold a row, 1 / sqrt(mean + eps), and the whole numbers of the 8-bit form.
#pragma once

#include "i8.hpp"

namespace sgemm {

// 16 bytes of a row at an address aligned to its element only, as FP32.
template <class T>
struct Chunk {
    static constexpr int N = 16 / (int)sizeof(T);
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

// Whole numbers of a chunk to a row of int8.
template <int N>
__device__ __forceinline__ void store_levels(int8_t* row, int at, int n, const int (&q)[N]) {
    if (at + N <= n) {
        typedef int W __attribute__((ext_vector_type(N / 4)));
        typedef W Wu __attribute__((aligned(1)));
        W w;
#pragma unroll
        for (int i = 0; i < N / 4; ++i)
            w[i] = (q[4 * i] & 255) | (q[4 * i + 1] & 255) << 8 | (q[4 * i + 2] & 255) << 16 | q[4 * i + 3] << 24;
        *(Wu*)(row + at) = w;
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (at + e < n) row[at + e] = (int8_t)q[e];
    }
}

struct Plus {
    template <class V>
    __device__ __forceinline__ V operator()(V a, V b) const { return a + b; }
};
struct Max {
    __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
    __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};

// f over the LANES lanes of a row, the same in all of them (LANES <= 64: parts of a
// wave; beyond, whole waves of one workgroup through `red`, a word for each).
template <int LANES, class V, class Fn>
__device__ __forceinline__ V over_row(V v, Fn f, V* red) {
#pragma unroll
    for (int off = (LANES < 64 ? LANES : 64) / 2; off > 0; off >>= 1) v = f(v, __shfl_xor(v, off));
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

// Squares whose FP32 sum says nothing: beyond its range, or so small that
// single squares have lost their bits.
__device__ __forceinline__ bool sum_lost(float ss) { return !(ss <= 3.0e38f) || ss < 1.0e-30f; }
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

// round(127 v / top), halves to even, of FP32 v and top. The FP32 product with
// 127 / top is off by at most 127 x 3 x 2^-24 < 0.00003, so its nearest whole
// number is the quotient's unless it lies that close to a half; those few take the 64-bit quotient,
// which operands of 24 bits never round across a half. top is an ordinary number
// (`ordinary`).
__device__ __forceinline__ bool ordinary(float top) { return top >= 1.0e-30f && top <= 3.0e38f; }
__device__ __forceinline__ int level(float v, float inv, float top) {
    const float x = v * inv;
    float n = rintf(x);
    if (fabsf(x - n) > 0.4999f) n = (float)rint(127.0 * (double)v / (double)top);
    return (int)n;
}
// The same in 64 bits: products of two FP32 numbers, and FP32 numbers next to the ends of their range.
__device__ __forceinline__ int level(double v, double inv, double top) {
    const double x = v * inv;
    double n = rint(x);
    if (fabs(x - n) > 0.4999999999) n = rint(127.0 * v / top);
    return (int)n;
}

}  // namespace sgemm

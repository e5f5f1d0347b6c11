// The 4-bit form of a weight matrix: quantisation with group scales (and zero
// points), and its expansion.
#include "ffn.hpp"

namespace sgemm {

static inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The stored number of w, from the exact quotient w / s rounded to even: the
// FP32 product with 1 / s is within 2^-19 of the quotient (at most 16 in
// magnitude, each of three roundings 2^-24 of it), so unless it lies that close
// to a half its nearest whole number is the quotient's. Closer ones take the
// 64-bit quotient: operands of 24 bits against halves of small whole numbers,
// which it never rounds across.
__device__ __forceinline__ uint32_t quantise(float w, float s, float inv, float z) {
    const float x = w * inv;
    float n = rintf(x);
    if (fabsf(x - n) > 0.49999f) n = (float)rint((double)w / (double)s);
    n = fminf(fmaxf(n + z, 0.0f), 15.0f);
    return (uint32_t)(int)n;
}

// A group's scale and zero point, and what its numbers are made with.
template <class T>
struct GroupForm {
    T scale;
    float s, inv, z;
    bool flat, far;

    // lo <= 0 and hi >= 0 are the group's extremes; `bad` is not 0 if it holds
    // an infinity or NaN.
    __device__ __forceinline__ GroupForm(float lo, float hi, float bad, bool asym) {
        const double exact = asym ? ((double)hi - (double)lo) / 15.0 : (double)fmaxf(hi, -lo) / 7.0;
        scale = bad == 0.0f ? (T)(float)exact : (T)__builtin_nanf("");
        s = (float)scale;
        z = 8.0f;
        if (asym) z = s > 0.0f ? fminf((float)rint(-(double)lo / (double)s), 15.0f) : 0.0f;
        flat = !(s > 0.0f);   // no scale (0 or NaN): every number is the zero point
        inv = flat ? 0.0f : 1.0f / s;
        far = !(inv <= 3.0e38f);   // 1 / s overflows: only the 64-bit quotient serves
    }
    __device__ __forceinline__ uint32_t number(float x) const {
        if (flat) return (uint32_t)(int)z;
        if (far) return (uint32_t)(int)fmin(fmax(rint((double)x / (double)s) + z, 0.0), 15.0);
        return quantise(x, s, inv, z);
    }
};

// Groups of 32 to 512 weights, a power of two: eight weights a lane, so a wave
// takes 512 consecutive weights of a row and each group's extremes
// are reduced over its LANES = group / 8 lanes. W is read once; bound by
// that: 8192 x 8192 FP32 71 us (303 MB, 4.3 TB/s).
template <class T, int LANES>
__global__ __launch_bounds__(256) void k_w4_quantize_row(PackArgs a) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    typedef T8 T8u __attribute__((aligned(sizeof(T))));
    typedef uint32_t u32_u1 __attribute__((aligned(1)));
    const int chunks = (a.K + 511) / 512;
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int64_t row = at / chunks;
    const int k = (int)(at - row * chunks) * 512 + 8 * lane;
    if (row >= a.F) return;
    const T* w = (const T*)a.W + row * a.ldw + k;
    float x[8];
    if (k + 8 <= a.K) {
        const T8 v = *(const T8u*)w;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = k + e < a.K ? (float)w[e] : 0.0f;
    }
    float lo = 0.0f, hi = 0.0f, bad = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        lo = fminf(lo, x[e]);
        hi = fmaxf(hi, x[e]);
        bad += x[e] - x[e];   // 0, or NaN for an infinity or NaN
    }
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, off));
        hi = fmaxf(hi, __shfl_xor(hi, off));
        bad += __shfl_xor(bad, off);
    }
    if (k >= a.K) return;
    const bool asym = a.Z != nullptr;
    const GroupForm<T> form(lo, hi, bad, asym);
    if (lane % LANES == 0) {
        const int g = k / (8 * LANES);
        ((T*)a.S)[row * a.lds + g] = form.scale;
        if (asym) ((T*)a.Z)[row * a.ldz + g] = (T)form.z;
    }
    uint32_t v = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) v |= (k + e < a.K ? form.number(x[e]) : 0u) << (4 * e);
    uint8_t* q = a.Q + row * a.ldq + (k >> 1);
    if (k + 8 <= a.K) {
        *(u32_u1*)q = v;
    } else {
        for (int e = 0; k + e < a.K; e += 2) q[e >> 1] = (uint8_t)(v >> (4 * e));
    }
}

// Any other group: one wave each, W read twice.
template <class T>
__global__ __launch_bounds__(256) void k_w4_quantize(PackArgs a) {
    const int groups = (a.K + a.group - 1) / a.group;
    const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int64_t row = at / groups;
    const int g = (int)(at - row * groups);
    if (row >= a.F) return;
    const int k0 = g * a.group, k1 = a.K - k0 < a.group ? a.K : k0 + a.group;
    const T* w = (const T*)a.W + row * a.ldw;
    float lo = 0.0f, hi = 0.0f, bad = 0.0f;
    for (int k = k0 + lane; k < k1; k += 64) {
        const float x = (float)w[k];
        lo = fminf(lo, x);
        hi = fmaxf(hi, x);
        bad += x - x;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, off));
        hi = fmaxf(hi, __shfl_xor(hi, off));
        bad += __shfl_xor(bad, off);
    }
    const bool asym = a.Z != nullptr;
    const GroupForm<T> form(lo, hi, bad, asym);
    if (lane == 0) {
        ((T*)a.S)[row * a.lds + g] = form.scale;
        if (asym) ((T*)a.Z)[row * a.ldz + g] = (T)form.z;
    }
    uint8_t* q = a.Q + row * a.ldq;
    for (int k = k0 + 2 * lane; k < k1; k += 128) {
        uint32_t v = form.number((float)w[k]);
        if (k + 1 < a.K) v |= form.number((float)w[k + 1]) << 4;
        q[k >> 1] = (uint8_t)v;
    }
}

// Eight weights (four bytes) a thread, all of one group. Bound by the bytes
// written: 8192 x 8192 FP32 49 us (the packed form still cached), 6.2 TB/s.
template <class T>
__global__ __launch_bounds__(256) void k_w4_dequantize(PackArgs a) {
    typedef T T8 __attribute__((ext_vector_type(8)));
    typedef T8 T8u __attribute__((aligned(sizeof(T))));
    typedef uint32_t u32_u1 __attribute__((aligned(1)));
    const int words = (a.K + 7) / 8;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = at / words;
    const int k = (int)(at - row * words) * 8;
    if (row >= a.F) return;
    const uint8_t* q = a.Q + row * a.ldq + (k >> 1);
    const int g = k / a.group;
    const float s = (float)((const T*)a.S)[row * a.lds + g];
    const float z = a.Z != nullptr ? (float)((const T*)a.Z)[row * a.ldz + g] : 8.0f;
    T* w = const_cast<T*>((const T*)a.W) + row * a.ldw + k;
    if (k + 8 <= a.K) {
        const uint32_t v = *(const u32_u1*)q;
        T8 x;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (T)(((float)((v >> (4 * e)) & 15) - z) * s);
        *(T8u*)w = x;
    } else {
        for (int e = 0; k + e < a.K; ++e) w[e] = (T)(((float)((q[e >> 1] >> (4 * (e & 1))) & 15) - z) * s);
    }
}

// Whether k_w4_quantize_row takes the call's groups (a group of at least K is one a row, so it may
// be any multiple of 32).
static bool by_row(const PackArgs& a) { return a.group <= 512 && (a.group & (a.group - 1)) == 0; }
static int64_t quantize_wgs(const PackArgs& a) {
    return cdiv((int64_t)a.F * (by_row(a) ? cdiv(a.K, 512) : cdiv(a.K, a.group)), 4);
}
static int64_t dequantize_wgs(const PackArgs& a) { return cdiv((int64_t)a.F * cdiv(a.K, 8), 256); }

int check_w4_pack(const PackArgs& a) {
    return quantize_wgs(a) <= max_workgroups(256) && dequantize_wgs(a) <= max_workgroups(256)
               ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

hipError_t launch_w4_quantize(int dtype, const PackArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        const dim3 grid((unsigned)quantize_wgs(a)), block(256);
        if (!by_row(a))
            hipLaunchKernelGGL((k_w4_quantize<T>), grid, block, 0, s, a);
        else if (a.group == 32)
            hipLaunchKernelGGL((k_w4_quantize_row<T, 4>), grid, block, 0, s, a);
        else if (a.group == 64)
            hipLaunchKernelGGL((k_w4_quantize_row<T, 8>), grid, block, 0, s, a);
        else if (a.group == 128)
            hipLaunchKernelGGL((k_w4_quantize_row<T, 16>), grid, block, 0, s, a);
        else if (a.group == 256)
            hipLaunchKernelGGL((k_w4_quantize_row<T, 32>), grid, block, 0, s, a);
        else
            hipLaunchKernelGGL((k_w4_quantize_row<T, 64>), grid, block, 0, s, a);
        return hipGetLastError();
    });
}

hipError_t launch_w4_dequantize(int dtype, const PackArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        hipLaunchKernelGGL((k_w4_dequantize<T>), dim3((unsigned)dequantize_wgs(a)), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace sgemm

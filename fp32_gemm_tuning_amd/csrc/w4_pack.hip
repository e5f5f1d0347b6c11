// The 4-bit form of a weight matrix: quantisation with group scales (and zero
// points), and its expansion.
#include "ffn.hpp"

namespace sgemm {

static inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The stored number of w: quotient, rounding and offset in 64 bits. The
// operands have at most 24 significant bits and the quotient is compared with
// halves of small whole numbers, so the 64-bit quotient never rounds across a
// half that the exact one does not reach.
__device__ __forceinline__ uint32_t quantise(float w, double s, double z) {
    double q = (s != 0.0 ? rint((double)w / s) : 0.0) + z;
    q = q < 0.0 ? 0.0 : q > 15.0 ? 15.0 : q;
    return q == q ? (uint32_t)(int)q : (uint32_t)(int)z;
}

// One wave per group of one row.
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
        bad += x - x;   // 0, or NaN for an infinity or NaN
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        lo = fminf(lo, __shfl_xor(lo, off));
        hi = fmaxf(hi, __shfl_xor(hi, off));
        bad += __shfl_xor(bad, off);
    }
    const bool asym = a.Z != nullptr;
    const double exact = asym ? ((double)hi - (double)lo) / 15.0 : (double)fmaxf(hi, -lo) / 7.0;
    const T st = bad == 0.0f ? (T)(float)exact : (T)__builtin_nanf("");
    const double s = (double)(float)st;
    double z = 8.0;
    if (asym) {
        z = s > 0.0 ? rint(-(double)lo / s) : 0.0;
        z = z > 15.0 ? 15.0 : z;
    }
    if (lane == 0) {
        ((T*)a.S)[row * a.lds + g] = st;
        if (asym) ((T*)a.Z)[row * a.ldz + g] = (T)(float)z;
    }
    uint8_t* q = a.Q + row * a.ldq;
    for (int k = k0 + 2 * lane; k < k1; k += 128) {
        const uint32_t q0 = quantise((float)w[k], s, z);
        const uint32_t q1 = k + 1 < a.K ? quantise((float)w[k + 1], s, z) : 0u;
        q[k >> 1] = (uint8_t)(q0 | (q1 << 4));
    }
}

// Two weights (one byte) per thread.
template <class T>
__global__ __launch_bounds__(256) void k_w4_dequantize(PackArgs a) {
    const int bytes = (a.K + 1) / 2;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = at / bytes;
    const int b = (int)(at - row * bytes);
    if (row >= a.F) return;
    const uint32_t q = a.Q[row * a.ldq + b];
    const int g = 2 * b / a.group;
    const float s = (float)((const T*)a.S)[row * a.lds + g];
    const float z = a.Z != nullptr ? (float)((const T*)a.Z)[row * a.ldz + g] : 8.0f;
    T* w = const_cast<T*>((const T*)a.W) + row * a.ldw;
    w[2 * b] = (T)(((float)(q & 15) - z) * s);
    if (2 * b + 1 < a.K) w[2 * b + 1] = (T)(((float)(q >> 4) - z) * s);
}

static int64_t quantize_wgs(const PackArgs& a) { return cdiv((int64_t)a.F * cdiv(a.K, a.group), 4); }
static int64_t dequantize_wgs(const PackArgs& a) { return cdiv((int64_t)a.F * cdiv(a.K, 2), 256); }

int check_w4_pack(const PackArgs& a) {
    return quantize_wgs(a) <= max_workgroups(256) && dequantize_wgs(a) <= max_workgroups(256)
               ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

hipError_t launch_w4_quantize(int dtype, const PackArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        hipLaunchKernelGGL((k_w4_quantize<T>), dim3((unsigned)quantize_wgs(a)), dim3(256), 0, s, a);
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

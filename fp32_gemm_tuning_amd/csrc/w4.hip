// Products with 4-bit weights: Y = X W^T (w4) and the gated block over two
// such weights (w4_glu).
//
// With q the stored numbers of a group, sum (q - z) s x = s (sum q x - z sum x):
// the scale and zero point are applied once per group and lane.
#include "ffn.hpp"

namespace sgemm {

typedef uint32_t u32_u1 __attribute__((aligned(1)));

// Eight weights of a row from column k (a multiple of 8), as one word: bytes past the row's end
// (bytes in all) read as zero.
__device__ __forceinline__ uint32_t load_w8(const uint8_t* row, int k, int bytes) {
    const int at = k >> 1;
    if (at + 4 <= bytes) return *(const u32_u1*)(row + at);
    uint32_t v = 0;
    for (int i = 0; at + i < bytes; ++i) v |= (uint32_t)row[at + i] << (8 * i);
    return v;
}

// One wave per output feature and up to MB rows of X; lanes take 8
// consecutive k in turn.
template <class T, bool DUAL, int MB>
__global__ __launch_bounds__(256) void k_w4(W4Args a) {
    const int lane = threadIdx.x & 63;
    const int64_t f = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int m0 = blockIdx.y * MB;
    if (f >= a.F) return;
    const int bytes = (a.K + 1) / 2;
    float acc[DUAL ? 2 : 1][MB] = {};
    for (int k = lane * 8; k < a.K; k += 512) {
        const int g = k / a.group;
        float x[MB][8], sx[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            sx[m] = 0.0f;
            const T* p = (const T*)a.X + (int64_t)(m0 + m) * a.ldx + k;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[m][e] = m0 + m < a.M && k + e < a.K ? (float)p[e] : 0.0f;
                sx[m] += x[m][e];
            }
        }
#pragma unroll
        for (int d = 0; d < (DUAL ? 2 : 1); ++d) {
            const uint32_t w = load_w8(a.Q[d] + f * a.ldq, k, bytes);
            const float s = (float)((const T*)a.S[d])[f * a.lds + g];
            const float z = a.Z[d] != nullptr ? (float)((const T*)a.Z[d])[f * a.ldz + g] : 8.0f;
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                float v = -z * sx[m];
#pragma unroll
                for (int e = 0; e < 8; ++e) v = __builtin_fmaf((float)((w >> (4 * e)) & 15), x[m][e], v);
                acc[d][m] = __builtin_fmaf(s, v, acc[d][m]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int d = 0; d < (DUAL ? 2 : 1); ++d) {
            v[d] = acc[d][m];
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) v[d] += __shfl_xor(v[d], off);
        }
        if (lane == 0 && m0 + m < a.M)
            ((T*)a.Y)[(int64_t)(m0 + m) * a.ldy + f] = (T)(DUAL ? act_value(a.act, v[0]) * v[1] : v[0]);
    }
}

constexpr int W4_MB = 4;

int check_w4(const W4Args& a, bool) {
    return (a.M + W4_MB - 1) / W4_MB <= 65535 ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

hipError_t launch_w4(int dtype, const W4Args& a, bool dual, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        const dim3 grid((unsigned)((a.F + 3) / 4), (unsigned)((a.M + W4_MB - 1) / W4_MB));
        if (dual)
            hipLaunchKernelGGL((k_w4<T, true, W4_MB>), grid, dim3(256), 0, s, a);
        else
            hipLaunchKernelGGL((k_w4<T, false, W4_MB>), grid, dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace sgemm

// The backward pass of the root-mean-square norm: dX row by row, dW as partial sums
// over blocks of rows that are then added in their order.
#include "norm_core.hpp"

namespace sgemm {

// dX of rows of any length: a workgroup a row, read twice.
constexpr int LONG_NT = 1024;
template <class T>
__global__ __launch_bounds__(LONG_NT) void k_norm_dx_long(NormBwdArgs a) {
    constexpr int N = Chunk<T>::N, STEP = LONG_NT * N;
    __shared__ float red[LONG_NT / 64];
    const int first = threadIdx.x * N;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const T* dy = (const T*)a.dY + m * a.lddy;
        const T* h = (const T*)a.H + m * a.ldh;
        const float rstd = a.rstd[m];
        float along = 0.0f;
        for (int at = first; at < a.K; at += STEP) {
            Chunk<T> d, w, n;
            d.load(dy, at, a.K);
            w.load((const T*)a.W, at, a.K);
            n.load(h, at, a.K);
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (at + e < a.K) along = __builtin_fmaf(d.v[e] * w.v[e], n.v[e] * rstd, along);
        }
        along = over_row<LONG_NT>(along, Plus{}, red) / (float)a.K;
        for (int at = first; at < a.K; at += STEP) {
            Chunk<T> d, w, n, o;
            d.load(dy, at, a.K);
            w.load((const T*)a.W, at, a.K);
            n.load(h, at, a.K);
            if (a.dH != nullptr) o.load((const T*)a.dH + m * a.lddh, at, a.K);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float g = rstd * __builtin_fmaf(-(n.v[e] * rstd), along, d.v[e] * w.v[e]);
                o.v[e] = a.dH != nullptr ? o.v[e] + g : g;
            }
            o.store((T*)a.dX + m * a.lddx, at, a.K);
        }
    }
}

// Partial sums of dW: a thread one chunk of columns of the rows of part blockIdx.y.
template <class T>
__global__ __launch_bounds__(256) void k_norm_dw_part(NormBwdArgs a, int rows) {
    constexpr int N = Chunk<T>::N;
    const int at = (blockIdx.x * 256 + threadIdx.x) * N;
    if (at >= a.K) return;
    const int64_t m0 = (int64_t)blockIdx.y * rows, m1 = m0 + rows < a.M ? m0 + rows : a.M;
    float s[N] = {};
    for (int64_t m = m0; m < m1; ++m) {
        Chunk<T> d, n;
        d.load((const T*)a.dY + m * a.lddy, at, a.K);
        n.load((const T*)a.H + m * a.ldh, at, a.K);
        const float rstd = a.rstd[m];
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = __builtin_fmaf(d.v[e], n.v[e] * rstd, s[e]);
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (at + e < a.K) a.part[(int64_t)blockIdx.y * a.K + at + e] = s[e];
}

// The parts' sums, in their order.
template <class T>
__global__ __launch_bounds__(256) void k_norm_dw_sum(NormBwdArgs a, int parts) {
    const int k = blockIdx.x * 256 + threadIdx.x;
    if (k >= a.K) return;
    float s = 0.0f;
    for (int p = 0; p < parts; ++p) s += a.part[(int64_t)p * a.K + k];
    ((T*)a.dW)[k] = (T)s;
}

// Rows of a part, and parts.
static int part_rows(int64_t M) {
    const int64_t r = (M + 255) / 256;
    return (int)(r < 16 ? 16 : r);
}
static int parts(int64_t M) { return (int)((M + part_rows(M) - 1) / part_rows(M)); }

size_t norm_part_bytes(int, int64_t M, int64_t K) { return (size_t)parts(M) * (size_t)K * sizeof(float); }
int check_norm_bwd(const NormBwdArgs&) { return 0; }

hipError_t launch_norm_bwd(int dtype, const NormBwdArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        constexpr int N = Chunk<T>::N;
        if (a.dW != nullptr) {   // first: dX may be written over dY
            const int n = a.M > 0 ? parts(a.M) : 0;
            if (n > 0)
                hipLaunchKernelGGL((k_norm_dw_part<T>), dim3((unsigned)((a.K + 256 * N - 1) / (256 * N)), (unsigned)n),
                                   dim3(256), 0, s, a, part_rows(a.M));
            hipLaunchKernelGGL((k_norm_dw_sum<T>), dim3((unsigned)((a.K + 255) / 256)), dim3(256), 0, s, a, n);
        }
        if (a.dX != nullptr)
            hipLaunchKernelGGL((k_norm_dx_long<T>), dim3((unsigned)(a.M < (1 << 20) ? a.M : 1 << 20)), dim3(LONG_NT),
                               0, s, a);
        return hipGetLastError();
    });
}

}  // namespace sgemm

// The elementwise step of the gated block's backward pass:
// dU = dH * act(G), dG = dH * U * act'(G), in FP32, rounded once to the type
// that the products after it read.
#include "ffn.hpp"

namespace sgemm {

// Four consecutive columns of a row, as loaded (loads need only element
// alignment); zero from column F on.
template <class T>
struct Four {
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef T4 T4u __attribute__((aligned(sizeof(T))));
    typedef f32x4 F4u __attribute__((aligned(4)));
    f32x4 g = {}, u = {};
    T4 dh = {};

    __device__ __forceinline__ void load(const GluGradArgs& a, int64_t row, int col) {
        const float* p = a.P + row * a.ldp + col;
        const T* h = (const T*)a.dH + row * a.lddh + col;
        if (col + 4 <= a.F) {
            g = *(const F4u*)p;
            u = *(const F4u*)(p + a.F);
            dh = *(const T4u*)h;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (col + e < a.F) {
                    g[e] = p[e];
                    u[e] = p[a.F + e];
                    dh[e] = h[e];
                }
        }
    }
    __device__ __forceinline__ float grad_u(int act, int e) const {
        return (float)dh[e] * act_value<sizeof(T) == 4>(act, g[e]);
    }
    __device__ __forceinline__ float grad_g(int act, int e) const {
        return (float)dh[e] * u[e] * act_slope<sizeof(T) == 4>(act, g[e]);
    }
};

__device__ __forceinline__ bool finite(float v) { return fabsf(v) <= 3.4028234663852886e38f; }
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
    return v;
}

// Half spans 2^-24 to 65504, FP32 sums and the gradients built from them far more:
// dG and dU kept as they are overflow where dX is an ordinary number (dH = 8000,
// U = 10), and lose their bits where they are small beside the weights' gradients
// (dH = 5e-5, U = 0.01: dWg off by 5% in the norm, 0.35% by its rounding alone). So
// both are kept times one power of two, 2^shift, that brings the largest finite
// magnitude of the two to the top of the type's range. The products multiply
// their FP32 sums back, exactly. What is kept is then off by half a step, or
// by 2^-40 of that magnitude where this is more. An infinity or NaN stays what it
// is and does not move the scale.
//
// Its price is this pass over P and dH before the one that writes, bound by their
// bytes: 4096 x 8192 79 us (336 MB, 4.2 TB/s) of a training step of 1576 (K = 4096;
// 1500 without), 77 x 1000 4.9 us. bfloat16 has FP32's range and needs none.
constexpr int PEAK_NT = 1024;
template <class T>
__global__ __launch_bounds__(PEAK_NT) void k_glu_peak(GluGradArgs a) {
    __shared__ float red[PEAK_NT / 64];
    const int64_t per_row = a.ldd / 4, n = a.M * per_row;
    float top = 0.0f;
    for (int64_t i = (int64_t)blockIdx.x * PEAK_NT + threadIdx.x; i < n; i += (int64_t)gridDim.x * PEAK_NT) {
        const int64_t row = i / per_row;
        Four<T> x;
        x.load(a, row, (int)(i - row * per_row) * 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float u = fabsf(x.grad_u(a.act, e)), g = fabsf(x.grad_g(a.act, e));
            top = fmaxf(top, fmaxf(finite(u) ? u : 0.0f, finite(g) ? g : 0.0f));
        }
    }
    top = wave_max(top);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < PEAK_NT / 64; ++w) top = fmaxf(top, red[w]);
        a.peaks[blockIdx.x] = top;
    }
}

// The power of two from all workgroups' magnitudes (at most 256, one a thread of
// a workgroup of 256).
__device__ __forceinline__ int shift_of(const float* peaks, int n) {
    __shared__ float red[4];
    const float mine = wave_max((int)threadIdx.x < n ? peaks[threadIdx.x] : 0.0f);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mine;
    __syncthreads();
    const float top = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    if (top == 0.0f) return 0;
    const int k = 16 - __builtin_amdgcn_frexp_expf(top);   // top * 2^k in [2^15, 2^16)
    return __builtin_amdgcn_ldexpf(top, k) > 65504.0f ? k - 1 : k;
}

// Four consecutive columns a thread (ldd is a multiple of 64, so four
// never straddle a row of the results).
// Bound by its bytes, P and dH read, dG and dU written: 4096 x 8192 bf16
// 470 MB in 92 us, 5.1 TB/s, the rate of a large copy.
template <class T>
__global__ __launch_bounds__(256) void k_glu_grad(GluGradArgs a, int npeaks) {
    using T4 = typename Four<T>::T4;
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    const int64_t row = at / a.ldd;
    const int col = (int)(at - row * a.ldd);
    Four<T> x;
    if (row < a.M) x.load(a, row, col);
    int shift = 0;
    if constexpr (std::is_same_v<T, f16>) {
        shift = shift_of(a.peaks, npeaks);
        if (at == 0) *a.shift = shift;
    }
    if (row >= a.M) return;
    T4 dg = {}, du = {}, dgl = {}, dul = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (col + e >= a.F) break;
        float vu = x.grad_u(a.act, e), vg = x.grad_g(a.act, e);
        if constexpr (std::is_same_v<T, f16>) {
            vu = __builtin_amdgcn_ldexpf(vu, shift);
            vg = __builtin_amdgcn_ldexpf(vg, shift);
        }
        du[e] = (T)vu;
        dg[e] = (T)vg;
        const float ru = vu - (float)du[e], rg = vg - (float)dg[e];
        dul[e] = (T)(fabsf(ru) <= 3.0e38f ? ru : 0.0f);   // (nothing is left of an infinity or NaN)
        dgl[e] = (T)(fabsf(rg) <= 3.0e38f ? rg : 0.0f);
    }
    *(T4*)((T*)a.dG + at) = dg;
    *(T4*)((T*)a.dU + at) = du;
    if (a.dGl != nullptr) {
        *(T4*)((T*)a.dGl + at) = dgl;
        *(T4*)((T*)a.dUl + at) = dul;
    }
}

static int64_t workgroups(const GluGradArgs& a) { return ((int64_t)a.M * a.ldd / 4 + 255) / 256; }

int check_glu_grad(const GluGradArgs& a) {
    return workgroups(a) <= max_workgroups(256) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

// Workgroups of k_glu_peak: one a compute unit of MI355X at the most, so that one
// of k_glu_grad reads a magnitude a thread.
int32_t glu_peaks(int64_t M, int64_t ldd) {
    const int64_t n = (M * (ldd / 4) + PEAK_NT - 1) / PEAK_NT;
    return (int32_t)(n < 256 ? n : 256);
}

hipError_t launch_glu_grad(int dtype, const GluGradArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        int npeaks = 0;
        if constexpr (std::is_same_v<T, f16>) {
            npeaks = glu_peaks(a.M, a.ldd);
            hipLaunchKernelGGL((k_glu_peak<T>), dim3((unsigned)npeaks), dim3(PEAK_NT), 0, s, a);
            const hipError_t e = hipGetLastError();
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((k_glu_grad<T>), dim3((unsigned)workgroups(a)), dim3(256), 0, s, a, npeaks);
        return hipGetLastError();
    });
}

}  // namespace sgemm

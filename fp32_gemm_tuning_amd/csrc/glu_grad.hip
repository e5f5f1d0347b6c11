// The elementwise step of the gated block's backward pass:
// dU = dH * act(G), dG = dH * U * act'(G), in FP32, rounded once to the type
// that the products after it read.
#include "ffn.hpp"

namespace sgemm {

// Four consecutive columns a thread (ldd is a multiple of 64, so four
// never straddle a row of the results; loads need only element alignment).
// Bound by its bytes, P and dH read, dG and dU written: 4096 x 8192 bf16
// 470 MB in 92 us, 5.1 TB/s, the rate of a large copy.
template <class T>
__global__ __launch_bounds__(256) void k_glu_grad(GluGradArgs a) {
    typedef T T4 __attribute__((ext_vector_type(4)));
    typedef T4 T4u __attribute__((aligned(sizeof(T))));
    typedef f32x4 F4u __attribute__((aligned(4)));
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    const int64_t row = at / a.ldd;
    const int col = (int)(at - row * a.ldd);
    if (row >= a.M) return;
    T4 dg = {}, du = {}, dgl = {}, dul = {};
    const float* p = a.P + row * a.ldp + col;
    const T* h = (const T*)a.dH + row * a.lddh + col;
    f32x4 g = {}, u = {};
    T4 dh = {};
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
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (col + e >= a.F) break;
        const float d = (float)dh[e];
        const float vu = d * act_value<sizeof(T) == 4>(a.act, g[e]);
        const float vg = d * u[e] * act_slope<sizeof(T) == 4>(a.act, g[e]);
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

hipError_t launch_glu_grad(int dtype, const GluGradArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        hipLaunchKernelGGL((k_glu_grad<T>), dim3((unsigned)workgroups(a)), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace sgemm

// The elementwise step of the gated block's backward pass:
// dU = dH * act(G), dG = dH * U * act'(G), in FP32, rounded once to the type
// that the products after it read.
#include "ffn.hpp"

namespace sgemm {

// One thread per element of the M x ldd results; columns from F on are zero.
template <class T>
__global__ __launch_bounds__(256) void k_glu_grad(GluGradArgs a) {
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = at / a.ldd;
    const int col = (int)(at - row * a.ldd);
    if (row >= a.M) return;
    float dg = 0.0f, du = 0.0f;
    if (col < a.F) {
        const float g = a.P[row * a.ldp + col], u = a.P[row * a.ldp + a.F + col];
        const float dh = (float)((const T*)a.dH)[row * a.lddh + col];
        du = dh * act_value(a.act, g);
        dg = dh * u * act_slope(a.act, g);
    }
    ((T*)a.dG)[at] = (T)dg;
    ((T*)a.dU)[at] = (T)du;
}

static int64_t workgroups(const GluGradArgs& a) { return ((int64_t)a.M * a.ldd + 255) / 256; }

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

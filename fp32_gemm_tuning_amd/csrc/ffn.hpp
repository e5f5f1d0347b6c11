// Shared pieces of the gated feed-forward and 4-bit kernels
// (include/sgemm_f32_ffn.h): the element types, the gate's activations, the
// argument blocks and the launchers that ffn_api.hip calls.
#pragma once

#include "kernels.hpp"

#include <type_traits>

#include "sgemm_f32_ffn.h"

namespace sgemm {

typedef __bf16 bf16;
typedef _Float16 f16;

// f(type tag) with the call's element type; the tag's ::type is float, bf16
// or f16.
template <class T>
struct TypeTag {
    using type = T;
};
template <class Fn>
static inline hipError_t with_dtype(int dtype, Fn&& f) {
    if (dtype == SGEMM_F32_DTYPE_F32) return f(TypeTag<float>{});
    if (dtype == SGEMM_F32_DTYPE_BF16) return f(TypeTag<bf16>{});
    return f(TypeTag<f16>{});
}
static inline int64_t dtype_bytes(int dtype) { return dtype == SGEMM_F32_DTYPE_F32 ? 4 : 2; }

// Activations and their slopes, in FP32. Both sigmoid forms (silu, and gelu_tanh
// as (1 + tanh v) / 2 = 1 / (1 + exp(-2v))) go through exp(-|x|) <= 1, which
// neither overflows nor loses the small side; a slope's second term, whose
// factor has underflowed to 0, is dropped rather than multiplied by a large g.
// 16-bit results take the exponential and the reciprocal of the hardware: with
// the library's, the epilogue of a 256 x 256 tile took a tenth of the product's
// time. The hardware's exponential gives 0 below 2^-126, where g exp(g) is still an
// ordinary bfloat16 number (silu(-90) = -7.4e-38), so exp(-|x|) is the square of
// exp(-|x| / 2). Its relative error is that of the rounded argument and of its
// factor 1 / (2 ln 2), doubled by the square, |x| 2^-23 and less (2^-20 at 8, 2^-16.5 at
// 87), and a few 2^-23: under half a step of the types. FP32 results take the
// library's exponential and one Newton step on the reciprocal.
template <bool F32>
__device__ __forceinline__ float sigmoid(float x) {
    const float m = -fabsf(x);
    float p, r;
    if constexpr (F32) {
        p = expf(m);
        const float d = 1.0f + p;
        r = __builtin_amdgcn_rcpf(d);
        r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
    } else {
        const float q = __builtin_amdgcn_exp2f(0.72134752044448170f * m);
        p = q * q;
        r = __builtin_amdgcn_rcpf(1.0f + p);
    }
    return x < 0.0f ? p * r : r;   // NaN: p and r are NaN
}
template <bool F32 = true>
__device__ __forceinline__ float act_value(int act, float g) {
    switch (act) {
        case SGEMM_F32_ACT_SILU: return g * sigmoid<F32>(g);
        case SGEMM_F32_ACT_GELU: return 0.5f * g * erfcf(-0.70710678118654752f * g);
        case SGEMM_F32_ACT_GELU_TANH:
            return g * sigmoid<F32>(1.59576912160573071f * (g + 0.044715f * g * g * g));
        default: return g < 0.0f ? 0.0f : g;       // NaN stays NaN
    }
}
template <bool F32 = true>
__device__ __forceinline__ float act_slope(int act, float g) {
    switch (act) {
        case SGEMM_F32_ACT_SILU: {
            const float s = sigmoid<F32>(g), t = s * (1.0f - s);
            return t == 0.0f ? s : s + g * t;
        }
        case SGEMM_F32_ACT_GELU: {
            const float cdf = 0.5f * erfcf(-0.70710678118654752f * g);
            const float pdf = 0.39894228040143268f * expf(-0.5f * g * g);
            return pdf == 0.0f ? cdf : cdf + g * pdf;
        }
        case SGEMM_F32_ACT_GELU_TANH: {
            const float s = sigmoid<F32>(1.59576912160573071f * (g + 0.044715f * g * g * g)), t = s * (1.0f - s);
            return t == 0.0f ? s : s + g * t * 1.59576912160573071f * (1.0f + 0.134145f * g * g);
        }
        default: return g > 0.0f ? 1.0f : (g != g ? g : 0.0f);
    }
}

// One forward call of the gated block: H = act(X Wg^T) * (X Wu^T), and the
// pre-activations in P where it is not null.
struct GluArgs {
    const void* X;
    const void* Wg;
    const void* Wu;
    void* H;
    float* P;
    int64_t ldx, ldwg, ldwu, ldh, ldp;
    int32_t M, F, K;
    int32_t act;
};

// The elementwise step of the backward pass: dG and dU (M x F in the type,
// leading dimension ldd, columns F .. ldd-1 written as zero) from P and dH.
struct GluGradArgs {
    const float* P;
    const void* dH;
    void* dG;
    void* dU;
    // What the rounding of dG and dU left, rounded itself (glu_two_parts), or
    // null.
    void* dGl;
    void* dUl;
    int64_t ldp, lddh, ldd;
    int32_t M, F;
    int32_t act;
    // Half: the largest finite magnitude that each workgroup of k_glu_peak found
    // (glu_peaks of them), and the power of two that dG and dU are kept times.
    float* peaks;
    int32_t* shift;
};

// A product of the backward pass. dX: C0 = dG W[0] + dU W[1]; dW:
// C0 = dG^T X, C1 = dU^T X (either may be null). D are dG and dU (M x F,
// leading dimension ldd); part is the space of split products' partial sums
// (glu_prod_bytes).
struct GluProdArgs {
    const void* D[2];
    const void* L[2];   // their second parts, summed after them, or null
    const void* W[2];
    const void* X;
    void* C[2];
    float* part;
    int64_t ldd, ldw[2], ldx, ldc[2];
    int32_t M, F, K;
    const int32_t* shift;   // half: D and L are kept times 2^*shift, or null
};

// A call over 4-bit weights: one matrix (w4) or two (w4_glu).
struct W4Args {
    const void* X;
    const uint8_t* Q[2];
    const void* S[2];
    const void* Z[2];
    void* Y;
    int64_t ldx, ldq, lds, ldz, ldy;
    int32_t M, F, K;
    int32_t group;
    int32_t act;
};

struct PackArgs {
    const void* W;   // the matrix quantised; dequantisation writes it
    uint8_t* Q;
    void* S;
    void* Z;
    int64_t ldw, ldq, lds, ldz;
    int32_t F, K;
    int32_t group;
};

// glu_tile.hip
int check_glu(const GluArgs& a);
hipError_t launch_glu(int dtype, const GluArgs& a, hipStream_t s);
int check_glu_prod(const GluProdArgs& a);
// Whether a 16-bit backward pass keeps dG and dU in two parts: where few
// values carry the sums, the roundings of single ones show in the gradients
// instead of averaging out (one part: the error's norm is 1.41 times that of
// rounding the gradients alone, give or take 2% at 16384 values, and 1.5 times and
// more for a few hundred; two parts: 1.00 times). The doubled sums are small
// there. Beyond, the gradients keep the 1.41: two parts would make it 1.00 at every
// size, for 1431 -> 2262 us of a 4096 x 8192 x 4096 bf16 step, 119 -> 204 of a backward
// pass of 512 x 4096 x 4096 and 20 -> 25 of 77 x 1000 x 511.
static inline bool glu_two_parts(int dtype, int64_t M, int64_t F) {
    return dtype != SGEMM_F32_DTYPE_F32 && M * F <= 16384;
}
// Whether the backward products of these sizes run on launch_glu_dx and
// launch_glu_dw (16-bit ones do) or, FP32, on sgemm_f32_ws.
bool glu_dx_here(int dtype, int64_t M, int64_t K);
bool glu_dw_here(int dtype, int64_t F, int64_t K, int64_t ldd, int64_t ldx);
size_t glu_prod_bytes(int dtype, int64_t M, int64_t F, int64_t K);
hipError_t launch_glu_dx(int dtype, const GluProdArgs& a, hipStream_t s);
hipError_t launch_glu_dw(int dtype, const GluProdArgs& a, hipStream_t s);
// glu_grad.hip
int32_t glu_peaks(int64_t M, int64_t ldd);
int check_glu_grad(const GluGradArgs& a);
hipError_t launch_glu_grad(int dtype, const GluGradArgs& a, hipStream_t s);
// w4.hip
int check_w4(const W4Args& a, bool dual);
hipError_t launch_w4(int dtype, const W4Args& a, bool dual, hipStream_t s);
// w4_pack.hip
int check_w4_pack(const PackArgs& a);
hipError_t launch_w4_quantize(int dtype, const PackArgs& a, hipStream_t s);
hipError_t launch_w4_dequantize(int dtype, const PackArgs& a, hipStream_t s);

}  // namespace sgemm

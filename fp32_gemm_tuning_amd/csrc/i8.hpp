// Shared pieces of the norm and 8-bit kernels (include/sgemm_f32_i8.h): the
// argument blocks and the launchers that i8_api.hip calls.
#pragma once

#include "ffn.hpp"

#include "sgemm_f32_i8.h"

namespace sgemm {

// A pass over rows: the norm of X + R (to Y, or to Q and S), or, without W,
// X itself to Q and S.
struct NormArgs {
    const void* X;
    const void* R;      // null: none
    const void* W;
    void* H;            // null: not wanted
    float* rstd;        // null: not wanted
    void* Y;
    int8_t* Q;
    float* S;
    int64_t ldx, ldr, ldh, ldy, ldq;
    int32_t M, K;
    float eps;
};

struct NormBwdArgs {
    const void* dY;
    const void* W;
    const void* H;
    const float* rstd;
    const void* dH;     // null: none
    void* dX;           // null: not wanted
    void* dW;           // null: not wanted
    float* part;        // partial sums of dW, rows of K (norm_part_bytes of them)
    int64_t lddy, ldh, lddh, lddx;
    int32_t M, K;
};

// A product of matrices in 8 bits: one weight (i8), or two (i8_glu).
struct I8Args {
    const int8_t* X;
    const float* Sx;
    const int8_t* W[2];
    const float* Sw[2];
    void* Y;
    int64_t ldx, ldw[2], ldy;
    int32_t M, F, K;
    int32_t dtype, act;
};

struct DequantArgs {
    const int8_t* Q;
    const float* S;
    void* X;
    int64_t ldq, ldx;
    int32_t M, K;
};

// norm.hip
hipError_t launch_norm(int dtype, const NormArgs& a, hipStream_t s);
hipError_t launch_norm_i8(int dtype, const NormArgs& a, hipStream_t s);
hipError_t launch_i8_quantize(int dtype, const NormArgs& a, hipStream_t s);
int check_i8_dequantize(const DequantArgs& a);
hipError_t launch_i8_dequantize(int dtype, const DequantArgs& a, hipStream_t s);
// norm_bwd.hip
size_t norm_part_bytes(int dtype, int64_t M, int64_t K);
hipError_t launch_norm_bwd(int dtype, const NormBwdArgs& a, hipStream_t s);
// i8.hip
int check_i8(const I8Args& a, bool dual);
const char* i8_kernel_name(const I8Args& a, bool dual);   // of the kernel that launch_i8 launches
hipError_t launch_i8(const I8Args& a, bool dual, hipStream_t s);

}  // namespace sgemm

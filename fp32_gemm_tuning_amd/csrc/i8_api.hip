// C-ABI entry points of include/sgemm_f32_i8.h: argument checks, quick
// returns and the launches; and the name of the kernel that a product takes
// (include/sgemm_f32_probe.h).
#include <hip/hip_runtime.h>

#include <cmath>

#include "i8.hpp"

#include "sgemm_f32_probe.h"

namespace sgemm {
namespace {

// No extent above this: the kernels step k in 32-bit arithmetic past the end.
constexpr int64_t kMaxExtent = 1 << 30;
// The longest sum of products of -128..127 that 32 bits hold: 131071 * 128 * 128 < 2^31.
constexpr int64_t kMaxSum = 131071;

bool bad_ptr(bool used, const void* p, int64_t bytes) {
    return used && (p == nullptr || (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0);
}
bool misaligned(const void* p, int64_t bytes) { return p != nullptr && bad_ptr(true, p, bytes); }
bool short_ld(int64_t ld, int64_t extent) { return ld < (extent > 1 ? extent : 1); }

int check_sizes(int dtype, int64_t M, int64_t F, int64_t K) {
    if (dtype < SGEMM_F32_DTYPE_F32 || dtype > SGEMM_F32_DTYPE_F16) return -17;
    if (M < 0) return -1;
    if (F < 0) return -2;
    if (K < 0) return -3;
    return 0;
}
bool too_large(int64_t M, int64_t F, int64_t K) { return M > kMaxExtent || F > kMaxExtent || K > kMaxExtent; }
int status(hipError_t e) { return e == hipSuccess ? 0 : (int)e; }

// What the two forms of the norm share: sizes and inputs, and, looked at after rms_norm_i8's own
// outputs, the sum's output.
int check_inputs(int dtype, int64_t M, int64_t K, float eps, const void* X, int64_t ldx, const void* R,
                 int64_t ldr, const void* W) {
    const int rc = check_sizes(dtype, M, 0, K);
    if (rc) return rc;
    if (!(eps >= 0.0f) || std::isinf(eps)) return -40;
    const int64_t e = dtype_bytes(dtype);
    const bool used = M > 0 && K > 0;
    if (bad_ptr(used, X, e)) return -5;
    if (short_ld(ldx, K)) return -6;
    if (used && misaligned(R, e)) return -38;
    if (R != nullptr && short_ld(ldr, K)) return -39;
    if (bad_ptr(used, W, e)) return -7;
    return 0;
}
int check_total(int dtype, int64_t M, int64_t K, const void* H, int64_t ldh) {
    if (M > 0 && K > 0 && misaligned(H, dtype_bytes(dtype))) return -41;
    if (H != nullptr && short_ld(ldh, K)) return -42;
    return 0;
}

// The checks of a product; `a` is filled where 0 is returned and there is something to launch.
int check_product(int dtype, bool dual, int act, int64_t M, int64_t F, int64_t K, const int8_t* X, int64_t ldx,
                  const float* Sx, const int8_t* W0, int64_t ldw0, const float* S0, const int8_t* W1, int64_t ldw1,
                  const float* S1, void* Y, int64_t ldy, I8Args& a) {
    a.Y = nullptr;
    int rc = check_sizes(dtype, 0, 0, 0);
    if (rc == 0 && dual && (act < SGEMM_F32_ACT_SILU || act > SGEMM_F32_ACT_RELU)) rc = -18;
    if (rc == 0) rc = check_sizes(dtype, M, F, K);
    if (rc) return rc;
    const bool out = M > 0 && F > 0, in = out && K > 0;
    if (bad_ptr(in, X, 1)) return -5;
    if (short_ld(ldx, K)) return -6;
    if (bad_ptr(in, Sx, 4)) return -44;
    if (bad_ptr(in, W0, 1)) return -7;
    if (short_ld(ldw0, K)) return -8;
    if (bad_ptr(in, S0, 4)) return -32;
    if (dual) {
        if (bad_ptr(in, W1, 1)) return -19;
        if (short_ld(ldw1, K)) return -20;
        if (bad_ptr(in, S1, 4)) return -36;
    }
    if (bad_ptr(out, Y, dtype_bytes(dtype))) return -10;
    if (short_ld(ldy, F)) return -11;
    if (!out) return 0;
    if (too_large(M, F, K) || K > kMaxSum) return SGEMM_F32_ERR_TOO_LARGE;
    a = I8Args{X, Sx, {W0, W1}, {S0, S1}, Y, ldx, {ldw0, ldw1}, ldy, (int32_t)M, (int32_t)F, (int32_t)K, dtype, act};
    return check_i8(a, dual);
}
int run_i8(int dtype, bool dual, int act, int64_t M, int64_t F, int64_t K, const int8_t* X, int64_t ldx,
           const float* Sx, const int8_t* W0, int64_t ldw0, const float* S0, const int8_t* W1, int64_t ldw1,
           const float* S1, void* Y, int64_t ldy, void* stream) {
    I8Args a;
    const int rc = check_product(dtype, dual, act, M, F, K, X, ldx, Sx, W0, ldw0, S0, W1, ldw1, S1, Y, ldy, a);
    if (rc || a.Y == nullptr) return rc;
    return status(launch_i8(a, dual, reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

SGEMM_F32_API int sgemm_f32_rms_norm(int dtype, int64_t M, int64_t K, float eps, const void* X,
                                     int64_t ldx, const void* R, int64_t ldr, const void* W, void* H,
                                     int64_t ldh, float* rstd, void* Y, int64_t ldy, void* stream) {
    int rc = check_inputs(dtype, M, K, eps, X, ldx, R, ldr, W);
    if (rc == 0) rc = check_total(dtype, M, K, H, ldh);
    if (rc) return rc;
    if (M > 0 && misaligned(rstd, 4)) return -43;
    if (bad_ptr(M > 0 && K > 0, Y, dtype_bytes(dtype))) return -10;
    if (short_ld(ldy, K)) return -11;
    if (M == 0 || (K == 0 && rstd == nullptr)) return 0;
    if (too_large(M, 0, K)) return SGEMM_F32_ERR_TOO_LARGE;
    const NormArgs a = {X, R, W, H, rstd, Y, nullptr, nullptr, ldx, ldr, ldh, ldy, 1, (int32_t)M, (int32_t)K, eps};
    return status(launch_norm(dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

SGEMM_F32_API int sgemm_f32_rms_norm_i8(int dtype, int64_t M, int64_t K, float eps, const void* X,
                                        int64_t ldx, const void* R, int64_t ldr, const void* W, void* H,
                                        int64_t ldh, int8_t* Q, int64_t ldq, float* S, void* stream) {
    int rc = check_inputs(dtype, M, K, eps, X, ldx, R, ldr, W);
    if (rc) return rc;
    if (bad_ptr(M > 0 && K > 0, Q, 1)) return -7;
    if (short_ld(ldq, K)) return -8;
    if (bad_ptr(M > 0, S, 4)) return -32;
    rc = check_total(dtype, M, K, H, ldh);
    if (rc) return rc;
    if (M == 0) return 0;
    if (too_large(M, 0, K)) return SGEMM_F32_ERR_TOO_LARGE;
    const NormArgs a = {X, R, W, H, nullptr, nullptr, Q, S, ldx, ldr, ldh, 1, ldq, (int32_t)M, (int32_t)K, eps};
    return status(launch_norm_i8(dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

SGEMM_F32_API int sgemm_f32_rms_norm_bwd_ws_size(int dtype, int64_t M, int64_t K, size_t* bytes) {
    const int rc = check_sizes(dtype, M, 0, K);
    if (rc) return rc;
    if (bytes == nullptr) return -12;
    *bytes = 0;
    if (too_large(M, 0, K)) return SGEMM_F32_ERR_TOO_LARGE;
    if (M > 0 && K > 0) *bytes = norm_part_bytes(dtype, M, K);
    return 0;
}

SGEMM_F32_API int sgemm_f32_rms_norm_bwd(int dtype, int64_t M, int64_t K, const void* dY, int64_t lddy,
                                         const void* W, const void* H, int64_t ldh, const float* rstd,
                                         const void* dH, int64_t lddh, void* dX, int64_t lddx, void* dW,
                                         void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_sizes(dtype, M, 0, K);
    if (rc) return rc;
    const int64_t e = dtype_bytes(dtype);
    const bool want_x = dX != nullptr && M > 0 && K > 0, want_w = dW != nullptr && K > 0;
    const bool used = want_x || (want_w && M > 0);
    if (bad_ptr(used, dY, e)) return -45;
    if (short_ld(lddy, K)) return -46;
    if (bad_ptr(want_x, W, e)) return -7;
    if (bad_ptr(used, H, e)) return -41;
    if (short_ld(ldh, K)) return -42;
    if (bad_ptr(used, rstd, 4)) return -43;
    if (want_x && misaligned(dH, e)) return -23;
    if (dH != nullptr && short_ld(lddh, K)) return -24;
    if (want_x && misaligned(dX, e)) return -25;
    if (dX != nullptr && short_ld(lddx, K)) return -26;
    if (want_w && misaligned(dW, e)) return -27;
    if (workspace_bytes > 0 && (workspace == nullptr || misaligned(workspace, 16))) return -16;
    if (!want_x && !want_w) return 0;
    if (too_large(M, 0, K)) return SGEMM_F32_ERR_TOO_LARGE;
    if (want_w && M > 0 && workspace_bytes < norm_part_bytes(dtype, M, K)) return SGEMM_F32_ERR_WORKSPACE;
    const NormBwdArgs a = {dY, W, H, rstd, dH, want_x ? dX : nullptr, want_w ? dW : nullptr, (float*)workspace,
                           lddy, ldh, lddh, lddx, (int32_t)M, (int32_t)K};
    return status(launch_norm_bwd(dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

SGEMM_F32_API int sgemm_f32_i8_quantize(int dtype, int64_t M, int64_t K, const void* X, int64_t ldx,
                                        int8_t* Q, int64_t ldq, float* S, void* stream) {
    int rc = check_sizes(dtype, M, 0, K);
    if (rc) return rc;
    if (bad_ptr(M > 0 && K > 0, X, dtype_bytes(dtype))) return -5;
    if (short_ld(ldx, K)) return -6;
    if (bad_ptr(M > 0 && K > 0, Q, 1)) return -7;
    if (short_ld(ldq, K)) return -8;
    if (bad_ptr(M > 0, S, 4)) return -32;
    if (M == 0) return 0;
    if (too_large(M, 0, K)) return SGEMM_F32_ERR_TOO_LARGE;
    const NormArgs a = {X, nullptr, nullptr, nullptr, nullptr, nullptr, Q, S, ldx, 1, 1, 1, ldq, (int32_t)M,
                        (int32_t)K, 0.0f};
    return status(launch_i8_quantize(dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

SGEMM_F32_API int sgemm_f32_i8_dequantize(int dtype, int64_t M, int64_t K, const int8_t* Q, int64_t ldq,
                                          const float* S, void* X, int64_t ldx, void* stream) {
    int rc = check_sizes(dtype, M, 0, K);
    if (rc) return rc;
    const bool out = M > 0 && K > 0;
    if (bad_ptr(out, Q, 1)) return -7;
    if (short_ld(ldq, K)) return -8;
    if (bad_ptr(out, S, 4)) return -32;
    if (bad_ptr(out, X, dtype_bytes(dtype))) return -10;
    if (short_ld(ldx, K)) return -11;
    if (!out) return 0;
    if (too_large(M, 0, K)) return SGEMM_F32_ERR_TOO_LARGE;
    const DequantArgs a = {Q, S, X, ldq, ldx, (int32_t)M, (int32_t)K};
    rc = check_i8_dequantize(a);
    if (rc) return rc;
    return status(launch_i8_dequantize(dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

SGEMM_F32_API int sgemm_f32_i8(int dtype, int64_t M, int64_t F, int64_t K, const int8_t* X, int64_t ldx,
                               const float* Sx, const int8_t* W, int64_t ldw, const float* Sw, void* Y,
                               int64_t ldy, void* stream) {
    return run_i8(dtype, false, 0, M, F, K, X, ldx, Sx, W, ldw, Sw, nullptr, 1, nullptr, Y, ldy, stream);
}

SGEMM_F32_API int sgemm_f32_i8_glu(int dtype, int act, int64_t M, int64_t F, int64_t K, const int8_t* X,
                                   int64_t ldx, const float* Sx, const int8_t* Wg, int64_t ldwg,
                                   const float* Sg, const int8_t* Wu, int64_t ldwu, const float* Su,
                                   void* H, int64_t ldh, void* stream) {
    return run_i8(dtype, true, act, M, F, K, X, ldx, Sx, Wg, ldwg, Sg, Wu, ldwu, Su, H, ldh, stream);
}

SGEMM_F32_API const char* sgemm_f32_i8_kernel(int gated, int64_t M, int64_t F, int64_t K, const int8_t* X,
                                              int64_t ldx, const int8_t* Wg, int64_t ldwg, const int8_t* Wu,
                                              int64_t ldwu) {
    // (the choice does not look at the type, the scales or the output: any that pass the checks)
    alignas(16) static float any[1];
    I8Args a;
    const int rc = check_product(SGEMM_F32_DTYPE_F32, gated != 0, SGEMM_F32_ACT_SILU, M, F, K, X, ldx, any, Wg, ldwg, any,
                                 gated ? Wu : nullptr, gated ? ldwu : 1, any, any, F > 1 ? F : 1, a);
    return rc || a.Y == nullptr ? nullptr : i8_kernel_name(a, gated != 0);
}

}  // extern "C"

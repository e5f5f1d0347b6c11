// C-ABI entry points of include/sgemm_f32_ffn.h: argument checks, quick
// returns, the workspace's layout and the launches.
#include <hip/hip_runtime.h>

#include "ffn.hpp"

namespace sgemm {
namespace {

// No extent above this: the kernels step k in 32-bit arithmetic past the end.
constexpr int64_t kMaxExtent = 1 << 30;

bool misaligned(const void* p, int64_t bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) != 0;
}
bool bad_ptr(bool used, const void* p, int64_t bytes) {
    return used && (p == nullptr || misaligned(p, bytes));
}
bool short_ld(int64_t ld, int64_t extent) { return ld < (extent > 1 ? extent : 1); }
int64_t cdiv(int64_t a, int64_t b) { return a / b + (a % b != 0); }
size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

int check_sizes(int dtype, int64_t M, int64_t F, int64_t K) {
    if (dtype < SGEMM_F32_DTYPE_F32 || dtype > SGEMM_F32_DTYPE_F16) return -17;
    if (M < 0) return -1;
    if (F < 0) return -2;
    if (K < 0) return -3;
    return 0;
}
int check_act(int act) { return act < SGEMM_F32_ACT_SILU || act > SGEMM_F32_ACT_RELU ? -18 : 0; }
bool too_large(int64_t M, int64_t F, int64_t K) {
    return M > kMaxExtent || F > kMaxExtent || K > kMaxExtent;
}

// A group of at least K is one group a row; the kernels then see K rounded up
// to whole blocks of 32.
bool bad_group(int64_t group, int64_t K) { return group < 1 || (group % 32 != 0 && group < K); }
int32_t group_of(int64_t group, int64_t K) {
    return (int32_t)(group >= K ? cdiv(K > 0 ? K : 1, 32) * 32 : group);
}

// The backward pass's workspace: dG and dU, each M rows of ldd elements (F
// rounded up to whole 64-element slices, so that their rows are whole 16-byte
// chunks), where they are kept in two parts their second ones, then the partial sums of products that are split, or, for large
// FP32 products, what the stream-K kernels may use, and for half the power of two
// that dG and dU are kept times, with the magnitudes it comes from.
struct BwdSpace {
    int64_t ldd;
    size_t one, sk_at, sk_bytes, shift_at, total;   // dG at 0, the others `one` apart
};
int bwd_space(int dtype, int64_t M, int64_t F, int64_t K, int num_cus, BwdSpace* o) {
    o->ldd = cdiv(F > 0 ? F : 1, 64) * 64;
    const size_t one = up256((size_t)M * (size_t)o->ldd * (size_t)dtype_bytes(dtype));
    o->one = one;
    o->sk_at = (glu_two_parts(dtype, M, F) ? 4 : 2) * one;
    size_t most = glu_prod_bytes(dtype, M, F, K);
    if (dtype == SGEMM_F32_DTYPE_F32) {
        size_t dx = 0, dw = 0;
        int rc = sgemm_f32_ws_size(-1, SGEMM_F32_ROW_MAJOR, SGEMM_F32_NO_TRANS, SGEMM_F32_NO_TRANS, M, K,
                                   F, num_cus, &dx);
        if (rc == 0)
            rc = sgemm_f32_ws_size(-1, SGEMM_F32_ROW_MAJOR, SGEMM_F32_TRANS, SGEMM_F32_NO_TRANS, F, K, M,
                                   num_cus, &dw);
        if (rc) return rc;
        most = dx > most ? dx : most;
        most = dw > most ? dw : most;
    }
    o->sk_bytes = up256(most);
    o->shift_at = o->sk_at + o->sk_bytes;
    o->total = o->shift_at;
    if (dtype == SGEMM_F32_DTYPE_F16 && M > 0 && F > 0)
        o->total += up256(16 + sizeof(float) * (size_t)glu_peaks(M, o->ldd));
    return 0;
}

int current_cus(int* cus) {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return SGEMM_F32_ERR_DEVICE;
    if (hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || *cus <= 0)
        return SGEMM_F32_ERR_DEVICE;
    return 0;
}

int status(hipError_t e) { return e == hipSuccess ? 0 : (int)e; }

int run_w4(int dtype, bool dual, int act, int64_t M, int64_t F, int64_t K, int64_t group, const void* X,
           int64_t ldx, const void* Q0, const void* Q1, int64_t ldq, const void* S0, const void* S1,
           int64_t lds, const void* Z0, const void* Z1, int64_t ldz, void* Y, int64_t ldy, void* stream) {
    int rc = check_sizes(dtype, 0, 0, 0);
    if (rc == 0 && dual) rc = check_act(act);
    if (rc == 0) rc = check_sizes(dtype, M, F, K);
    if (rc) return rc;
    if (bad_group(group, K)) return -31;
    const int64_t e = dtype_bytes(dtype), groups = K > 0 ? cdiv(K, group) : 0;
    const bool out = M > 0 && F > 0, in = out && K > 0;
    if (bad_ptr(in, X, e)) return -5;
    if (short_ld(ldx, K)) return -6;
    if (bad_ptr(in, Q0, 1)) return -7;
    if (dual && bad_ptr(in, Q1, 1)) return -19;
    if (short_ld(ldq, cdiv(K, 2))) return -8;
    if (bad_ptr(in, S0, e)) return -32;
    if (dual && bad_ptr(in, S1, e)) return -36;
    if (short_ld(lds, groups)) return -33;
    if (in && Z0 != nullptr && misaligned(Z0, e)) return -34;
    if (dual && in && ((Z0 == nullptr) != (Z1 == nullptr) || (Z1 != nullptr && misaligned(Z1, e)))) return -37;
    if (Z0 != nullptr && short_ld(ldz, groups)) return -35;
    if (bad_ptr(out, Y, e)) return -10;
    if (short_ld(ldy, F)) return -11;
    if (!out) return 0;
    if (too_large(M, F, K)) return SGEMM_F32_ERR_TOO_LARGE;
    const W4Args a = {X, {(const uint8_t*)Q0, (const uint8_t*)Q1}, {S0, S1}, {Z0, Z1}, Y, ldx, ldq, lds,
                      ldz, ldy, (int32_t)M, (int32_t)F, (int32_t)K, group_of(group, K), act};
    rc = check_w4(a, dual);
    if (rc) return rc;
    return status(launch_w4(dtype, a, dual, reinterpret_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace sgemm

using namespace sgemm;

extern "C" {

SGEMM_F32_API int sgemm_f32_glu(int dtype, int act, int64_t M, int64_t F, int64_t K, const void* X,
                                int64_t ldx, const void* Wg, int64_t ldwg, const void* Wu,
                                int64_t ldwu, void* H, int64_t ldh, float* P, int64_t ldp,
                                void* stream) {
    int rc = check_sizes(dtype, 0, 0, 0);
    if (rc == 0) rc = check_act(act);
    if (rc == 0) rc = check_sizes(dtype, M, F, K);
    if (rc) return rc;
    const int64_t e = dtype_bytes(dtype);
    const bool out = M > 0 && F > 0, in = out && K > 0;
    if (bad_ptr(in, X, e)) return -5;
    if (short_ld(ldx, K)) return -6;
    if (bad_ptr(in, Wg, e)) return -7;
    if (short_ld(ldwg, K)) return -8;
    if (bad_ptr(in, Wu, e)) return -19;
    if (short_ld(ldwu, K)) return -20;
    if (P != nullptr && out && misaligned(P, 4)) return -21;
    if (P != nullptr && short_ld(ldp, 2 * F)) return -22;
    if (bad_ptr(out, H, e)) return -10;
    if (short_ld(ldh, F)) return -11;
    if (!out) return 0;
    if (too_large(M, F, K)) return SGEMM_F32_ERR_TOO_LARGE;
    const GluArgs a = {X, Wg, Wu, H, P, ldx, ldwg, ldwu, ldh, ldp, (int32_t)M, (int32_t)F, (int32_t)K, act};
    rc = check_glu(a);
    if (rc) return rc;
    return status(launch_glu(dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

SGEMM_F32_API int sgemm_f32_glu_bwd_ws_size(int dtype, int64_t M, int64_t F, int64_t K, int num_cus,
                                            size_t* bytes) {
    const int rc = check_sizes(dtype, M, F, K);
    if (rc) return rc;
    if (bytes == nullptr) return -12;
    *bytes = 0;
    if (too_large(M, F, K)) return SGEMM_F32_ERR_TOO_LARGE;
    BwdSpace sp;
    const int r = bwd_space(dtype, M, F, K, num_cus, &sp);
    if (r == 0) *bytes = sp.total;
    return r;
}

SGEMM_F32_API int sgemm_f32_glu_bwd(int dtype, int act, int64_t M, int64_t F, int64_t K,
                                    const void* X, int64_t ldx, const void* Wg, int64_t ldwg,
                                    const void* Wu, int64_t ldwu, const float* P, int64_t ldp,
                                    const void* dH, int64_t lddh, void* dX, int64_t lddx,
                                    void* dWg, int64_t lddwg, void* dWu, int64_t lddwu,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    int rc = check_sizes(dtype, 0, 0, 0);
    if (rc == 0) rc = check_act(act);
    if (rc == 0) rc = check_sizes(dtype, M, F, K);
    if (rc) return rc;
    const int64_t e = dtype_bytes(dtype);
    const bool want_x = dX != nullptr && M > 0 && K > 0;
    const bool want_g = dWg != nullptr && F > 0 && K > 0, want_u = dWu != nullptr && F > 0 && K > 0;
    const bool grads = M > 0 && F > 0 && (want_x || want_g || want_u);
    if (bad_ptr(grads && (want_g || want_u), X, e)) return -5;
    if (short_ld(ldx, K)) return -6;
    if (bad_ptr(grads && want_x, Wg, e)) return -7;
    if (short_ld(ldwg, K)) return -8;
    if (bad_ptr(grads && want_x, Wu, e)) return -19;
    if (short_ld(ldwu, K)) return -20;
    if (bad_ptr(grads, P, 4)) return -21;
    if (short_ld(ldp, 2 * F)) return -22;
    if (bad_ptr(grads, dH, e)) return -23;
    if (short_ld(lddh, F)) return -24;
    if (want_x && misaligned(dX, e)) return -25;
    if (dX != nullptr && short_ld(lddx, K)) return -26;
    if (want_g && misaligned(dWg, e)) return -27;
    if (dWg != nullptr && short_ld(lddwg, K)) return -28;
    if (want_u && misaligned(dWu, e)) return -29;
    if (dWu != nullptr && short_ld(lddwu, K)) return -30;
    if (workspace_bytes > 0 && (workspace == nullptr || misaligned(workspace, 16))) return -16;
    if (!want_x && !want_g && !want_u) return 0;
    if (too_large(M, F, K)) return SGEMM_F32_ERR_TOO_LARGE;
    int cus = 0;
    if (dtype == SGEMM_F32_DTYPE_F32) {
        rc = current_cus(&cus);
        if (rc) return rc;
    }
    BwdSpace sp;
    rc = bwd_space(dtype, M, F, K, cus, &sp);
    if (rc) return rc;
    if (workspace_bytes < sp.total) return SGEMM_F32_ERR_WORKSPACE;
    char* const ws = (char*)workspace;
    const hipStream_t s = reinterpret_cast<hipStream_t>(stream);

    const bool two = glu_two_parts(dtype, M, F);
    char* const second[2] = {two ? ws + 2 * sp.one : nullptr, two ? ws + 3 * sp.one : nullptr};
    int32_t* const shift = grads && dtype == SGEMM_F32_DTYPE_F16 ? (int32_t*)(ws + sp.shift_at) : nullptr;
    GluProdArgs p = {{ws, ws + sp.one}, {second[0], second[1]}, {Wg, Wu}, X, {nullptr, nullptr}, (float*)(ws + sp.sk_at), sp.ldd, {ldwg, ldwu}, ldx,
                     {0, 0}, (int32_t)M, (int32_t)F, (int32_t)K, shift};
    const GluGradArgs g = {P, dH, ws, ws + sp.one, second[0], second[1], ldp, lddh, sp.ldd, (int32_t)M, (int32_t)F, act,
                           (float*)(ws + sp.shift_at + 16), shift};
    rc = check_glu_grad(g);
    if (rc == 0) rc = check_glu_prod(p);
    if (rc) return rc;
    if (grads) {
        rc = status(launch_glu_grad(dtype, g, s));
        if (rc) return rc;
    }
    const float* dg = (const float*)p.D[0];
    const float* du = (const float*)p.D[1];
    void* sk = ws + sp.sk_at;
    const int R = SGEMM_F32_ROW_MAJOR, N = SGEMM_F32_NO_TRANS, T = SGEMM_F32_TRANS;
    if (want_x) {
        if (glu_dx_here(dtype, M, K)) {
            p.C[0] = dX;
            p.ldc[0] = lddx;
            rc = status(launch_glu_dx(dtype, p, s));
        } else {
            rc = sgemm_f32_ws(R, N, N, M, K, F, 1.0f, dg, sp.ldd, (const float*)Wg, ldwg, 0.0f, (float*)dX,
                              lddx, sk, sp.sk_bytes, stream);
            if (rc == 0)
                rc = sgemm_f32_ws(R, N, N, M, K, F, 1.0f, du, sp.ldd, (const float*)Wu, ldwu, 1.0f,
                                  (float*)dX, lddx, sk, sp.sk_bytes, stream);
        }
        if (rc) return rc;
    }
    if ((want_g || want_u) && glu_dw_here(dtype, F, K, sp.ldd, ldx)) {
        p.C[0] = want_g ? dWg : nullptr;
        p.C[1] = want_u ? dWu : nullptr;
        p.ldc[0] = lddwg;
        p.ldc[1] = lddwu;
        return status(launch_glu_dw(dtype, p, s));
    }
    if (want_g)
        rc = sgemm_f32_ws(R, T, N, F, K, M, 1.0f, dg, sp.ldd, (const float*)X, ldx, 0.0f, (float*)dWg, lddwg,
                          sk, sp.sk_bytes, stream);
    if (rc == 0 && want_u)
        rc = sgemm_f32_ws(R, T, N, F, K, M, 1.0f, du, sp.ldd, (const float*)X, ldx, 0.0f, (float*)dWu, lddwu,
                          sk, sp.sk_bytes, stream);
    return rc;
}

SGEMM_F32_API int sgemm_f32_w4_quantize(int dtype, int64_t F, int64_t K, int64_t group,
                                        const void* W, int64_t ldw, void* Q, int64_t ldq, void* S,
                                        int64_t lds, void* Z, int64_t ldz, void* stream) {
    int rc = check_sizes(dtype, 0, F, K);
    if (rc) return rc;
    if (bad_group(group, K)) return -31;
    const int64_t e = dtype_bytes(dtype), groups = K > 0 ? cdiv(K, group) : 0;
    const bool out = F > 0 && K > 0;
    if (bad_ptr(out, W, e)) return -5;
    if (short_ld(ldw, K)) return -6;
    if (bad_ptr(out, Q, 1)) return -7;
    if (short_ld(ldq, cdiv(K, 2))) return -8;
    if (bad_ptr(out, S, e)) return -32;
    if (short_ld(lds, groups)) return -33;
    if (out && Z != nullptr && misaligned(Z, e)) return -34;
    if (Z != nullptr && short_ld(ldz, groups)) return -35;
    if (!out) return 0;
    if (too_large(0, F, K)) return SGEMM_F32_ERR_TOO_LARGE;
    const PackArgs a = {W, (uint8_t*)Q, S, Z, ldw, ldq, lds, ldz, (int32_t)F, (int32_t)K, group_of(group, K)};
    rc = check_w4_pack(a);
    if (rc) return rc;
    return status(launch_w4_quantize(dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

SGEMM_F32_API int sgemm_f32_w4_dequantize(int dtype, int64_t F, int64_t K, int64_t group,
                                          const void* Q, int64_t ldq, const void* S, int64_t lds,
                                          const void* Z, int64_t ldz, void* W, int64_t ldw,
                                          void* stream) {
    int rc = check_sizes(dtype, 0, F, K);
    if (rc) return rc;
    if (bad_group(group, K)) return -31;
    const int64_t e = dtype_bytes(dtype), groups = K > 0 ? cdiv(K, group) : 0;
    const bool out = F > 0 && K > 0;
    if (bad_ptr(out, Q, 1)) return -7;
    if (short_ld(ldq, cdiv(K, 2))) return -8;
    if (bad_ptr(out, S, e)) return -32;
    if (short_ld(lds, groups)) return -33;
    if (out && Z != nullptr && misaligned(Z, e)) return -34;
    if (Z != nullptr && short_ld(ldz, groups)) return -35;
    if (bad_ptr(out, W, e)) return -10;
    if (short_ld(ldw, K)) return -11;
    if (!out) return 0;
    if (too_large(0, F, K)) return SGEMM_F32_ERR_TOO_LARGE;
    const PackArgs a = {W, (uint8_t*)const_cast<void*>(Q), const_cast<void*>(S), const_cast<void*>(Z), ldw, ldq,
                        lds, ldz, (int32_t)F, (int32_t)K, group_of(group, K)};
    rc = check_w4_pack(a);
    if (rc) return rc;
    return status(launch_w4_dequantize(dtype, a, reinterpret_cast<hipStream_t>(stream)));
}

SGEMM_F32_API int sgemm_f32_w4(int dtype, int64_t M, int64_t F, int64_t K, int64_t group,
                               const void* X, int64_t ldx, const void* Q, int64_t ldq,
                               const void* S, int64_t lds, const void* Z, int64_t ldz, void* Y,
                               int64_t ldy, void* stream) {
    return run_w4(dtype, false, 0, M, F, K, group, X, ldx, Q, nullptr, ldq, S, nullptr, lds, Z, nullptr, ldz,
                  Y, ldy, stream);
}

SGEMM_F32_API int sgemm_f32_w4_glu(int dtype, int act, int64_t M, int64_t F, int64_t K,
                                   int64_t group, const void* X, int64_t ldx, const void* Qg,
                                   const void* Qu, int64_t ldq, const void* Sg, const void* Su,
                                   int64_t lds, const void* Zg, const void* Zu, int64_t ldz,
                                   void* H, int64_t ldh, void* stream) {
    return run_w4(dtype, true, act, M, F, K, group, X, ldx, Qg, Qu, ldq, Sg, Su, lds, Zg, Zu, ldz, H, ldh,
                  stream);
}

}  // extern "C"

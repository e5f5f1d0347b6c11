// Tile kernels of the gated block: the forward pass (both projections, the
// activation and the product in one kernel) and, for 16-bit types, the two
// products of the backward pass. FP32's backward products go through the
// library's own dispatch (ffn_api.hip).
#include "glu_core.hpp"

namespace sgemm {

static inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int GLU_GROUP_M = 8;

// H = act(X Wg^T) * (X Wu^T). A tile's columns alternate between the two
// weights in blocks of 32, so a wave holds G and U of the same outputs in
// registers, and neither is written unless the backward pass wants them.
template <class T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_glu_fwd(GluArgs a, int tiles_m,
                                                                       int tiles_n, int xcd) {
    using Core = TileCore<T, BM, BN, WM, WN, false, false, true>;
    static_assert(Core::BJ % 2 == 0, "a wave holds whole pairs of column blocks");
    __shared__ __attribute__((aligned(16))) char lds[2 * Core::STAGE];
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, GLU_GROUP_M, xcd != 0, tm, tn);
    const int m0 = tm * BM, f0 = tn * (BN / 2);
    f32x16 acc[Core::BI][Core::BJ];
    auto src = [&](int s, Lines<T>& la, Lines<T>* lb) {
        la = Lines<T>{(const T*)a.X, a.ldx, a.M, a.K};
        lb[0] = Lines<T>{(const T*)a.Wg, a.ldwg, a.F, a.K};
        lb[1] = Lines<T>{(const T*)a.Wu, a.ldwu, a.F, a.K};
        return s * Elem<T>::SLICE;
    };
    Core::run(lds, m0, f0, (a.K + Elem<T>::SLICE - 1) / Elem<T>::SLICE, src, acc);
    Core::each([&](int bi, int bj, int r, int i, int j) {
        if (bj & 1) return;
        const int row = m0 + i, f = f0 + (j >> 6) * 32 + (j & 31);
        if (row >= a.M || f >= a.F) return;
        const float g = acc[bi][bj][r], u = acc[bi][bj + 1][r];
        ((T*)a.H)[(int64_t)row * a.ldh + f] = (T)(act_value(a.act, g) * u);
        if (a.P != nullptr) {
            a.P[(int64_t)row * a.ldp + f] = g;
            a.P[(int64_t)row * a.ldp + a.F + f] = u;
        }
    });
}

// dX = dG Wg + dU Wu as one sum over 2F: first the slices of dG and Wg, then
// those of dU and Wu.
template <class T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_glu_dx(GluProdArgs a, int tiles_m,
                                                                      int tiles_n, int xcd) {
    using Core = TileCore<T, BM, BN, WM, WN, false, true, false>;
    __shared__ __attribute__((aligned(16))) char lds[2 * Core::STAGE];
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, GLU_GROUP_M, xcd != 0, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int half = (a.F + Elem<T>::SLICE - 1) / Elem<T>::SLICE;
    f32x16 acc[Core::BI][Core::BJ];
    auto src = [&](int s, Lines<T>& la, Lines<T>* lb) {
        const int u = s >= half;
        la = Lines<T>{(const T*)a.D[u], a.ldd, a.M, a.F};
        lb[0] = Lines<T>{(const T*)a.W[u], a.ldw[u], a.F, a.K};
        return (s - u * half) * Elem<T>::SLICE;
    };
    Core::run(lds, m0, n0, 2 * half, src, acc);
    Core::each([&](int bi, int bj, int r, int i, int j) {
        const int row = m0 + i, col = n0 + j;
        if (row < a.M && col < a.K) ((T*)a.C[0])[(int64_t)row * a.ldc[0] + col] = (T)acc[bi][bj][r];
    });
}

// dWg = dG^T X (blockIdx.y 0) and dWu = dU^T X (1): sums over the M tokens.
template <class T, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__((BM / WM) * (BN / WN) * 64) void k_glu_dw(GluProdArgs a, int tiles_m,
                                                                      int tiles_n, int xcd) {
    using Core = TileCore<T, BM, BN, WM, WN, true, true, false>;
    __shared__ __attribute__((aligned(16))) char lds[2 * Core::STAGE];
    const int u = a.C[0] == nullptr ? 1 : blockIdx.y;
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, GLU_GROUP_M, xcd != 0, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    f32x16 acc[Core::BI][Core::BJ];
    auto src = [&](int s, Lines<T>& la, Lines<T>* lb) {
        la = Lines<T>{(const T*)a.D[u], a.ldd, a.M, a.F};
        lb[0] = Lines<T>{(const T*)a.X, a.ldx, a.M, a.K};
        return s * Elem<T>::SLICE;
    };
    Core::run(lds, m0, n0, (a.M + Elem<T>::SLICE - 1) / Elem<T>::SLICE, src, acc);
    Core::each([&](int bi, int bj, int r, int i, int j) {
        const int f = m0 + i, col = n0 + j;
        if (f < a.F && col < a.K) ((T*)a.C[u])[(int64_t)f * a.ldc[u] + col] = (T)acc[bi][bj][r];
    });
}

constexpr int GB = 128, GW = 64;   // block and wave tile
constexpr int GNT = (GB / GW) * (GB / GW) * 64;

int check_glu(const GluArgs& a) {
    const int64_t tiles = cdiv(a.M, GB) * cdiv(a.F, GB / 2);
    return tiles <= max_workgroups(GNT) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

hipError_t launch_glu(int dtype, const GluArgs& a, hipStream_t s) {
    const int tm = (int)cdiv(a.M, GB), tn = (int)cdiv(a.F, GB / 2);
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        hipLaunchKernelGGL((k_glu_fwd<T, GB, GB, GW, GW>), dim3((unsigned)((int64_t)tm * tn)), dim3(GNT),
                           0, s, a, tm, tn, xcd_remap_enabled());
        return hipGetLastError();
    });
}

int check_glu_prod(const GluProdArgs& a) {
    const int64_t x = cdiv(a.M, GB) * cdiv(a.K, GB), w = cdiv(a.F, GB) * cdiv(a.K, GB);
    return x <= max_workgroups(GNT) && w <= max_workgroups(GNT) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

template <class Fn>
static hipError_t with_half(int dtype, Fn&& f) {
    if (dtype == SGEMM_F32_DTYPE_BF16) return f(TypeTag<bf16>{});
    return f(TypeTag<f16>{});
}

hipError_t launch_glu_dx(int dtype, const GluProdArgs& a, hipStream_t s) {
    const int tm = (int)cdiv(a.M, GB), tn = (int)cdiv(a.K, GB);
    return with_half(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        hipLaunchKernelGGL((k_glu_dx<T, GB, GB, GW, GW>), dim3((unsigned)((int64_t)tm * tn)), dim3(GNT),
                           0, s, a, tm, tn, xcd_remap_enabled());
        return hipGetLastError();
    });
}

hipError_t launch_glu_dw(int dtype, const GluProdArgs& a, hipStream_t s) {
    const int tm = (int)cdiv(a.F, GB), tn = (int)cdiv(a.K, GB);
    const unsigned both = a.C[0] != nullptr && a.C[1] != nullptr ? 2 : 1;
    return with_half(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        hipLaunchKernelGGL((k_glu_dw<T, GB, GB, GW, GW>), dim3((unsigned)((int64_t)tm * tn), both),
                           dim3(GNT), 0, s, a, tm, tn, xcd_remap_enabled());
        return hipGetLastError();
    });
}

}  // namespace sgemm

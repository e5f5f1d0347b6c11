// Products of matrices in 8 bits: Y = X W^T (i8) and the gated block over two such
// weights (i8_glu). The matrix cores sum the stored numbers exactly in 32 bits; the
// scales of a token and of a feature multiply each sum once, at the end.
#include "glu_core.hpp"
#include "i8.hpp"

namespace sgemm {

// A scale as mantissa and exponent: sum * Sx * Sw then leaves FP32's range, or its
// normal numbers, only where the result does (Sx = 2^-100, Sw = 2^90 and the other
// way round are ordinary).
struct Scale {
    float m;
    int e;
    __device__ __forceinline__ explicit Scale(float s)
        : m(__builtin_amdgcn_frexp_mantf(s)), e(__builtin_amdgcn_frexp_expf(s)) {}
};
__device__ __forceinline__ float scaled(int sum, const Scale& x, const Scale& w) {
    return __builtin_amdgcn_ldexpf((float)sum * x.m * w.m, x.e + w.e);
}
// The gate of the call's type: 16-bit results take the hardware's exponential.
template <class O>
__device__ __forceinline__ float gated(int act, float g, float u) {
    return act_value<sizeof(O) == 4>(act, g) * u;
}

// A tile's results: blocks of 32 rows of 32 (KS = 2: 16) features, or, without a gate, of all the
// wave's features together where they are next to each other.
template <class O, class Tl, class Core, bool DUAL>
__device__ __forceinline__ void put_i8(const I8Args& a, char* own, int m0, int n0,
                                       const i32x16 (&acc)[Core::BI][Core::BJ]) {
    const typename Tl::Map map;
    constexpr int REGS = Tl::Map::REGS, KS = 16 / REGS, STEP = DUAL ? 2 : KS == 1 ? Core::BJ : 1;
    constexpr int TOGETHER = DUAL ? 1 : STEP, COLS = 2 * REGS * TOGETHER;
    const RowsOut<O, COLS> o = {own, map.lane};
    static_assert(RowsOut<O, COLS>::BYTES <= Core::PER_WAVE, "staging");
    const int half = 4 * (map.lane >> 5);
#pragma unroll
    for (int bi = 0; bi < Core::BI; ++bi) {
        const int row = m0 + map.wm + 32 * bi, mine = row + (map.lane & 31);
        const Scale sx(a.Sx[mine < a.M ? mine : a.M - 1]);
#pragma unroll
        for (int bj = 0; bj < Core::BJ; bj += STEP) {
            const int f = n0 + (DUAL ? (map.wn + 32 * bj) >> 1 : map.wn + 32 * bj) + 2 * REGS * map.kk;
#pragma unroll
            for (int j = 0; j < TOGETHER; ++j)
#pragma unroll
                for (int r = 0; r < REGS; r += 4) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int c = f + 32 * j + 2 * r + half + e, at = c < a.F ? c : a.F - 1;
                        const float g = scaled(acc[bi][bj + j][r + e], sx, Scale(a.Sw[0][at]));
                        if constexpr (DUAL)
                            v[e] = gated<O>(a.act, g, scaled(acc[bi][bj + 1][r + e], sx, Scale(a.Sw[1][at])));
                        else
                            v[e] = g;
                    }
                    o.put(32 * j + 2 * r, v[0], v[1], v[2], v[3]);
                }
            o.flush((O*)a.Y + f, a.ldy, row, a.M, a.F - f);
        }
    }
}

// Y or H, tile by tile.
template <class Tl, bool DUAL>
__global__ __launch_bounds__(Tl::NT) void k_i8_tile(I8Args a, int tiles_m, int tiles_n, int xcd) {
    using Core = typename Tl::template Core<int8_t, false, false, DUAL>;
    static_assert(!DUAL || Core::BJ % 2 == 0, "a wave holds whole pairs of column blocks");
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, GLU_GROUP_M, xcd != 0, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * Tl::BM);
    const int n0 = __builtin_amdgcn_readfirstlane(tn * (DUAL ? Tl::BN / 2 : Tl::BN));
    i32x16 acc[Core::BI][Core::BJ];
    auto src = [&](int s, Lines<int8_t>& la, Lines<int8_t>* lb) {
        la = Lines<int8_t>{a.X, a.ldx, a.M, a.K};
        lb[0] = Lines<int8_t>{a.W[0], a.ldw[0], a.F, a.K};
        if (DUAL) lb[1] = Lines<int8_t>{a.W[1], a.ldw[1], a.F, a.K};
        return s * Elem<int8_t>::SLICE;
    };
    char* const own = product<Core, Tl::DMA>(m0, n0, 0, (a.K + Elem<int8_t>::SLICE - 1) / Elem<int8_t>::SLICE, src, acc);
    if (a.dtype == SGEMM_F32_DTYPE_F32)
        put_i8<float, Tl, Core, DUAL>(a, own, m0, n0, acc);
    else if (a.dtype == SGEMM_F32_DTYPE_BF16)
        put_i8<bf16, Tl, Core, DUAL>(a, own, m0, n0, acc);
    else
        put_i8<f16, Tl, Core, DUAL>(a, own, m0, n0, acc);
}

// Empty sums: zeros, without a look at the scales.
__global__ __launch_bounds__(256) void k_i8_zero(I8Args a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, m = i / a.F;
    if (m >= a.M) return;
    const int64_t at = m * a.ldy + (i - m * a.F);
    if (a.dtype == SGEMM_F32_DTYPE_F32)
        ((float*)a.Y)[at] = 0.0f;
    else
        ((uint16_t*)a.Y)[at] = 0;
}

int check_i8(const I8Args& a, bool dual) {
    const int64_t tiles = cdiv(a.M, 64) * cdiv(a.F, dual ? 32 : 64);
    const int64_t zeros = a.K == 0 ? cdiv((int64_t)a.M * a.F, 256) : 0;
    return tiles <= max_workgroups(512) && zeros <= max_workgroups(256) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

template <bool DUAL>
static hipError_t launch(const I8Args& a, hipStream_t s) {
    auto go = [&](auto tile) {
        using Tl = typename decltype(tile)::type;
        const int tm = (int)cdiv(a.M, Tl::BM), tn = (int)cdiv(a.F, DUAL ? Tl::BN / 2 : Tl::BN);
        hipLaunchKernelGGL((k_i8_tile<Tl, DUAL>), dim3((unsigned)((int64_t)tm * tn)), dim3(Tl::NT), 0, s, a, tm, tn,
                           xcd_remap_enabled());
        return hipGetLastError();
    };
    if (a.K < Elem<int8_t>::EPC) return go(TypeTag<TileShort>{});
    return go(TypeTag<TileReg>{});
}

hipError_t launch_i8(const I8Args& a, bool dual, hipStream_t s) {
    if (a.K == 0) {
        hipLaunchKernelGGL(k_i8_zero, dim3((unsigned)cdiv((int64_t)a.M * a.F, 256)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    return dual ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace sgemm

// Kernels of the gated block: the forward pass (both projections, the activation
// and the product in one kernel) and the two products of the backward pass.
// Large FP32 ones of those go through the library's own dispatch (ffn_api.hip).
#include "glu_core.hpp"

namespace sgemm {

constexpr int GLU_GROUP_M = 4;

// A core's product in LDS of its own: two stages for each operand, as objects
// apart so that the compiler can tell the stage being filled from the one
// being read.
// Returns LDS of the wave's own for the results.
template <class Core, bool DMA, class Src>
__device__ __forceinline__ char* product(int m0, int n0, int s_begin, int s_end, Src&& src,
                                        f32x16 (&acc)[Core::BI][Core::BJ]) {
    if constexpr (DMA) {
        __shared__ __attribute__((aligned(16))) char a0[Core::LDS_A], b0[Core::LDS_B], a1[Core::LDS_A],
            b1[Core::LDS_B];
        Core::run(a0, b0, a1, b1, m0, n0, s_begin, s_end, src, acc);
        return Core::own(a0, b0, a1, b1);
    } else {
        __shared__ __attribute__((aligned(16))) char lds[2 * Core::STAGE];
        Core::run(lds, m0, n0, s_begin, s_end, src, acc);
        return lds + (threadIdx.x >> 6) * Core::PER_WAVE;
    }
}

// Block and wave tile, and how it is filled: buffer-to-LDS loads (DMA) or
// through registers, element by element where rows are shorter than 16 bytes.
template <int BM_, int BN_, int WM_, int WN_, int KS_, bool DMA_, bool SHORT_ = false>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, NT = (BM_ / WM_) * (BN_ / WN_) * KS_ * 64;
    static constexpr bool DMA = DMA_;
    using Map = WaveMap<BM_, BN_, WM_, WN_, KS_>;
    template <class T, bool ARC, bool BRC, bool PAIR>
    using Core = std::conditional_t<DMA_, DmaCore<T, BM_, BN_, WM_, WN_, ARC, BRC, PAIR, KS_>,
                                    TileCore<T, BM_, BN_, WM_, WN_, ARC, BRC, PAIR, KS_, SHORT_>>;
};

// H = act(X Wg^T) * (X Wu^T). A tile's columns alternate between the two
// weights in blocks of 32, so a wave holds G and U of the same outputs in
// registers, and neither is written unless the backward pass wants them. Bound by the
// matrix cores: 4096 x 8192 x 4096 bf16 436-441 us (1.25 PFLOP/s, 82% of a
// large library product), 484-500 with the pre-activations (268 MB more
// written); FP32 2048 x 4096 x 2048 484 us (142 TFLOP/s, 93%).
template <class T, class Tl>
__global__ __launch_bounds__(Tl::NT) void k_glu_fwd(GluArgs a, int tiles_m, int tiles_n, int xcd) {
    using Core = typename Tl::template Core<T, false, false, true>;
    static_assert(Core::BJ % 2 == 0, "a wave holds whole pairs of column blocks");
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, GLU_GROUP_M, xcd != 0, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * Tl::BM), f0 = __builtin_amdgcn_readfirstlane(tn * (Tl::BN / 2));
    f32x16 acc[Core::BI][Core::BJ];
    auto src = [&](int s, Lines<T>& la, Lines<T>* lb) {
        la = Lines<T>{(const T*)a.X, a.ldx, a.M, a.K};
        lb[0] = Lines<T>{(const T*)a.Wg, a.ldwg, a.F, a.K};
        lb[1] = Lines<T>{(const T*)a.Wu, a.ldwu, a.F, a.K};
        return s * Elem<T>::SLICE;
    };
    char* const own = product<Core, Tl::DMA>(m0, f0, 0, (a.K + Elem<T>::SLICE - 1) / Elem<T>::SLICE, src, acc);
    // Block by block: 32 rows of the 32 (KS = 2: 16) features of a pair.
    const typename Tl::Map map;
    constexpr int REGS = Tl::Map::REGS, COLS = 2 * REGS;
    const RowsOut<T, COLS> h = {own, map.lane};
    const RowsOut<float, COLS> pg = {own, map.lane}, pu = {own + RowsOut<float, COLS>::BYTES, map.lane};
    static_assert(Core::PER_WAVE >= 2 * RowsOut<float, COLS>::BYTES, "staging");
#pragma unroll
    for (int bi = 0; bi < Core::BI; ++bi)
#pragma unroll
        for (int bj = 0; bj < Core::BJ; bj += 2) {
            const int row = m0 + map.wm + 32 * bi;
            const int f = f0 + ((map.wn + 32 * bj) >> 1) + COLS * map.kk;
            const f32x16 &g = acc[bi][bj], &u = acc[bi][bj + 1];
            if (a.P != nullptr) {
#pragma unroll
                for (int r = 0; r < REGS; r += 4) {
                    pg.put(2 * r, g[r], g[r + 1], g[r + 2], g[r + 3]);
                    pu.put(2 * r, u[r], u[r + 1], u[r + 2], u[r + 3]);
                }
                pg.flush(a.P + f, a.ldp, row, a.M, a.F - f);
                pu.flush(a.P + a.F + f, a.ldp, row, a.M, a.F - f);
            }
#pragma unroll
            for (int r = 0; r < REGS; r += 4) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = act_value<sizeof(T) == 4>(a.act, g[r + e]) * u[r + e];
                h.put(2 * r, v[0], v[1], v[2], v[3]);
            }
            h.flush((T*)a.H + f, a.ldh, row, a.M, a.F - f);
        }
}

// Sums over the wave's 64 lanes, of four values at a time: lane 16 r + x ends with
// value r's, in an order of additions that is fixed.
template <int CTRL>
__device__ __forceinline__ float plus_dpp(float v) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true);
    return v + __builtin_bit_cast(float, o);
}
__device__ __forceinline__ float lane_sums(float a, float b, float c, float d) {
    auto halves = [](float x, float y) {
        const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                        __builtin_bit_cast(uint32_t, y), false, false);
        return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
    };
    const float p = halves(a, c), q = halves(b, d);
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, p), __builtin_bit_cast(uint32_t, q),
                                                    false, false);
    float v = __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
    v = plus_dpp<0xB1>(v);
    v = plus_dpp<0x4E>(v);
    v = plus_dpp<0x141>(v);
    return plus_dpp<0x140>(v);
}

// The forward pass of very few rows on the vector units: a workgroup takes two
// features (four weight rows) and up to MR rows of X, and its four waves take K's
// kibibytes of each in turn, so that even a layer of a thousand features has all compute
// units reading its weights; 16 to 32 waves a unit keep enough loads in flight
// without a ring. Bound by the weights' bytes: one row of 8192 x 4096 bf16 23.9 us
// (134 MB, 5.6 TB/s), FP32 46 (5.8 TB/s); a row more costs MR's multiply-adds, 8 of FP32 62.
template <class T, int MR, bool SHORT>
__global__ __launch_bounds__(256) void k_glu_few(GluArgs a) {
    constexpr int EPC = Elem<T>::EPC, FW = 2, STEP = 64 * EPC;
    typedef T Vec __attribute__((ext_vector_type(EPC)));
    __shared__ float red[4][MR][4];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int f0 = blockIdx.x * FW, m0 = blockIdx.y * MR;
    const Lines<T> lx = {(const T*)a.X, a.ldx, a.M, a.K};
    const Lines<T> lw[2] = {{(const T*)a.Wg, a.ldwg, a.F, a.K}, {(const T*)a.Wu, a.ldwu, a.F, a.K}};
    float acc[MR][4] = {};   // [row][2 matrix + feature]
    for (int k0 = w * STEP; k0 < a.K; k0 += 4 * STEP) {
        const int at = k0 + lane * EPC;
        i32x4 v[4], x[MR];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load_chunk<SHORT>(lw[i >> 1], f0 + (i & 1), at);
#pragma unroll
        for (int m = 0; m < MR; ++m) x[m] = load_chunk<SHORT>(lx, m0 + m, at);
        if (k0 + STEP > a.K) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = place_chunk<SHORT>(v[i], lw[i >> 1], f0 + (i & 1), at);
#pragma unroll
            for (int m = 0; m < MR; ++m) x[m] = place_chunk<SHORT>(x[m], lx, m0 + m, at);
        }
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const Vec xs = __builtin_bit_cast(Vec, x[m]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Vec vs = __builtin_bit_cast(Vec, v[i]);
#pragma unroll
                for (int e = 0; e < EPC; ++e) acc[m][i] = __builtin_fmaf((float)xs[e], (float)vs[e], acc[m][i]);
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        const float v = lane_sums(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
        if ((lane & 15) == 0) red[w][m][lane >> 4] = v;
    }
    __syncthreads();
    const int m = threadIdx.x >> 1, f = threadIdx.x & 1;
    if (m < MR && m0 + m < a.M && f0 + f < a.F) {
        const float g = red[0][m][f] + red[1][m][f] + red[2][m][f] + red[3][m][f];
        const float u = red[0][m][2 + f] + red[1][m][2 + f] + red[2][m][2 + f] + red[3][m][2 + f];
        if (a.P != nullptr) {
            float* p = a.P + (int64_t)(m0 + m) * a.ldp + f0 + f;
            p[0] = g;
            p[a.F] = u;
        }
        ((T*)a.H)[(int64_t)(m0 + m) * a.ldh + f0 + f] = (T)(act_value<sizeof(T) == 4>(a.act, g) * u);
    }
}

// The forward pass of few rows: the weights' bytes are the work. A workgroup takes
// BM rows of X and 32 features; its KW waves take K's slices in turn, each with a
// ring of LDS stages of its own, so no wave waits for another before the sums
// are added in wave order at the end. Three stages keep two slices of every wave
// in flight (96 KiB a compute unit at BM = 32). 16 rows of 8192 x 4096 bf16
// from HBM 35.7 us (134.6 MB, 3.8 TB/s of the 5.1 that a large copy moves).
constexpr int KW = 4;
template <class T, int BM, bool DMA, bool SHORT>
__global__ __launch_bounds__(KW * 64) void k_glu_rows(GluArgs a) {
    constexpr int BN = 64, BI = BM / 32, STAGES = DMA && BM == 32 ? 3 : 2, STAGE = (BM + BN) * 128;
    static_assert(STAGES * STAGE >= BI * 2 * 16 * 64 * 4, "the sums fit in the rings");
    __shared__ __attribute__((aligned(16))) char lds[KW * STAGES * STAGE];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int f0 = blockIdx.x * 32, m0 = blockIdx.y * BM;
    const int nslices = (a.K + Elem<T>::SLICE - 1) / Elem<T>::SLICE;
    const int count = nslices > w ? (nslices - w + KW - 1) / KW : 0;
    char* const ring = lds + w * (STAGES * STAGE);
    const Lines<T> x = {(const T*)a.X, a.ldx, a.M, a.K};
    const Lines<T> wgt[2] = {{(const T*)a.Wg, a.ldwg, a.F, a.K}, {(const T*)a.Wu, a.ldwu, a.F, a.K}};
    f32x16 acc[BI][2];
#pragma unroll
    for (int i = 0; i < BI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    auto compute = [&](const char* A) {
        const char* B = A + BM * 128;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const i32x4 g = read_frag<T, BN, false>(B, 0, lane, v), u = read_frag<T, BN, false>(B, 32, lane, v);
#pragma unroll
            for (int i = 0; i < BI; ++i) {
                const i32x4 xv = read_frag<T, BM, false>(A, 32 * i, lane, v);
                mma_chunk(T{}, xv, g, acc[i][0]);
                mma_chunk(T{}, xv, u, acc[i][1]);
            }
        }
    };
    auto k_of = [&](int i) { return (w + KW * i) * Elem<T>::SLICE; };
    if constexpr (DMA) {
        DmaFill<T, BM, 64, false> fa;
        DmaFill<T, BN, 64, false> fb;
        fa.template init<false>(&x, m0, lane);
        fb.template init<true>(wgt, f0, lane);
        auto issue = [&](int i, char* st) {   // slices past K read as zeros
            fa.template issue<false>(&x, m0, k_of(i), lane, st);
            fb.template issue<true>(wgt, f0, k_of(i), lane, st + BM * 128);
        };
        if (count > 0) {
#pragma unroll
            for (int i = 0; i < STAGES - 1; ++i) issue(i, ring + i * STAGE);
            int at = 0;
            for (int i = 0; i < count; ++i) {
                const int to = at == 0 ? STAGES - 1 : at - 1;   // the stage read one slice ago
                lds_wait();
                issue(i + STAGES - 1, ring + to * STAGE);
                wave_wait<(STAGES - 1) * (decltype(fa)::G + decltype(fb)::G)>();
                compute(ring + at * STAGE);
                at = at == STAGES - 1 ? 0 : at + 1;
            }
            wave_wait<0>();
        }
    } else if (count > 0) {
        RegFill<T, BM, 64, false, SHORT> fa;
        RegFill<T, BN, 64, false, SHORT> fb;
        auto load = [&](int i) {
            fa.template load<false>(&x, m0, k_of(i), lane);
            fb.template load<true>(wgt, f0, k_of(i), lane);
        };
        load(0);
        for (int i = 0; i < count; ++i) {
            char* st = ring + (i & 1) * STAGE;
            fa.template store<false>(st, &x, m0, k_of(i), lane);
            fb.template store<true>(st + BM * 128, wgt, f0, k_of(i), lane);
            load(i + 1 < count ? i + 1 : i);
            compute(st);
        }
    }
    // Sums over the waves in their order.
    __syncthreads();
    float* const red = (float*)lds;
    constexpr int PER_WAVE = STAGES * STAGE / 4;
#pragma unroll
    for (int i = 0; i < BI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) red[w * PER_WAVE + ((i * 2 + j) * 16 + r) * 64 + lane] = acc[i][j][r];
    __syncthreads();
#pragma unroll
    for (int o = 0; o < BI * 16 / KW; ++o) {
        const int ir = w * (BI * 16 / KW) + o, i = ir >> 4, r = ir & 15;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int ww = 0; ww < KW; ++ww) {
            g += red[ww * PER_WAVE + (i * 32 + r) * 64 + lane];
            u += red[ww * PER_WAVE + (i * 32 + 16 + r) * 64 + lane];
        }
        const int row = m0 + 32 * i + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3), f = f0 + (lane & 31);
        if (row >= a.M || f >= a.F) continue;
        ((T*)a.H)[(int64_t)row * a.ldh + f] = (T)(act_value<sizeof(T) == 4>(a.act, g) * u);
        if (a.P != nullptr) {
            a.P[(int64_t)row * a.ldp + f] = g;
            a.P[(int64_t)row * a.ldp + a.F + f] = u;
        }
    }
}

// Where a backward product's sums go: the result, or, split over its slices
// (blockIdx.z of gridDim.z parts), FP32 partial sums that k_glu_sum adds in order.
// A wave's blocks of a block row go out together where their columns are
// next to each other (KS = 1).
template <class O, class Tl, class Core>
__device__ __forceinline__ void put_rows(char* own, O* out, int64_t ld, int m0, int n0, int rows, int cols,
                                         const f32x16 (&acc)[Core::BI][Core::BJ]) {
    const typename Tl::Map map;
    constexpr int REGS = Tl::Map::REGS, KS = 16 / REGS, TOGETHER = KS == 1 ? Core::BJ : 1, COLS = 2 * REGS * TOGETHER;
    const RowsOut<O, COLS> o = {own, map.lane};
    static_assert(RowsOut<O, COLS>::BYTES <= Core::PER_WAVE, "staging");
#pragma unroll
    for (int bi = 0; bi < Core::BI; ++bi)
#pragma unroll
        for (int bj = 0; bj < Core::BJ; bj += TOGETHER) {
            const int col = n0 + map.wn + 32 * bj + 2 * REGS * map.kk;
#pragma unroll
            for (int j = 0; j < TOGETHER; ++j)
#pragma unroll
                for (int r = 0; r < REGS; r += 4) {
                    const f32x16& v = acc[bi][bj + j];
                    o.put(32 * j + 2 * r, v[r], v[r + 1], v[r + 2], v[r + 3]);
                }
            o.flush(out + col, ld, m0 + map.wm + 32 * bi, rows, cols - col);
        }
}
template <class T, class Tl, class Core>
__device__ __forceinline__ void put(const GluProdArgs& a, int u, int rows, int m0, int n0, char* own,
                                    const f32x16 (&acc)[Core::BI][Core::BJ]) {
    if (gridDim.z > 1)
        put_rows<float, Tl, Core>(own, a.part + (int64_t)(blockIdx.z * gridDim.y + blockIdx.y) * rows * a.K, a.K, m0, n0,
                                  rows, a.K, acc);
    else
        put_rows<T, Tl, Core>(own, (T*)(u ? a.C[1] : a.C[0]), u ? a.ldc[1] : a.ldc[0], m0, n0, rows, a.K, acc);
}
// The sums of operands kept times a power of two (GluProdArgs::shift), without it:
// exact, but for sums below FP32's normal range.
template <class T, class Core>
__device__ __forceinline__ void unscale(const GluProdArgs& a, f32x16 (&acc)[Core::BI][Core::BJ]) {
    if constexpr (std::is_same_v<T, f16>) {
        if (a.shift == nullptr) return;
        const int n = -*a.shift;
#pragma unroll
        for (int i = 0; i < Core::BI; ++i)
#pragma unroll
            for (int j = 0; j < Core::BJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_amdgcn_ldexpf(acc[i][j][r], n);
    }
}
// This part's slices of n.
__device__ __forceinline__ void part_of(int n, int& begin, int& end) {
    const int per = (n + gridDim.z - 1) / gridDim.z;
    begin = blockIdx.z * per < n ? blockIdx.z * per : n;
    end = begin + per < n ? begin + per : n;
}

// dX = dG Wg + dU Wu as one sum over 2F: first the slices of dG and Wg, then
// those of dU and Wu; then, where dG and dU have second parts, the same with those.
// W is read [k][row], through transposed LDS reads. 4096 x 8192 x 4096 bf16
// 425-450 us (1.22-1.29 PFLOP/s).
template <class T, class Tl>
__global__ __launch_bounds__(Tl::NT) void k_glu_dx(GluProdArgs a, int tiles_m, int tiles_n, int xcd) {
    using Core = typename Tl::template Core<T, false, true, false>;
    int tm, tn, s0, s1;
    tile_of(blockIdx.x, tiles_m, tiles_n, GLU_GROUP_M, xcd != 0, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * Tl::BM), n0 = __builtin_amdgcn_readfirstlane(tn * Tl::BN);
    const int half = (a.F + Elem<T>::SLICE - 1) / Elem<T>::SLICE;
    part_of(a.L[0] != nullptr ? 4 * half : 2 * half, s0, s1);
    f32x16 acc[Core::BI][Core::BJ];
    auto src = [&](int s, Lines<T>& la, Lines<T>* lb) {
        // (slices past the last one are asked for too: their k lies past the sums)
        const bool second = a.L[0] != nullptr && s >= 2 * half;
        if (second) s -= 2 * half;
        const int u = s >= half;
        // (dG and dU are zero from F to whole slices)
        la = Lines<T>{(const T*)(second ? (u ? a.L[1] : a.L[0]) : (u ? a.D[1] : a.D[0])), a.ldd, a.M, half * Elem<T>::SLICE};
        lb[0] = Lines<T>{(const T*)(u ? a.W[1] : a.W[0]), a.ldw[0], a.F, a.K};
        if (!Tl::DMA) lb[0].ld = u ? a.ldw[1] : a.ldw[0];
        return (s - u * half) * Elem<T>::SLICE;
    };
    char* const own = product<Core, Tl::DMA>(m0, n0, s0, s1, src, acc);
    unscale<T, Core>(a, acc);
    put<T, Tl, Core>(a, 0, a.M, m0, n0, own, acc);
}

// dWg = dG^T X (blockIdx.y 0) and dWu = dU^T X (1): sums over the M tokens, of
// the second parts after the first where there are any. Both operands are
// read [k][row]. 4096 x 8192 x 4096 bf16 419-427 us (1.3 PFLOP/s).
template <class T, class Tl>
__global__ __launch_bounds__(Tl::NT) void k_glu_dw(GluProdArgs a, int tiles_m, int tiles_n, int xcd) {
    using Core = typename Tl::template Core<T, true, true, false>;
    const int u = a.C[0] == nullptr ? 1 : blockIdx.y;
    int tm, tn, s0, s1;
    tile_of(blockIdx.x, tiles_m, tiles_n, GLU_GROUP_M, xcd != 0, tm, tn);
    const int m0 = __builtin_amdgcn_readfirstlane(tm * Tl::BM), n0 = __builtin_amdgcn_readfirstlane(tn * Tl::BN);
    const int once = (a.M + Elem<T>::SLICE - 1) / Elem<T>::SLICE;
    part_of(a.L[0] != nullptr ? 2 * once : once, s0, s1);
    f32x16 acc[Core::BI][Core::BJ];
    auto src = [&](int s, Lines<T>& la, Lines<T>* lb) {
        const bool second = a.L[0] != nullptr && s >= once;
        if (second) s -= once;
        la = Lines<T>{(const T*)(second ? (u ? a.L[1] : a.L[0]) : (u ? a.D[1] : a.D[0])), a.ldd, a.M,
                      (a.F + 63) / 64 * 64};
        lb[0] = Lines<T>{(const T*)a.X, a.ldx, a.M, a.K};
        return s * Elem<T>::SLICE;
    };
    char* const own = product<Core, Tl::DMA>(m0, n0, s0, s1, src, acc);
    unscale<T, Core>(a, acc);
    put<T, Tl, Core>(a, u, a.F, m0, n0, own, acc);
}

// The sums of a split product's parts, in their order (bound by a launch at these
// sizes: 3-4 us).
template <class T>
__global__ __launch_bounds__(256) void k_glu_sum(GluProdArgs a, int rows, int parts) {
    const int64_t n = (int64_t)rows * a.K, at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= n) return;
    const int u = a.C[0] == nullptr ? 1 : blockIdx.y;
    float v = 0.0f;
    for (int z = 0; z < parts; ++z) v += a.part[((int64_t)z * gridDim.y + blockIdx.y) * n + at];
    const int64_t row = at / a.K;
    ((T*)(u ? a.C[1] : a.C[0]))[row * (u ? a.ldc[1] : a.ldc[0]) + (at - row * a.K)] = (T)v;
}

using TileReg = Tile<128, 128, 64, 64, 1, false>;
using TileReg64 = Tile<64, 64, 32, 64, 2, false>;
using TileDma64 = Tile<64, 64, 32, 64, 2, true>;
using TileShort = Tile<128, 128, 64, 64, 1, false, true>;
using TileMid = Tile<128, 128, 64, 64, 1, true>;
using TileBig = Tile<256, 256, 128, 64, 1, true>;

// Whether an operand of `lines` lines can be filled by buffer-to-LDS loads:
// whole 16-byte chunks, and a tile's span within 31-bit byte offsets.
static bool dma_ok(int dtype, const void* p, int64_t ld, int64_t extent, int64_t tile_lines) {
    const int64_t e = dtype_bytes(dtype), chunk = 16 / e;
    // (ld by itself first: a single line's may be anything)
    return aligned16(p) && ld % chunk == 0 && extent % chunk == 0 && ld < (int64_t)kRange &&
           ((tile_lines - 1) * ld + extent) * e < (int64_t)kRange;
}

// Times that the choice of a tile goes by, in microseconds, measured on MI355X
// (products of 300 x 1000 x 511 to 4096 x 8192 x 4096): a call takes about
//     fixed + n max(alone, tiles per compute unit * busy)
// for n slices, with `alone` a slice of a lone tile and `busy` a slice's share of a
// unit that holds several. FP32 slices hold half the k and take the matrix
// cores eight times as long; register-filled tiles wait longer per slice.
struct TileCost {
    double fixed, alone, busy;
    double of(int64_t tiles, int64_t slices) const {
        const double per_unit = (double)((tiles + 255) / 256), b = per_unit * busy;
        return fixed + (double)slices * (b > alone ? b : alone);
    }
};
// [FP32][filled through registers]
static const TileCost kBig[2] = {{9.0, 1.8, 1.8}, {9.0, 7.3, 7.3}};
static const TileCost kMid[2][2] = {{{7.0, 0.45, 0.52}, {7.0, 1.1, 0.85}}, {{7.0, 2.2, 2.0}, {7.0, 2.8, 2.2}}};
static const TileCost k64[2][2] = {{{6.0, 0.25, 0.19}, {6.0, 0.50, 0.30}}, {{6.0, 0.60, 0.60}, {6.0, 0.80, 0.73}}};

// f(tile tag): the tile that the model above finds fastest; filled through registers
// where an operand is not whole chunks (never the big tile: its registers
// are taken). SMALL: a product that is split, or an FP32 one, which only the
// 64 x 64 tiles take.
template <bool SMALL, class Fn>
static hipError_t with_tile(int dtype, int K, bool dma, int64_t rows, int64_t cols, int64_t copies, int64_t slices,
                            Fn&& f) {
    if (K < 16 / dtype_bytes(dtype)) return f(TypeTag<TileShort>{});
    if constexpr (!SMALL) {
        const int f32 = dtype == SGEMM_F32_DTYPE_F32;
        auto tiles = [&](int64_t b) { return cdiv(rows, b) * cdiv(cols, b) * copies; };
        const double small = k64[f32][!dma].of(tiles(64), slices), mid = kMid[f32][!dma].of(tiles(128), slices);
        if (dma) {
            const double big = kBig[f32].of(tiles(256), slices);
            if (big < mid && big < small) return f(TypeTag<TileBig>{});
            if (mid < small) return f(TypeTag<TileMid>{});
        } else if (mid < small) {
            return f(TypeTag<TileReg>{});
        }
    }
    return dma ? f(TypeTag<TileDma64>{}) : f(TypeTag<TileReg64>{});
}

// Parts that a product of few tiles is split into: as many as make 512 of the
// 64 x 64 tiles, or 1280 in FP32, whose slices take longer than their partial sums
// (dX of 1000 x 1531 x 777 84 us with 512, 78 with 1280; bf16 23 and 28), of at least
// four slices each. By sizes alone, so that the workspace's size does not
// depend on alignment.
static int parts(int dtype, int64_t rows, int64_t cols, int64_t copies, int64_t slices, int K) {
    const int64_t tiles = cdiv(rows, 64) * cdiv(cols, 64) * copies;
    if (tiles >= 256 || K < 8) return 1;
    const int64_t by_tiles = (dtype == SGEMM_F32_DTYPE_F32 ? 1280 : 512) / tiles, by_slices = slices / 4;
    const int64_t n = by_tiles < by_slices ? by_tiles : by_slices;
    return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}
static int64_t slice_of(int dtype) { return 128 / dtype_bytes(dtype); }
static int64_t dx_slices(int dtype, int64_t M, int64_t F) {
    return (glu_two_parts(dtype, M, F) ? 4 : 2) * cdiv(F, slice_of(dtype));
}
static int64_t dw_slices(int dtype, int64_t M, int64_t F) {
    return (glu_two_parts(dtype, M, F) ? 2 : 1) * cdiv(M, slice_of(dtype));
}
static int dx_parts(int dtype, int64_t M, int64_t F, int64_t K) {
    return parts(dtype, M, K, 1, dx_slices(dtype, M, F), (int)K);
}
// (as for both gradients, so that one alone has the same bits)
static int dw_parts(int dtype, int64_t M, int64_t F, int64_t K) {
    return parts(dtype, F, K, 2, dw_slices(dtype, M, F), (int)K);
}
// FP32 products up to 640 tiles run here, larger ones on the library's own dispatch
// (tiles of 64 x 64: dX of 77 x 1000 x 511 16.4 us against 18.3, 1000 x 1531 x 777 83
// against 89, dW of 4096 x 500 x 500 45 against 54; dX of 2000 x 2000 x 1500
// 230 against 214).
static bool here(int dtype, int64_t rows, int64_t cols, int64_t copies) {
    return dtype != SGEMM_F32_DTYPE_F32 || cdiv(rows, 64) * cdiv(cols, 64) * copies <= 640;
}
bool glu_dx_here(int dtype, int64_t M, int64_t K) { return here(dtype, M, K, 1); }
// (Of rows too far apart for the 32-bit offsets that the library's kernels take
// a transposed product's slice by, dW is made here too: tiles filled through
// registers, by 64-bit addresses. dX's plain product has a form for such rows.)
bool glu_dw_here(int dtype, int64_t F, int64_t K, int64_t ldd, int64_t ldx) {
    const int64_t ld = ldd > ldx ? ldd : ldx;
    return here(dtype, F, K, 2) || ld >= (int64_t)kRange / (64 * 4);
}
size_t glu_prod_bytes(int dtype, int64_t M, int64_t F, int64_t K) {
    if (M == 0 || F == 0 || K == 0) return 0;
    size_t most = 0;
    const int dx = dx_parts(dtype, M, F, K);
    if (dx > 1) most = (size_t)dx * M * K * 4;
    const int dw = dw_parts(dtype, M, F, K);
    if (dw > 1 && (size_t)dw * 2 * F * K * 4 > most) most = (size_t)dw * 2 * F * K * 4;
    return most;
}

int check_glu(const GluArgs& a) {
    const int64_t tiles = cdiv(a.M, 64) * cdiv(a.F, 32);
    return tiles <= max_workgroups(512) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

template <class T, int BM>
static hipError_t launch_glu_rows(const GluArgs& a, bool dma, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(a.F, 32), (unsigned)cdiv(a.M, BM));
    if (a.K < Elem<T>::EPC)
        hipLaunchKernelGGL((k_glu_rows<T, BM, false, true>), grid, dim3(KW * 64), 0, s, a);
    else if (dma)
        hipLaunchKernelGGL((k_glu_rows<T, BM, true, false>), grid, dim3(KW * 64), 0, s, a);
    else
        hipLaunchKernelGGL((k_glu_rows<T, BM, false, false>), grid, dim3(KW * 64), 0, s, a);
    return hipGetLastError();
}

template <class T, int MR>
static hipError_t launch_glu_few(const GluArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(a.F, 2), (unsigned)cdiv(a.M, MR));
    if (a.K < Elem<T>::EPC)
        hipLaunchKernelGGL((k_glu_few<T, MR, true>), grid, dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((k_glu_few<T, MR, false>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_glu(int dtype, const GluArgs& a, hipStream_t s) {
    const bool dma = dma_ok(dtype, a.X, a.ldx, a.K, 256) && dma_ok(dtype, a.Wg, a.ldwg, a.K, 128) &&
                     dma_ok(dtype, a.Wu, a.ldwu, a.K, 128);
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        // Very few rows, or few features: the vector units. In us, here against
        // k_glu_rows: F x K = 8192 x 4096 bf16 one row 24 and 35, four 26 and 35, eight
        // 34 and 36 (odd sizes 44 and 34), FP32 eight 62 and 67, sixteen 98 and 66; 1024 x
        // 4096 bf16 sixteen rows 10 and 13, 32 rows 15 and 14, FP32 15 and 43, 23
        // and 43; 1810 x 7435 FP32 one row 22 and 136, 32 rows 78 and 129.
        constexpr bool F32 = sizeof(T) == 4;
        const int64_t times = cdiv(a.M, 8);   // that the weights are read
        if (a.M <= 32 && cdiv(a.F, 2) <= max_workgroups(256) &&
            (a.M <= 4 || (a.M <= 8 && F32) || times * a.F <= (F32 ? 8192 : 4096))) {
            if (a.M <= 1) return launch_glu_few<T, 1>(a, s);
            if (a.M <= 2) return launch_glu_few<T, 2>(a, s);
            if (a.M <= 4) return launch_glu_few<T, 4>(a, s);
            return launch_glu_few<T, 8>(a, s);
        }
        // Few rows, or few tiles: the workgroups that split K (128 x 4096 x 4096
        // bf16 21 us against 35 on 64 x 64 tiles, 512 x 2048 x 2048 level).
        const int64_t wgs64 = cdiv(a.M, 64) * cdiv(a.F, 32), wgs32 = cdiv(a.M, 32) * cdiv(a.F, 32);
        if (a.M <= 32 || wgs32 <= 256) return launch_glu_rows<T, 32>(a, dma, s);
        if (a.M <= 64 || wgs64 <= 256) return launch_glu_rows<T, 64>(a, dma, s);
        return with_tile<false>(dtype, a.K, dma, a.M, 2 * (int64_t)a.F, 1, cdiv(a.K, Elem<T>::SLICE), [&](auto tile) {
            using Tl = typename decltype(tile)::type;
            const int tm = (int)cdiv(a.M, Tl::BM), tn = (int)cdiv(a.F, Tl::BN / 2);
            hipLaunchKernelGGL((k_glu_fwd<T, Tl>), dim3((unsigned)((int64_t)tm * tn)), dim3(Tl::NT), 0, s, a, tm,
                               tn, xcd_remap_enabled());
            return hipGetLastError();
        });
    });
}

int check_glu_prod(const GluProdArgs& a) {
    const int64_t x = cdiv(a.M, 64) * cdiv(a.K, 64), w = cdiv(a.F, 64) * cdiv(a.K, 64);
    return x <= max_workgroups(512) && w <= max_workgroups(512) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

// The tile of a backward product in n parts.
template <class T, class Fn>
static hipError_t pick(int dtype, int n, int K, bool dma, int64_t rows, int64_t cols, int64_t copies, int64_t slices,
                       Fn&& f) {
    if constexpr (sizeof(T) == 2)
        if (n == 1) return with_tile<false>(dtype, K, dma, rows, cols, copies, slices, f);
    return with_tile<true>(dtype, K, dma, rows, cols, copies, slices, f);
}

template <class T>
static hipError_t launch_sum(const GluProdArgs& a, int64_t rows, unsigned copies, int n, hipStream_t s) {
    hipLaunchKernelGGL((k_glu_sum<T>), dim3((unsigned)cdiv(rows * a.K, 256), copies), dim3(256), 0, s, a, (int)rows, n);
    return hipGetLastError();
}

hipError_t launch_glu_dx(int dtype, const GluProdArgs& a, hipStream_t s) {
    // One tile's lines: 256 rows of dG, or a slice's 64 of W.
    const bool dma = dma_ok(dtype, a.D[0], a.ldd, a.ldd, 256) && dma_ok(dtype, a.W[0], a.ldw[0], a.K, 64) &&
                     dma_ok(dtype, a.W[1], a.ldw[1], a.K, 64) && a.ldw[0] == a.ldw[1];
    const int n = dx_parts(dtype, a.M, a.F, a.K);
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        auto go = [&](auto tile) {
            using Tl = typename decltype(tile)::type;
            const int tm = (int)cdiv(a.M, Tl::BM), tn = (int)cdiv(a.K, Tl::BN);
            hipLaunchKernelGGL((k_glu_dx<T, Tl>), dim3((unsigned)((int64_t)tm * tn), 1, (unsigned)n), dim3(Tl::NT),
                               0, s, a, tm, tn, xcd_remap_enabled());
            return hipGetLastError();
        };
        const hipError_t e = pick<T>(dtype, n, a.K, dma, a.M, a.K, 1, dx_slices(dtype, a.M, a.F), go);
        return e != hipSuccess || n == 1 ? e : launch_sum<T>(a, a.M, 1, n, s);
    });
}

hipError_t launch_glu_dw(int dtype, const GluProdArgs& a, hipStream_t s) {
    const unsigned both = a.C[0] != nullptr && a.C[1] != nullptr ? 2 : 1;
    const bool dma = dma_ok(dtype, a.D[0], a.ldd, a.ldd, 64) && dma_ok(dtype, a.X, a.ldx, a.K, 64);
    const int n = dw_parts(dtype, a.M, a.F, a.K);
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        auto go = [&](auto tile) {
            using Tl = typename decltype(tile)::type;
            const int tm = (int)cdiv(a.F, Tl::BM), tn = (int)cdiv(a.K, Tl::BN);
            hipLaunchKernelGGL((k_glu_dw<T, Tl>), dim3((unsigned)((int64_t)tm * tn), both, (unsigned)n),
                               dim3(Tl::NT), 0, s, a, tm, tn, xcd_remap_enabled());
            return hipGetLastError();
        };
        const hipError_t e = pick<T>(dtype, n, a.K, dma, a.F, a.K, 2, dw_slices(dtype, a.M, a.F), go);
        return e != hipSuccess || n == 1 ? e : launch_sum<T>(a, a.F, both, n, s);
    });
}

}  // namespace sgemm

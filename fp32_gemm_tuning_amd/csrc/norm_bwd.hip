// The backward pass of the root-mean-square norm: dX row by row, and with the same
// reads dW as partial sums over the rows of each workgroup, which are then added in
// their order.
#include "norm_core.hpp"

namespace sgemm {

// N = H rstd, and the gradient that leaves the norm: rstd (dY W - N mean(dY W N)).
__device__ __forceinline__ float through(float dy, float w, float n, float rstd, float along) {
    return rstd * __builtin_fmaf(-n, along, dy * w);
}

// Rows that stay in registers, as in the forward pass: LANES lanes hold a row in C chunks each. A
// workgroup takes every gridDim.x-th row (group of rows), and each lane sums dW for its
// columns over them, so that one read of dY and H serves both gradients; the lanes' sums of the groups of a workgroup
// meet in LDS. Bound by its bytes (dY, H and dH read, dX written): 4096 x 8192 bf16 49 us in a kernel trace (268
// MB and 17 MB of partial sums, 5.8 TB/s); one pass for dX and one for dW took 79. At most two chunks a
// lane of 16-bit rows: their FP32 sums are twice the registers.
// X: dX is wanted, D: with a dH.
template <class T, int LANES, int C, bool SHORT, bool X, bool D>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES, 4) void k_norm_bwd(NormBwdArgs a) {
    constexpr int NT = LANES < 256 ? 256 : LANES, RPW = NT / LANES, N = Raw<T>::N, WIDTH = LANES * C * N;
    __shared__ float red[RPW > 1 ? RPW * WIDTH : NT / 64];
    const int lane = RPW == 1 ? threadIdx.x : threadIdx.x % LANES;
    const int sub = RPW == 1 ? 0 : LANES == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : threadIdx.x / LANES;
    int at[C];
    uint32_t place[C];
    Raw<T> w[C];
    float dw[C][N];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        at[c] = (c * LANES + lane) * N;
        place[c] = Raw<T>::template place_of<SHORT>(at[c], a.K);
        if constexpr (X) w[c].template load<SHORT>((const T*)a.W, place[c], a.K);
#pragma unroll
        for (int e = 0; e < N; ++e) dw[c][e] = 0.0f;
    }
    for (int64_t m0 = (int64_t)blockIdx.x * RPW; m0 < a.M; m0 += (int64_t)gridDim.x * RPW) {
        const int64_t mine = m0 + sub, m = mine < a.M ? mine : a.M - 1;
        const bool there = RPW == 1 || mine < a.M;
        Raw<T> d[C], h[C], o[C];
        const float rstd = a.rstd[m];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            d[c].template load<SHORT>((const T*)a.dY + m * a.lddy, place[c], a.K);
            h[c].template load<SHORT>((const T*)a.H + m * a.ldh, place[c], a.K);
        }
        if constexpr (X) {
            if constexpr (D) {
#pragma unroll
                for (int c = 0; c < C; ++c) o[c].template load<SHORT>((const T*)a.dH + m * a.lddh, place[c], a.K);
            }
            float along = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                d[c].forget();
                h[c].forget();
                w[c].forget();
                if ((c + 1) * LANES * N <= a.K) {
#pragma unroll
                    for (int e = 0; e < N; ++e)
                        along = __builtin_fmaf((float)d[c].v[e] * (float)w[c].v[e], (float)h[c].v[e] * rstd, along);
                } else {
                    const int first = Raw<T>::first(at[c], place[c]);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float s = __builtin_fmaf((float)d[c].v[e] * (float)w[c].v[e], (float)h[c].v[e] * rstd, along);
                        along = e >= first ? s : along;
                    }
                }
            }
            // dH has arrived before the barriers of the sum: dX may be written over it, and a chunk moved back from
            // the row's end reads what another wave writes.
            if constexpr (D && LANES > 64) {
#pragma unroll
                for (int c = 0; c < C; ++c) o[c].forget();
            }
            along = over_row<LANES>(along, Plus{}, red) / (float)a.K;
            if (there) {
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    d[c].forget();
                    h[c].forget();
                    w[c].forget();
                    Raw<T> x;
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float n = (float)h[c].v[e] * rstd;
                        const float g = through((float)d[c].v[e], (float)w[c].v[e], n, rstd, along);
                        x.v[e] = (T)as_f32(D ? (float)o[c].v[e] + g : g);
                        dw[c][e] = __builtin_fmaf((float)d[c].v[e], n, dw[c][e]);
                    }
                    if (at[c] < a.K) x.template store<SHORT>((T*)a.dX + m * a.lddx, place[c], a.K);
                }
            }
        } else if (there) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    dw[c][e] = __builtin_fmaf((float)d[c].v[e], (float)h[c].v[e] * rstd, dw[c][e]);
        }
    }
    if (a.dW == nullptr) return;
    float* const part = a.part + (int64_t)blockIdx.x * a.K;
    if constexpr (RPW == 1) {
        // (a chunk moved back from the row's end has its neighbour's sums too, the same ones)
        typedef f32x4 F4u __attribute__((aligned(4)));
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < N; e += 4)
                if (at[c] < a.K)
                    *(F4u*)(part + place[c] + e) = f32x4{dw[c][e], dw[c][e + 1], dw[c][e + 2], dw[c][e + 3]};
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (at[c] < a.K) red[sub * WIDTH + place[c] + e] = dw[c][e];
        __syncthreads();
        for (int k = threadIdx.x; k < a.K; k += NT) {
            float s = red[k];
#pragma unroll
            for (int g = 1; g < RPW; ++g) s += red[g * WIDTH + k];
            part[k] = s;
        }
    }
}

// dX of longer rows: a workgroup a row, read twice; dW's kernels read dY and H once more. Bound by those reads: 512
// x 65536 bf16 with dH and dW 99 us (268 MB read and written once, 2.7 TB/s), 1024 x 28672 97 (2.4 TB/s), one row of
// 65536 20. In 16 bits this begins at 16385 elements: 1024 x 16384 in registers 32 us, 1024 x 16392 58.
constexpr int LONG_NT = 1024;
template <class T>
__global__ __launch_bounds__(LONG_NT) void k_norm_dx_long(NormBwdArgs a) {
    constexpr int N = Chunk<T>::N, STEP = LONG_NT * N;
    __shared__ float red[LONG_NT / 64];
    const int first = threadIdx.x * N;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const T* dy = (const T*)a.dY + m * a.lddy;
        const T* h = (const T*)a.H + m * a.ldh;
        const float rstd = a.rstd[m];
        float along = 0.0f;
        for (int at = first; at < a.K; at += STEP) {
            Chunk<T> d, w, n;
            d.load(dy, at, a.K);
            w.load((const T*)a.W, at, a.K);
            n.load(h, at, a.K);
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (at + e < a.K) along = __builtin_fmaf(d.v[e] * w.v[e], n.v[e] * rstd, along);
        }
        along = over_row<LONG_NT>(along, Plus{}, red) / (float)a.K;
        for (int at = first; at < a.K; at += STEP) {
            Chunk<T> d, w, n, o;
            d.load(dy, at, a.K);
            w.load((const T*)a.W, at, a.K);
            n.load(h, at, a.K);
            if (a.dH != nullptr) o.load((const T*)a.dH + m * a.lddh, at, a.K);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float g = through(d.v[e], w.v[e], n.v[e] * rstd, rstd, along);
                o.v[e] = as_f32(a.dH != nullptr ? o.v[e] + g : g);
            }
            o.store((T*)a.dX + m * a.lddx, at, a.K);
        }
    }
}

// Their partial sums of dW: a thread one chunk of columns of the rows of part blockIdx.y.
template <class T>
__global__ __launch_bounds__(256) void k_norm_dw_long(NormBwdArgs a, int rows) {
    constexpr int N = Chunk<T>::N;
    const int at = (blockIdx.x * 256 + threadIdx.x) * N;
    if (at >= a.K) return;
    const int64_t m0 = (int64_t)blockIdx.y * rows, m1 = m0 + rows < a.M ? m0 + rows : a.M;
    float s[N] = {};
    for (int64_t m = m0; m < m1; ++m) {
        Chunk<T> d, n;
        d.load((const T*)a.dY + m * a.lddy, at, a.K);
        n.load((const T*)a.H + m * a.ldh, at, a.K);
        const float rstd = a.rstd[m];
#pragma unroll
        for (int e = 0; e < N; ++e) s[e] = __builtin_fmaf(d.v[e], n.v[e] * rstd, s[e]);
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
        if (at + e < a.K) a.part[(int64_t)blockIdx.y * a.K + at + e] = s[e];
}

// The parts' sums: 64 columns a workgroup, whose sixteen waves take every sixteenth
// part and meet in their order. Bound by its launch and its loads' latency, eight parts a batch one after the
// other: 512 parts of 8192 4.7 us, 500 of 1531 5.6 in 24 workgroups, beside 6.3 for the pass before it (one thread a
// column 61 us for 256 parts of 8192).
template <class T>
__global__ __launch_bounds__(1024) void k_norm_dw_sum(NormBwdArgs a, int parts) {
    __shared__ float red[16][64];
    // (blockIdx.y: rows of 2^28 and more have more blocks of columns than one line of the grid has threads for)
    const int block = blockIdx.y * gridDim.x + blockIdx.x;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, k = block * 64 + lane;
    float s = 0.0f;
    if (k < a.K) {
#pragma unroll 8
        for (int p = w; p < parts; p += 16) s += a.part[(int64_t)p * a.K + k];
    }
    red[w][lane] = s;
    __syncthreads();
    if (w != 0 || k >= a.K) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) s += red[i][lane];
    ((T*)a.dW)[k] = (T)s;
}

// How rows of K are held, by their 16-byte chunks, and how many workgroups share the rows.
struct Hold {
    int lanes, chunks;   // lanes 0: long rows
    int64_t parts;
};
static Hold hold_of(int dtype, int64_t M, int64_t K) {
    const int64_t n = 16 / dtype_bytes(dtype), v = (K + n - 1) / n;
    Hold h;
    if (v <= 16) h = {16, 1, 0};
    else if (v <= 32) h = {16, 2, 0};
    else if (v <= 64) h = {64, 1, 0};
    else if (v <= 128) h = {64, 2, 0};
    else if (v <= 256) h = {256, 1, 0};
    else if (v <= 512) h = {256, 2, 0};
    else if (v <= 1024) h = {512, 2, 0};
    else if (v <= 2048) h = {1024, 2, 0};
    else if (v <= 4096 && dtype == SGEMM_F32_DTYPE_F32) h = {1024, 4, 0};
    else {
        const int64_t rows = (M + 255) / 256 < 16 ? 16 : (M + 255) / 256;
        return {0, (int)rows, (M + rows - 1) / rows};
    }
    // Two rows (groups of rows) a workgroup at least: its partial sums are half of a row's bytes (256 x
    // 8192 bf16 in 128 parts 10.4 us, 256 11.8, 64 12.7), and two workgroups a compute unit at most, one of
    // the largest (4096 x 8192 bf16 512 parts 49 us, 256 55; FP32, on 1024 lanes, 105 and 103, 1000 x 8192 31 and 26).
    const int64_t per = h.lanes < 256 ? 256 / h.lanes : 1, pairs = ((M + per - 1) / per + 1) / 2;
    const int64_t most = h.lanes == 1024 ? 256 : 512;
    h.parts = pairs < most ? pairs : most;
    return h;
}

size_t norm_part_bytes(int dtype, int64_t M, int64_t K) {
    return (size_t)hold_of(dtype, M, K).parts * (size_t)K * sizeof(float);
}

hipError_t launch_norm_bwd(int dtype, const NormBwdArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        constexpr int N = Raw<T>::N;
        int64_t parts = 0;
        hipError_t e = hipSuccess;
        auto held = [&](auto lanes, auto chunks, auto is_short) {
            constexpr int LANES = decltype(lanes)::value, C = decltype(chunks)::value;
            constexpr bool SHORT = decltype(is_short)::value;
            auto* const k = a.dX == nullptr ? k_norm_bwd<T, LANES, C, SHORT, false, false>
                            : a.dH == nullptr ? k_norm_bwd<T, LANES, C, SHORT, true, false>
                                              : k_norm_bwd<T, LANES, C, SHORT, true, true>;
            hipLaunchKernelGGL(k, dim3((unsigned)parts), dim3(LANES < 256 ? 256 : LANES), 0, s, a);
        };
        if (a.M > 0) {
            const Hold h = hold_of(dtype, a.M, a.K);
            parts = h.parts;
            using std::integral_constant;
            const std::false_type no;
            if (h.lanes == 0) {
                // dW first: dX may be written over dY
                if (a.dW != nullptr)
                    hipLaunchKernelGGL((k_norm_dw_long<T>), dim3((unsigned)((a.K + 256 * N - 1) / (256 * N)), (unsigned)parts),
                                       dim3(256), 0, s, a, h.chunks);
                if (a.dX != nullptr)
                    hipLaunchKernelGGL((k_norm_dx_long<T>), dim3((unsigned)(a.M < (1 << 20) ? a.M : 1 << 20)),
                                       dim3(LONG_NT), 0, s, a);
            } else if (a.K < N) {
                held(integral_constant<int, 16>{}, integral_constant<int, 1>{}, std::true_type{});
            } else if (h.lanes == 16) {
                if (h.chunks == 1) held(integral_constant<int, 16>{}, integral_constant<int, 1>{}, no);
                else held(integral_constant<int, 16>{}, integral_constant<int, 2>{}, no);
            } else if (h.lanes == 64) {
                if (h.chunks == 1) held(integral_constant<int, 64>{}, integral_constant<int, 1>{}, no);
                else held(integral_constant<int, 64>{}, integral_constant<int, 2>{}, no);
            } else if (h.lanes == 256) {
                if (h.chunks == 1) held(integral_constant<int, 256>{}, integral_constant<int, 1>{}, no);
                else held(integral_constant<int, 256>{}, integral_constant<int, 2>{}, no);
            } else if (h.lanes == 512) {
                held(integral_constant<int, 512>{}, integral_constant<int, 2>{}, no);
            } else if (h.chunks == 2) {
                held(integral_constant<int, 1024>{}, integral_constant<int, 2>{}, no);
            } else if constexpr (sizeof(T) == 4) {
                held(integral_constant<int, 1024>{}, integral_constant<int, 4>{}, no);
            }
            e = hipGetLastError();
        }
        if (e == hipSuccess && a.dW != nullptr) {
            const int blocks = (a.K + 63) / 64, line = 1 << 20, lines = (blocks + line - 1) / line;
            hipLaunchKernelGGL((k_norm_dw_sum<T>), dim3((unsigned)(lines > 1 ? line : blocks), (unsigned)lines),
                               dim3(1024), 0, s, a, (int)parts);
            e = hipGetLastError();
        }
        return e;
    });
}

}  // namespace sgemm

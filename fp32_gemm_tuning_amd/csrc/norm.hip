// Root-mean-square norm of rows, after the residual is added: to the type, or to 8
// bits; matrices to 8 bits and back.
#include "norm_core.hpp"

namespace sgemm {

enum NormMode { NORM_Y, NORM_Q, PACK_Q };

// One row of any length by the LANES lanes that hold it, N elements at a time, read again for every pass (from
// the sum H where that was written: X may be the same memory): rows too long for registers, and,
// element by element, which takes few registers, rows whose numbers are not ordinary.
template <class T, NormMode MODE, int LANES, int N>
__device__ __forceinline__ void norm_row(const NormArgs& a, int64_t m, int lane, double* red) {
    constexpr int STEP = LANES * N;
    const int first = lane * N;
    const T* x = (const T*)a.X + m * a.ldx;
    const T* r = MODE != PACK_Q && a.R != nullptr ? (const T*)a.R + m * a.ldr : nullptr;
    T* h = MODE != PACK_Q && a.H != nullptr ? (T*)a.H + m * a.ldh : nullptr;
    const T* w = (const T*)a.W;
    bool kept = false;   // H holds the sums
    // The sum of the residual stream, rounded to the type, as FP32.
    auto sum = [&](int at, Chunk<T, N>& c) {
        if (kept) {
            c.load(h, at, a.K);
            return;
        }
        c.load(x, at, a.K);
        if (r != nullptr) {
            Chunk<T, N> d;
            d.load(r, at, a.K);
#pragma unroll
            for (int e = 0; e < N; ++e) c.v[e] = (float)(T)as_f32(c.v[e] + d.v[e]);
        }
    };
    float rstd = 1.0f;
    if constexpr (MODE != PACK_Q) {
        float ss = 0.0f;
#pragma unroll 1
        for (int at = first; at < a.K; at += STEP) {
            Chunk<T, N> c;
            sum(at, c);
            if (h != nullptr) c.store(h, at, a.K);
#pragma unroll
            for (int e = 0; e < N; ++e) ss = __builtin_fmaf(c.v[e], c.v[e], ss);
        }
        kept = h != nullptr;
        ss = over_row<LANES>(ss, Plus{}, (float*)red);
        rstd = rstd_of(ss, a.K, a.eps);
        if (sum_lost(ss, a.eps)) {
            uint32_t top = 0;
#pragma unroll 1
            for (int at = first; at < a.K; at += STEP) {
                Chunk<T, N> c;
                sum(at, c);
#pragma unroll
                for (int e = 0; e < N; ++e) top = Max{}(top, __builtin_bit_cast(uint32_t, fabsf(c.v[e])));
            }
            top = over_row<LANES>(top, Max{}, (uint32_t*)red);
            if (top > 0 && top < 0x7F800000u) {
                const int shift = __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, top));
                ss = 0.0f;
#pragma unroll 1
                for (int at = first; at < a.K; at += STEP) {
                    Chunk<T, N> c;
                    sum(at, c);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float s = __builtin_amdgcn_ldexpf(c.v[e], -shift);
                        ss = __builtin_fmaf(s, s, ss);
                    }
                }
                ss = over_row<LANES>(ss, Plus{}, (float*)red);
                rstd = rstd_scaled(ss, shift, a.K, a.eps);
            }
        }
        if (a.rstd != nullptr && lane == 0) a.rstd[m] = rstd;
    }
    if constexpr (MODE == NORM_Y) {
        T* y = (T*)a.Y + m * a.ldy;
#pragma unroll 1
        for (int at = first; at < a.K; at += STEP) {
            Chunk<T, N> c, g;
            sum(at, c);
            g.load(w, at, a.K);
#pragma unroll
            for (int e = 0; e < N; ++e) c.v[e] = as_f32(c.v[e] * rstd * g.v[e]);
            c.store(y, at, a.K);
        }
    } else {
        // What is brought to 8 bits, in 64 bits: H W exactly, or X.
        auto value = [&](int at, double (&v)[N]) {
            Chunk<T, N> c, g;
            sum(at, c);
            if constexpr (MODE == NORM_Q) g.load(w, at, a.K);
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = MODE == NORM_Q ? (double)c.v[e] * (double)g.v[e] : (double)c.v[e];
        };
        double top = 0.0, bad = 0.0;
#pragma unroll 1
        for (int at = first; at < a.K; at += STEP) {
            double v[N];
            value(at, v);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                top = fmax(top, fabs(v[e]));
                bad = __builtin_fma(v[e], 0.0, bad);   // 0, or NaN of an infinity or NaN
            }
        }
        top = over_row<LANES>(top, Max{}, red);
        bad = over_row<LANES>(bad, Plus{}, red);
        const bool flat = !(bad == 0.0) || top == 0.0;
        if (lane == 0)
            a.S[m] = bad == 0.0 ? (a.K > 0 ? (float)(top * (double)rstd / 127.0) : 0.0f) : __builtin_nanf("");
        const double inv = flat ? 0.0 : 127.0 / top;
        int8_t* q = a.Q + m * a.ldq;
#pragma unroll 1
        for (int at = first; at < a.K; at += STEP) {
            double v[N];
            int n[N];
            value(at, v);
            levels(v, inv, flat ? 1.0 : top, n);
#pragma unroll
            for (int e = 0; e < N; ++e) n[e] = flat ? 0 : n[e];
            store_levels(q, at, a.K, n);
        }
    }
}

// Longer rows: a workgroup each, read from the caches or memory in every pass. Bound by those
// reads: 512 x 65536 bf16 with a residual 59 us (268 MB, 4.5 TB/s), one row 11. In 8 bits also by the passes'
// arithmetic, in 64 bits for every type: with a residual 76 us (235 MB, 3.1 TB/s), one row 23; a matrix alone 512 x
// 53248 bf16 30 (82 MB, 2.7 TB/s), FP32 38 (136 MB, 3.6 TB/s).
constexpr int LONG_NT = 1024;
template <class T, NormMode MODE>
__global__ __launch_bounds__(LONG_NT) void k_norm_long(NormArgs a) {
    __shared__ double red[LONG_NT / 64];
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) norm_row<T, MODE, LONG_NT, Raw<T>::N>(a, m, threadIdx.x, red);
}

// Rows that stay in registers: LANES lanes hold a row in C chunks each, part of a wave, a wave or a
// workgroup, so that it is read once. Bound by its bytes: calls back to back, 4096 x 8192 bf16 with a residual
// take 42 us (268 MB, 6.3 TB/s, some of it cached), 131072 x 128 f16 12 (5.4 TB/s), 4096 x 8192 bf16 with a residual
// to 8 bits 40 (235 MB, 5.8 TB/s), 8192 x 8192 FP32 to 8 bits 64 (335 MB, 5.2 TB/s), one row of 8192 bf16 2.6. What leaves the ordinary
// (squares or products next to the ends of FP32's range, infinities, NaN) is left to norm_row, which starts
// anew: nothing has been written by then.
template <class T, NormMode MODE, int LANES, int C, bool SHORT>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES, 4) void k_norm(NormArgs a) {
    constexpr int NT = LANES < 256 ? 256 : LANES, RPW = NT / LANES, N = Raw<T>::N;
    __shared__ double red[NT / 64];
    // A row's number is the same in all lanes of a wave or workgroup that holds it: its addresses are a
    // scalar and an offset.
    const int lane = RPW == 1 ? threadIdx.x : threadIdx.x % LANES;
    const int sub = RPW == 1 ? 0 : LANES == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : threadIdx.x / LANES;
    int at[C];
    uint32_t place[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        at[c] = (c * LANES + lane) * N;
        place[c] = Raw<T>::template place_of<SHORT>(at[c], a.K);
    }
    // W stays in registers from row to row, or, where the longest rows leave no room, is read with each.
    constexpr bool KEEP = MODE != PACK_Q && LANES * C < 4096;
    Raw<T> w[C];
    auto load_w = [&]() {
#pragma unroll
        for (int c = 0; c < C; ++c) w[c].template load<SHORT>((const T*)a.W, place[c], a.K);
    };
    if constexpr (KEEP) load_w();
    for (int64_t m0 = (int64_t)blockIdx.x * RPW; m0 < a.M; m0 += (int64_t)gridDim.x * RPW) {
        // Groups past the last row do its work again and write nothing.
        const int64_t mine = m0 + sub, m = mine < a.M ? mine : a.M - 1;
        const bool there = RPW == 1 || mine < a.M;
        Raw<T> h[C], r[C];
#pragma unroll
        for (int c = 0; c < C; ++c)
            h[c].template load<SHORT>((const T*)a.X + m * a.ldx, place[c], a.K);
        const bool add = MODE != PACK_Q && a.R != nullptr;
        if (add) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                r[c].template load<SHORT>((const T*)a.R + m * a.ldr, place[c], a.K);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < N; ++e) h[c].v[e] = (T)as_f32((float)h[c].v[e] + (float)r[c].v[e]);
        }
        float rstd = 1.0f;
        bool usual = true;
        if constexpr (MODE != PACK_Q) {
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if ((c + 1) * LANES * N <= a.K) {
#pragma unroll
                    for (int e = 0; e < N; ++e) ss = __builtin_fmaf((float)h[c].v[e], (float)h[c].v[e], ss);
                } else {
                    const int first = Raw<T>::first(at[c], place[c]);
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        const float x = e >= first ? (float)h[c].v[e] : 0.0f;
                        ss = __builtin_fmaf(x, x, ss);
                    }
                }
            }
            if constexpr (!KEEP) load_w();
            ss = over_row<LANES>(ss, Plus{}, (float*)red);
            rstd = rstd_of(ss, a.K, a.eps);
            usual = !sum_lost(ss, a.eps);
        }
        auto keep = [&]() {
            if constexpr (MODE != PACK_Q) {
                if (a.H != nullptr) {
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        if (at[c] < a.K) h[c].template store<SHORT>((T*)a.H + m * a.ldh, place[c], a.K);
                }
                if (a.rstd != nullptr && lane == 0) a.rstd[m] = rstd;
            }
        };
        if constexpr (MODE == NORM_Y) {
            if (usual && there) {
                keep();
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    Raw<T> y;
                    h[c].forget();
                    w[c].forget();
#pragma unroll
                    for (int e = 0; e < N; ++e) y.v[e] = (T)as_f32((float)h[c].v[e] * rstd * (float)w[c].v[e]);
                    if (at[c] < a.K) y.template store<SHORT>((T*)a.Y + m * a.ldy, place[c], a.K);
                }
            }
        } else {
            // 16-bit numbers and their products are FP32 numbers, FP32's products 64-bit ones.
            using V = std::conditional_t<sizeof(T) == 4 && MODE == NORM_Q, double, float>;
            auto value = [&](int c, int e) {
                return MODE == NORM_Q ? (V)(float)h[c].v[e] * (V)(float)w[c].v[e] : (V)(float)h[c].v[e];
            };
            V top, inv;
            if constexpr (sizeof(V) == 8) {
                double t = 0.0, bad = 0.0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    h[c].forget();
                    w[c].forget();
#pragma unroll
                    for (int e = 0; e < N; ++e) {
                        t = fmax(t, fabs(value(c, e)));
                        bad = __builtin_fma(value(c, e), 0.0, bad);
                    }
                }
                t = over_row<LANES>(bad == 0.0 ? t : __builtin_inf(), Max{}, red);
                usual = usual && t <= 1.0e300;
                top = t;
            } else {
                // (as whole numbers, so that infinities and NaN are the largest)
                uint32_t t = 0;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    h[c].forget();
                    if constexpr (MODE != PACK_Q) w[c].forget();
#pragma unroll
                    for (int e = 0; e < N; ++e) t = Max{}(t, __builtin_bit_cast(uint32_t, fabsf((float)value(c, e))));
                }
                top = __builtin_bit_cast(float, over_row<LANES>(t, Max{}, (uint32_t*)red));
                usual = usual && (ordinary(top) || top == 0.0f);
                if (top == 0.0f) {   // zeros, or products that have become zero
                    uint32_t any = 0;
#pragma unroll
                    for (int c = 0; c < C; ++c) any |= h[c].any();
                    usual = usual && over_row<LANES>(any, Or{}, (uint32_t*)red) == 0;
                }
            }
            inv = top > 0 ? (V)127 / top : 0;
            if (usual && there) {
                keep();
                // (a row of zeros with eps = 0: 0 * infinity)
                if (lane == 0) a.S[m] = (float)((double)top * (double)rstd / 127.0);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    V v[N];
                    int q[N];
                    h[c].forget();
                    if constexpr (MODE != PACK_Q) w[c].forget();
#pragma unroll
                    for (int e = 0; e < N; ++e) v[e] = value(c, e);
                    levels(v, inv, top, q);
                    if constexpr (SHORT)
                        store_levels(a.Q + m * a.ldq, at[c], a.K, q);
                    else if (at[c] < a.K)
                        Bytes<N>::store(a.Q + m * a.ldq + place[c], q);
                }
            }
        }
        if (!usual && there) norm_row<T, MODE, LANES, 1>(a, m, lane, red);
    }
}

// Values of matrices in 8 bits: the chunks of 16 bytes of all rows in a line, four a thread, a workgroup's threads side
// by side in each. Bound by the bytes written: 8192 x 8192 FP32 58 us (335 MB, 5.7 TB/s; 64 bytes a thread in a
// line, so that a store instruction leaves gaps, 98).
constexpr int DQ_NT = 256, DQ_CHUNKS = 4;
template <class T>
__global__ __launch_bounds__(DQ_NT) void k_i8_dequantize(DequantArgs a, int per_row) {
    constexpr int N = Raw<T>::N;
    typedef int W __attribute__((ext_vector_type(N / 4)));
    typedef W Wu __attribute__((aligned(1)));
    const int64_t chunk0 = (int64_t)blockIdx.x * (DQ_NT * DQ_CHUNKS), m0 = chunk0 / per_row;
    const uint32_t rest = (uint32_t)(chunk0 - m0 * per_row) + threadIdx.x;
    W v[DQ_CHUNKS];
    int64_t m[DQ_CHUNKS];
    uint32_t place[DQ_CHUNKS];   // the row's last elements where a chunk would reach past them
    float s[DQ_CHUNKS];
#pragma unroll
    for (int c = 0; c < DQ_CHUNKS; ++c) {
        const uint32_t i = rest + c * DQ_NT, r = i / (uint32_t)per_row;
        m[c] = m0 + r < a.M ? m0 + r : a.M;
        const int64_t row = m[c] < a.M ? m[c] : a.M - 1;
        s[c] = a.S[row];
        const int8_t* q = a.Q + row * a.ldq;
        if (a.K >= N) {
            place[c] = Raw<T>::template place_of<false>((int)(i - r * (uint32_t)per_row) * N, a.K);
            v[c] = *(const Wu*)(q + place[c]);
        } else {
            place[c] = 0;
#pragma unroll
            for (int j = 0; j < N / 4; ++j) v[c][j] = 0;
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (e < a.K) v[c][e / 4] |= (q[e] & 255) << (8 * (e % 4));
        }
    }
#pragma unroll
    for (int c = 0; c < DQ_CHUNKS; ++c) {
        Raw<T> y;
#pragma unroll
        for (int e = 0; e < N; ++e) y.v[e] = (T)as_f32((float)(int8_t)(v[c][e / 4] >> (8 * (e % 4))) * s[c]);
        if (m[c] >= a.M) continue;
        T* x = (T*)a.X + m[c] * a.ldx;
        if (a.K >= N)
            y.template store<false>(x, place[c], a.K);
        else
            y.template store<true>(x, 0, a.K);
    }
}

static int64_t dequantize_wgs(const DequantArgs& a, int64_t per_row) {
    return (a.M * per_row + DQ_NT * DQ_CHUNKS - 1) / (DQ_NT * DQ_CHUNKS);
}

int check_i8_dequantize(const DequantArgs& a) {
    return dequantize_wgs(a, (a.K + 3) / 4) <= max_workgroups(DQ_NT) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

template <class T, NormMode MODE, int LANES, int C, bool SHORT = false>
static hipError_t launch_rows(const NormArgs& a, hipStream_t s) {
    constexpr int NT = LANES < 256 ? 256 : LANES, RPW = NT / LANES;
    // Eight waves a SIMD at most, whatever the rows: each workgroup keeps W for several.
    const int64_t wgs = (a.M + RPW - 1) / RPW, most = 256 * 2048 / NT;
    hipLaunchKernelGGL((k_norm<T, MODE, LANES, C, SHORT>), dim3((unsigned)(wgs < most ? wgs : most)), dim3(NT), 0, s, a);
    return hipGetLastError();
}
template <NormMode MODE>
static hipError_t launch(int dtype, const NormArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        constexpr int N = Raw<T>::N;
        const int chunks = (a.K + N - 1) / N;
        // Lanes by the row's chunks. Up to a workgroup a compute unit, long rows get more lanes, for the
        // shorter way (with a residual, 16 x 8192 bf16 2.8 us on 1024 lanes and 3.2 on 256, to 8 bits 4.3 and 5.0);
        // beyond, fewer, so that a unit holds several rows (on 512 lanes and on 1024: 300 x 8192 FP32 9.5 and 10.5,
        // 4096 x 16384 bf16 to 8 bits 93 and 102; 8192 x 8192 FP32 level, 64 and 63 without the norm).
        const bool few = a.M <= 256;
        if (a.K > 0 && a.K < N) return launch_rows<T, MODE, 16, 1, true>(a, s);
        if (a.K > 0 && chunks <= 16) return launch_rows<T, MODE, 16, 1>(a, s);
        if (a.K > 0 && chunks <= 32) return launch_rows<T, MODE, 16, 2>(a, s);
        if (a.K > 0 && chunks <= 64) return launch_rows<T, MODE, 64, 1>(a, s);
        if (a.K > 0 && chunks <= 128) return launch_rows<T, MODE, 64, 2>(a, s);
        if (a.K > 0 && chunks <= 256) return launch_rows<T, MODE, 64, 4>(a, s);
        if (a.K > 0 && chunks <= 512) return launch_rows<T, MODE, 256, 2>(a, s);
        if (a.K > 0 && chunks <= 1024) return few ? launch_rows<T, MODE, 1024, 1>(a, s) : launch_rows<T, MODE, 256, 4>(a, s);
        if (a.K > 0 && chunks <= 2048) return few ? launch_rows<T, MODE, 1024, 2>(a, s) : launch_rows<T, MODE, 512, 4>(a, s);
        if (a.K > 0 && chunks <= 4096) return launch_rows<T, MODE, 1024, 4>(a, s);
        hipLaunchKernelGGL((k_norm_long<T, MODE>), dim3((unsigned)(a.M < (1 << 20) ? a.M : 1 << 20)), dim3(LONG_NT),
                           0, s, a);
        return hipGetLastError();
    });
}
hipError_t launch_norm(int dtype, const NormArgs& a, hipStream_t s) { return launch<NORM_Y>(dtype, a, s); }
hipError_t launch_norm_i8(int dtype, const NormArgs& a, hipStream_t s) { return launch<NORM_Q>(dtype, a, s); }
hipError_t launch_i8_quantize(int dtype, const NormArgs& a, hipStream_t s) { return launch<PACK_Q>(dtype, a, s); }

hipError_t launch_i8_dequantize(int dtype, const DequantArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        const int per_row = (a.K + Raw<T>::N - 1) / Raw<T>::N;
        hipLaunchKernelGGL((k_i8_dequantize<T>), dim3((unsigned)dequantize_wgs(a, per_row)), dim3(DQ_NT), 0, s, a,
                           per_row);
        return hipGetLastError();
    });
}

}  // namespace sgemm

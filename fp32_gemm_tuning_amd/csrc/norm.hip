// Root-mean-square norm of rows, after the residual is added: to the type, or to 8
// bits; matrices to 8 bits and back.
#include "norm_core.hpp"

namespace sgemm {

enum NormMode { NORM_Y, NORM_Q, PACK_Q };

// Rows of any length: a workgroup a row, which is read again for every pass (from the sum H
// where that was written: X may be the same memory).
constexpr int LONG_NT = 1024;
template <class T, NormMode MODE>
__global__ __launch_bounds__(LONG_NT) void k_norm_long(NormArgs a) {
    constexpr int N = Chunk<T>::N, STEP = LONG_NT * N;
    __shared__ double red[LONG_NT / 64];
    const int first = threadIdx.x * N;
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        const T* x = (const T*)a.X + m * a.ldx;
        const T* r = MODE != PACK_Q && a.R != nullptr ? (const T*)a.R + m * a.ldr : nullptr;
        T* h = MODE != PACK_Q && a.H != nullptr ? (T*)a.H + m * a.ldh : nullptr;
        const T* w = (const T*)a.W;
        bool kept = false;   // H holds the sums
        // The sum of the residual stream, rounded to the type, as FP32.
        auto sum = [&](int at, Chunk<T>& c) {
            if (kept) {
                c.load(h, at, a.K);
                return;
            }
            c.load(x, at, a.K);
            if (r != nullptr) {
                Chunk<T> d;
                d.load(r, at, a.K);
#pragma unroll
                for (int e = 0; e < N; ++e) c.v[e] = (float)(T)(c.v[e] + d.v[e]);
            }
        };
        float rstd = 1.0f;
        if constexpr (MODE != PACK_Q) {
            float ss = 0.0f;
            for (int at = first; at < a.K; at += STEP) {
                Chunk<T> c;
                sum(at, c);
                if (h != nullptr) c.store(h, at, a.K);
#pragma unroll
                for (int e = 0; e < N; ++e) ss = __builtin_fmaf(c.v[e], c.v[e], ss);
            }
            kept = h != nullptr;
            ss = over_row<LONG_NT>(ss, Plus{}, (float*)red);
            rstd = rstd_of(ss, a.K, a.eps);
            if (sum_lost(ss)) {
                uint32_t top = 0;
                for (int at = first; at < a.K; at += STEP) {
                    Chunk<T> c;
                    sum(at, c);
#pragma unroll
                    for (int e = 0; e < N; ++e) top = Max{}(top, __builtin_bit_cast(uint32_t, fabsf(c.v[e])));
                }
                top = over_row<LONG_NT>(top, Max{}, (uint32_t*)red);
                if (top > 0 && top < 0x7F800000u) {
                    const int shift = __builtin_amdgcn_frexp_expf(__builtin_bit_cast(float, top));
                    ss = 0.0f;
                    for (int at = first; at < a.K; at += STEP) {
                        Chunk<T> c;
                        sum(at, c);
#pragma unroll
                        for (int e = 0; e < N; ++e) {
                            const float s = __builtin_amdgcn_ldexpf(c.v[e], -shift);
                            ss = __builtin_fmaf(s, s, ss);
                        }
                    }
                    ss = over_row<LONG_NT>(ss, Plus{}, (float*)red);
                    rstd = rstd_scaled(ss, shift, a.K, a.eps);
                }
            }
            if (a.rstd != nullptr && threadIdx.x == 0) a.rstd[m] = rstd;
        }
        if constexpr (MODE == NORM_Y) {
            T* y = (T*)a.Y + m * a.ldy;
            for (int at = first; at < a.K; at += STEP) {
                Chunk<T> c, g;
                sum(at, c);
                g.load(w, at, a.K);
#pragma unroll
                for (int e = 0; e < N; ++e) c.v[e] = c.v[e] * rstd * g.v[e];
                c.store(y, at, a.K);
            }
        } else {
            // What is brought to 8 bits, in 64 bits: H W exactly, or X.
            auto value = [&](int at, double (&v)[N]) {
                Chunk<T> c, g;
                sum(at, c);
                if constexpr (MODE == NORM_Q) g.load(w, at, a.K);
#pragma unroll
                for (int e = 0; e < N; ++e) v[e] = MODE == NORM_Q ? (double)c.v[e] * (double)g.v[e] : (double)c.v[e];
            };
            double top = 0.0, bad = 0.0;
            for (int at = first; at < a.K; at += STEP) {
                double v[N];
                value(at, v);
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    top = fmax(top, fabs(v[e]));
                    bad = __builtin_fma(v[e], 0.0, bad);   // 0, or NaN of an infinity or NaN
                }
            }
            top = over_row<LONG_NT>(top, Max{}, red);
            bad = over_row<LONG_NT>(bad, Plus{}, red);
            const bool flat = !(bad == 0.0) || top == 0.0;
            if (threadIdx.x == 0)
                a.S[m] = bad == 0.0 ? (a.K > 0 ? (float)(top * (double)rstd / 127.0) : 0.0f) : __builtin_nanf("");
            const double inv = flat ? 0.0 : 127.0 / top;
            int8_t* q = a.Q + m * a.ldq;
            for (int at = first; at < a.K; at += STEP) {
                double v[N];
                int n[N];
                value(at, v);
#pragma unroll
                for (int e = 0; e < N; ++e) n[e] = flat ? 0 : level(v[e], inv, top);
                store_levels(q, at, a.K, n);
            }
        }
    }
}

// Values of matrices in 8 bits: 16 a thread.
template <class T>
__global__ __launch_bounds__(256) void k_i8_dequantize(DequantArgs a) {
    const int chunks = (a.K + 15) / 16;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, m = i / chunks;
    if (m >= a.M) return;
    const int at = (int)(i - m * chunks) * 16;
    const int8_t* q = a.Q + m * a.ldq + at;
    const float s = a.S[m];
    T* x = (T*)a.X + m * a.ldx;
    constexpr int N = Chunk<T>::N;
    int8_t v[16];
    if (at + 16 <= a.K) {
        __builtin_memcpy(v, q, 16);
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = at + e < a.K ? q[e] : 0;
    }
#pragma unroll
    for (int i0 = 0; i0 < 16; i0 += N) {
        Chunk<T> c;
#pragma unroll
        for (int e = 0; e < N; ++e) c.v[e] = (float)v[i0 + e] * s;
        c.store(x, at + i0, a.K);
    }
}

static int64_t dequantize_wgs(const DequantArgs& a) { return ((int64_t)a.M * ((a.K + 15) / 16) + 255) / 256; }

int check_i8_dequantize(const DequantArgs& a) {
    return dequantize_wgs(a) <= max_workgroups(256) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

template <NormMode MODE>
static hipError_t launch(int dtype, const NormArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        hipLaunchKernelGGL((k_norm_long<T, MODE>), dim3((unsigned)(a.M < (1 << 20) ? a.M : 1 << 20)), dim3(LONG_NT), 0, s, a);
        return hipGetLastError();
    });
}
hipError_t launch_norm(int dtype, const NormArgs& a, hipStream_t s) { return launch<NORM_Y>(dtype, a, s); }
hipError_t launch_norm_i8(int dtype, const NormArgs& a, hipStream_t s) { return launch<NORM_Q>(dtype, a, s); }
hipError_t launch_i8_quantize(int dtype, const NormArgs& a, hipStream_t s) { return launch<PACK_Q>(dtype, a, s); }

hipError_t launch_i8_dequantize(int dtype, const DequantArgs& a, hipStream_t s) {
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        hipLaunchKernelGGL((k_i8_dequantize<T>), dim3((unsigned)dequantize_wgs(a)), dim3(256), 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace sgemm

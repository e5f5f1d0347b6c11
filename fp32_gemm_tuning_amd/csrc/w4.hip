// Products with 4-bit weights: Y = X W^T (w4) and the gated block over two
// such weights (w4_glu).
//
// A stored number q becomes a 16-bit float without a conversion: the four bits
// go to the top of the mantissa of 16, which reads 16 + q exactly (bfloat16
// 0x4180 + (q << 3), half 0x4C00 + (q << 6)); one shift and one and-or make two of
// them. The matrix cores then sum (16 + q) x in FP32 over 32 k at a time, a
// further product with ones sums x, and for each group
//     sum (q - z) s x = s (sum (16 + q) x - (16 + z) sum x)
// is added to the result: the scale and zero point cost two multiply-adds per
// output and group, not one per weight. FP32 activations are split into three
// bfloat16 parts that add up to them exactly (8 + 8 + 8 bits), so each
// product is exact in every type.
#include "ffn.hpp"

namespace sgemm {

static inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_u1 __attribute__((aligned(1)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// What a type's activations are multiplied as.
template <class T>
struct W4Type {   // float: three bfloat16 parts
    static constexpr int PARTS = 3;
    static constexpr uint32_t MASK = 0x00780078u, BASE = 0x41804180u, ONES = 0x3F803F80u;
    static constexpr int SHIFT = 3;
    __device__ __forceinline__ static f32x4 mma(const i32x4& a, const i32x4& b, const f32x4& c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    }
};
template <>
struct W4Type<bf16> : W4Type<float> {
    static constexpr int PARTS = 1;
};
template <>
struct W4Type<f16> {
    static constexpr int PARTS = 1;
    static constexpr uint32_t MASK = 0x03C003C0u, BASE = 0x4C004C00u, ONES = 0x3C003C00u;
    static constexpr int SHIFT = 6;
    __device__ __forceinline__ static f32x4 mma(const i32x4& a, const i32x4& b, const f32x4& c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                      __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    }
};

// Eight stored numbers to eight 16 + q. Pair e of the result holds numbers e
// and e + 4, so the activations are paired the same way (pair_up).
template <class T>
__device__ __forceinline__ i32x4 unpack(uint32_t w) {
    using C = W4Type<T>;
    i32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int left = C::SHIFT - 4 * e;
        r[e] = (int)(((left >= 0 ? w << left : w >> -left) & C::MASK) | C::BASE);
    }
    return r;
}

// Eight consecutive activations of a row, as loaded.
template <class T>
struct XRaw {
    i32x4 v[sizeof(T) / 2];
    // `left` elements of the row remain at p; those past them are zero.
    __device__ __forceinline__ void load(const T* p, int left) {
        typedef i32x4 V __attribute__((aligned(2)));
        if (left >= 8) {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = ((const V*)p)[i];
        } else {
            constexpr int EPV = 16 / sizeof(T);
            typedef T E __attribute__((ext_vector_type(EPV)));
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                E x = __builtin_bit_cast(E, i32x4{0, 0, 0, 0});
#pragma unroll
                for (int e = 0; e < EPV; ++e)
                    if (i * EPV + e < left) x[e] = p[i * EPV + e];
                v[i] = __builtin_bit_cast(i32x4, x);
            }
        }
    }
};

// Halves of two words: the low or the high ones, a's first.
__device__ __forceinline__ int lows(int a, int b) {
    return (int)__builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x05040100u);
}
__device__ __forceinline__ int highs(int a, int b) {
    return (int)__builtin_amdgcn_perm((uint32_t)b, (uint32_t)a, 0x07060302u);
}

template <class T>
__device__ __forceinline__ void pair_up(const XRaw<T>& x, i32x4 (&p)[1]) {
    p[0] = i32x4{lows(x.v[0].x, x.v[0].z), highs(x.v[0].x, x.v[0].z), lows(x.v[0].y, x.v[0].w),
                 highs(x.v[0].y, x.v[0].w)};
}
// FP32: x = hi + mid + lo, each the leading 8 bits of what the ones before left
// (truncated, so every difference is exact and lo is what remains of 24 bits).
__device__ __forceinline__ void pair_up(const XRaw<float>& x, i32x4 (&p)[3]) {
    const f32x4 a = __builtin_bit_cast(f32x4, x.v[0]), b = __builtin_bit_cast(f32x4, x.v[1]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float r[2] = {a[e], b[e]};
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            p[i][e] = highs(__builtin_bit_cast(int, r[0]), __builtin_bit_cast(int, r[1]));
#pragma unroll
            for (int h = 0; h < 2; ++h)
                r[h] -= __builtin_bit_cast(float, __builtin_bit_cast(int, r[h]) & (int)0xFFFF0000);
        }
    }
}

// The 4 x 4 transpose between a lane's four words and the four quarters of
// the wave: word j of quarter q and word q of quarter j change places.
__device__ __forceinline__ void transpose4(i32x4& d) {
    const auto a = __builtin_amdgcn_permlane32_swap(d.x, d.z, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(d.y, d.w, false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d = i32x4{(int)c[0], (int)c[1], (int)e[0], (int)e[1]};
}

// Groups along k, in steps of 32: `steps` to a group (`shift` its logarithm, or
// -1), and `per` steps of a block of four between two uses of the scales.
struct W4Groups {
    int steps, shift, per;
};

// A workgroup takes 16 MB rows of X and 16 NB output features; its NW waves take
// blocks of 128 k in turn and their sums are added in wave order at the end.
// Per block a lane loads 16 bytes (32 numbers) of row lane % 16 of each 16
// features, so a row's four lanes read 64 contiguous bytes; the transpose then
// gives step j of the block the numbers k = 32 j + 8 (lane / 16) + 0..7, which is
// the operand layout of the 16x16x32 matrix instruction, and any group of
// whole steps can be scaled apart. X's operands come straight from memory
// (the cache holds them: X is small beside the weights).
template <class T, bool DUAL, int MB, int NB, int NW>
__global__ __launch_bounds__(NW * 64) void k_w4(W4Args a, W4Groups gr) {
    using C = W4Type<T>;
    constexpr int D = DUAL ? 2 : 1;
    __shared__ float red[NW][D][MB][4][68];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int q = lane >> 4, c = lane & 15;
    const int f0 = blockIdx.x * (16 * NB), m0 = blockIdx.y * (16 * MB);
    const int bytes = (a.K + 1) / 2;
    const int nblk = (a.K + 127) / 128;

    // Rows past the last one repeat it; their results are not stored.
    const T* xrow[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
        const int m = m0 + 16 * i + c;
        xrow[i] = (const T*)a.X + (int64_t)(m < a.M ? m : a.M - 1) * a.ldx;
    }
    const uint8_t* wrow[D][NB];
    const T* srow[D][NB];
    const T* zrow[D][NB];
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int n = 0; n < NB; ++n) {
            const int f = f0 + 16 * n + c;
            const int64_t r = f < a.F ? f : a.F - 1;
            wrow[d][n] = a.Q[d] + r * a.ldq;
            srow[d][n] = (const T*)a.S[d] + r * a.lds;
            zrow[d][n] = (const T*)a.Z[d] + r * a.ldz;
        }
    const bool zeros = a.Z[0] != nullptr;

    struct Blk {
        i32x4 w[D][NB];
        T s[D][NB][4], z[D][NB][4];
    };
    auto load = [&](int b, Blk& r) {
        const int at = 64 * b + 16 * q;
        const bool whole = 64 * b + 64 <= bytes;
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                const uint8_t* p = wrow[d][n] + at;
                if (whole) {
                    r.w[d][n] = *(const i32x4_u1*)p;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t v = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (at + 4 * j + i < bytes) v |= (uint32_t)p[4 * j + i] << (8 * i);
                        r.w[d][n][j] = (int)v;
                    }
                }
            }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if ((j & (gr.per - 1)) == 0 && 128 * b + 32 * j < a.K) {
                const int st = 4 * b + j;
                const int g = gr.shift >= 0 ? st >> gr.shift : st / gr.steps;
#pragma unroll
                for (int d = 0; d < D; ++d)
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        r.s[d][n][j] = srow[d][n][g];
                        if (zeros) r.z[d][n][j] = zrow[d][n][g];
                    }
            }
    };

    float sc[D][NB], zc[D][NB];   // the running group's scale and 16 + zero point
    f32x4 acc[D][MB][NB], part[D][MB][NB], sx[MB];
    const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int n = 0; n < NB; ++n) acc[d][i][n] = none;

    auto compute = [&](int b, Blk& r) {
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int n = 0; n < NB; ++n) transpose4(r.w[d][n]);
        const i32x4 ones = {(int)C::ONES, (int)C::ONES, (int)C::ONES, (int)C::ONES};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = 128 * b + 32 * j;
            if (k >= a.K) break;
            XRaw<T> x[MB];
#pragma unroll
            for (int i = 0; i < MB; ++i) x[i].load(xrow[i] + k + 8 * q, a.K - k - 8 * q);
            const bool first = (j & (gr.per - 1)) == 0;
            if (first) {
#pragma unroll
                for (int i = 0; i < MB; ++i) {
                    sx[i] = none;
#pragma unroll
                    for (int d = 0; d < D; ++d)
#pragma unroll
                        for (int n = 0; n < NB; ++n) part[d][i][n] = none;
                }
#pragma unroll
                for (int d = 0; d < D; ++d)
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        sc[d][n] = (float)r.s[d][n][j];
                        zc[d][n] = 16.0f + (zeros ? (float)r.z[d][n][j] : 8.0f);
                    }
            }
            i32x4 u[D][NB];
#pragma unroll
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int n = 0; n < NB; ++n) u[d][n] = unpack<T>((uint32_t)r.w[d][n][j]);
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                i32x4 p[C::PARTS];
                pair_up(x[i], p);
#pragma unroll
                for (int e = 0; e < C::PARTS; ++e) {
                    sx[i] = C::mma(p[e], ones, sx[i]);
#pragma unroll
                    for (int d = 0; d < D; ++d)
#pragma unroll
                        for (int n = 0; n < NB; ++n) part[d][i][n] = C::mma(p[e], u[d][n], part[d][i][n]);
                }
            }
            const bool last = ((j + 1) & (gr.per - 1)) == 0 || k + 32 >= a.K;
            if (last) {
#pragma unroll
                for (int d = 0; d < D; ++d)
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const float s = sc[d][n], z = zc[d][n];
#pragma unroll
                        for (int i = 0; i < MB; ++i)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                acc[d][i][n][e] =
                                    __builtin_fmaf(s, __builtin_fmaf(-z, sx[i][e], part[d][i][n][e]), acc[d][i][n][e]);
                    }
            }
        }
    };

    // This wave's blocks, two in flight: each next block's loads go out before
    // the current one's products.
    if (w < nblk) {
        Blk r0, r1;
        load(w, r0);
        for (int b = w; b < nblk; b += 2 * NW) {
            if (b + NW < nblk) load(b + NW, r1);
            __builtin_amdgcn_sched_barrier(0);
            compute(b, r0);
            __builtin_amdgcn_sched_barrier(0);
            if (b + 2 * NW < nblk) load(b + 2 * NW, r0);
            __builtin_amdgcn_sched_barrier(0);
            if (b + NW < nblk) compute(b + NW, r1);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    // Sums over the waves in their order, one block of 16 features at a time.
#pragma unroll
    for (int n = 0; n < NB; ++n) {
        if (n > 0) __syncthreads();
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int i = 0; i < MB; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) red[w][d][i][e][lane] = acc[d][i][n][e];
        __syncthreads();
        for (int o = threadIdx.x; o < MB * 256; o += NW * 64) {
            const int i = o >> 8, row = (o >> 4) & 15, col = o & 15;
            float v[2] = {0.0f, 0.0f};
#pragma unroll
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int ww = 0; ww < NW; ++ww) v[d] += red[ww][d][i][row & 3][(row >> 2) * 16 + col];
            const int m = m0 + 16 * i + row, f = f0 + 16 * n + col;
            if (m < a.M && f < a.F)
                ((T*)a.Y)[(int64_t)m * a.ldy + f] = (T)(DUAL ? act_value(a.act, v[0]) * v[1] : v[0]);
        }
    }
}

int check_w4(const W4Args& a, bool) {
    return cdiv(a.M, 16) <= 65535 && cdiv(a.F, 16) <= max_workgroups(1024) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

template <class T, bool DUAL, int MB, int NB, int NW>
static hipError_t launch(const W4Args& a, const W4Groups& gr, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(a.F, 16 * NB), (unsigned)cdiv(a.M, 16 * MB));
    hipLaunchKernelGGL((k_w4<T, DUAL, MB, NB, NW>), grid, dim3(NW * 64), 0, s, a, gr);
    return hipGetLastError();
}

hipError_t launch_w4(int dtype, const W4Args& a, bool dual, hipStream_t s) {
    W4Groups gr = {a.group / 32, -1, 1};
    if ((gr.steps & (gr.steps - 1)) == 0) gr.shift = __builtin_ctz(gr.steps);
    gr.per = gr.steps % 4 == 0 ? 4 : gr.steps % 2 == 0 ? 2 : 1;
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        if (a.M <= 16) {
            if (dual) return launch<T, true, 1, 1, 8>(a, gr, s);
            return launch<T, false, 1, 1, 8>(a, gr, s);
        }
        if (dual) return launch<T, true, 4, 1, 8>(a, gr, s);
        return launch<T, false, 4, 2, 8>(a, gr, s);
    });
}

}  // namespace sgemm

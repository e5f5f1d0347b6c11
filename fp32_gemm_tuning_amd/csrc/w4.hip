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
#include "mfma_pipecore.hpp"   // ring_barrier

namespace sgemm {

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
// The two constants come from registers the compiler cannot see through: one
// and-or instruction takes a scalar and a vector register, not two literals.
template <class T>
struct Unpack {
    uint32_t mask = W4Type<T>::MASK, base = W4Type<T>::BASE;
    __device__ __forceinline__ Unpack() { asm("" : "+s"(mask), "+v"(base)); }
    __device__ __forceinline__ i32x4 operator()(uint32_t w) const {
        i32x4 r;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int left = W4Type<T>::SHIFT - 4 * e;
            r[e] = (int)(((left >= 0 ? w << left : w >> -left) & mask) | base);
        }
        return r;
    }
};

// Eight consecutive activations of a row, as loaded.
template <class T>
struct XRaw {
    i32x4 v[sizeof(T) / 2];
    // Elements at .. at + 7 of a row of n >= 8 elements: fetch reads the last 8
    // where these would reach past the row's end, and place moves them down, zeros
    // behind. Apart, and without branches in fetch, so that many loads are in
    // flight: a value that a branch may set otherwise is waited for there.
    __device__ __forceinline__ void fetch(const T* row, int at, int n) {
        typedef i32x4 V __attribute__((aligned(2)));
        const T* p = row + (at < n - 8 ? at : n - 8);
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = ((const V*)p)[i];
    }
    __device__ __forceinline__ void place(int at, int n) {
        const int past = at - (n - 8);
        if constexpr (sizeof(T) == 2) {
            const unsigned __int128 x = __builtin_bit_cast(unsigned __int128, v[0]);
            v[0] = __builtin_bit_cast(i32x4, past >= 8 ? (unsigned __int128)0 : x >> (past > 0 ? 16 * past : 0));
        } else {
            const bool by4 = past & 4, by2 = past & 2, by1 = past & 1;
            int x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
            if (past >= 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0;
            } else if (past > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = by4 ? (e < 4 ? x[e + 4] : 0) : x[e];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = by2 ? (e < 6 ? x[e + 2] : 0) : x[e];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = by1 ? (e < 7 ? x[e + 1] : 0) : x[e];
            }
            v[0] = i32x4{x[0], x[1], x[2], x[3]};
            v[1] = i32x4{x[4], x[5], x[6], x[7]};
        }
    }
    // The same of a row of any length, element by element.
    __device__ __forceinline__ void fetch_short(const T* row, int at, int n) {
        constexpr int EPV = 16 / sizeof(T);
        typedef T E __attribute__((ext_vector_type(EPV)));
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
            E x;
#pragma unroll
            for (int e = 0; e < EPV; ++e) {
                const int k = at + i * EPV + e;
                const T y = row[k < n ? k : n - 1];
                x[e] = k < n ? y : (T)0.0f;
            }
            v[i] = __builtin_bit_cast(i32x4, x);
        }
    }
};

// 16 bytes (32 numbers) of a row of at least 16 bytes, from byte `at`: load_w32
// reads the last 16 where these would reach past the row's end, and place_w32
// shifts them down. (Numbers past the row's end meet activations that are
// zero.) Apart, so that many loads are in flight: a load whose value is used
// in a branch is waited for there.
__device__ __forceinline__ i32x4 load_w32(const uint8_t* row, int at, int bytes) {
    return *(const i32x4_u1*)(row + (at < bytes - 16 ? at : bytes - 16));
}
__device__ __forceinline__ i32x4 place_w32(const i32x4& v, int at, int bytes) {
    const int past = at - (bytes - 16);
    const unsigned __int128 x = __builtin_bit_cast(unsigned __int128, v);
    return __builtin_bit_cast(i32x4, x >> (past <= 0 ? 0 : past < 16 ? 8 * past : 120));
}

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

// Groups along k, in steps of 32: `steps` to a group, `shift` its logarithm or
// -1.
struct W4Groups {
    int steps, shift;
    __device__ __forceinline__ int of(int step) const { return shift >= 0 ? step >> shift : step / steps; }
};

// ---------------------------------------------------------------------------
// Few rows of X: vector units.
//
// A lane owns 32 consecutive k of every weight row, one 16-byte load, so a wave
// reads a row's 1 KiB in one piece, and a group's scale one element per lane, next
// to its neighbours'. The lane's activations stay in registers while it walks the
// rows. All of a wave's loads go out before its first product: with a
// launch that fills the chip once there is no loop to overlap them in. Bound
// by the weights' bytes and, close behind, by issue: about 60 vector
// instructions a lane for 32 weights. 8192 x 8192 from HBM, one row: bf16
// 10.5 us (3.3 TB/s, launch included), FP32 14.4; two rows bf16 13.2.
// ---------------------------------------------------------------------------
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float dot2(bf16, int a, int b, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, a), __builtin_bit_cast(bf16x2, b), c, false);
}
__device__ __forceinline__ float dot2(f16, int a, int b, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, a), __builtin_bit_cast(f16x2, b), c, false);
}

// A lane's 32 activations of one row and their sum.
template <class T>
struct LaneX {
    i32x4 p[4];   // paired as the numbers unpack
    float sum;
    __device__ __forceinline__ void set(const XRaw<T> (&r)[4]) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            i32x4 one[1];
            pair_up(r[j], one);
            p[j] = one[0];
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = dot2(T{}, p[j][e], (int)W4Type<T>::ONES, sum);
        }
    }
    // sum (16 + q) x, less 16 sum x with the zero point's part.
    __device__ __forceinline__ float times(const Unpack<T>& unpack, const i32x4& w, float z) const {
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const i32x4 u = unpack((uint32_t)w[j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e & 1] = dot2(T{}, p[j][e], u[e], v[e & 1]);
        }
        return __builtin_fmaf(-(16.0f + z), sum, v[0] + v[1]);
    }
};
template <>
struct LaneX<float> {
    float x[32];
    float sum;
    __device__ __forceinline__ void set(const XRaw<float> (&r)[4]) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const f32x4 a = __builtin_bit_cast(f32x4, r[j].v[0]), b = __builtin_bit_cast(f32x4, r[j].v[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[8 * j + e] = a[e];
                x[8 * j + 4 + e] = b[e];
                sum += a[e] + b[e];
            }
        }
    }
    __device__ __forceinline__ float times(const Unpack<float>&, const i32x4& w, float z) const {
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                v[e & 1] = __builtin_fmaf((float)(((uint32_t)w[j] >> (4 * e)) & 15), x[8 * j + e], v[e & 1]);
        return __builtin_fmaf(-z, sum, v[0] + v[1]);
    }
};

// The sums of four values over a wave's lanes: quarter i of the result (lanes
// 16 i ..) holds the sum of value i. Two lane swaps halve four values to one,
// and a row of 16 lanes is summed by data-parallel moves (a shuffle through LDS
// for each value and step cost more than the products).
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
    const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true);
    return v + __builtin_bit_cast(float, o);
}
__device__ __forceinline__ float add_halves(float a, float b) {   // a in lanes 0-31, b in 32-63
    const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a),
                                                    __builtin_bit_cast(uint32_t, b), false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float add_rows(float a, float b) {     // a in even rows of 16, b in odd ones
    const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a),
                                                    __builtin_bit_cast(uint32_t, b), false, false);
    return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float wave_sums(float a, float b, float c, float d) {
    float v = add_rows(add_halves(a, c), add_halves(b, d));
    v = add_dpp<0xB1>(v);    // quad_perm 1,0,3,2
    v = add_dpp<0x4E>(v);    // quad_perm 2,3,0,1
    v = add_dpp<0x141>(v);   // row_half_mirror
    return add_dpp<0x140>(v);   // row_mirror
}

// kw waves share the k of a row (64 lanes of 32 each) and add up in wave
// order; blockDim.x / (64 kw) such sets take RW features each.
template <class T, bool DUAL, int MR, bool RAGGED>
__global__ __launch_bounds__(512) void k_w4_few(W4Args a, W4Groups gr, int kw) {
    constexpr int D = DUAL ? 2 : 1, RW = DUAL ? 4 : 8;
    constexpr int N = D * RW * MR;   // sums per wave, value (d, r, m) at (d * RW + r) * MR + m
    __shared__ float red[8][N];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int set = w / kw, kp = w - set * kw, sets = (blockDim.x >> 6) / kw;
    const int f0 = (blockIdx.x * sets + set) * RW;
    const int bytes = (a.K + 1) / 2;
    const bool zeros = a.Z[0] != nullptr;
    const Unpack<T> unpack;
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;

    for (int kb = kp * 2048; kb < a.K; kb += kw * 2048) {
        const int k = kb + lane * 32, at = k >> 1;
        const int step = k >> 5, last = (a.K - 1) >> 5;
        const int g = gr.of(step < last ? step : last);
        XRaw<T> x[MR][4];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            const T* row = (const T*)a.X + (int64_t)(m < a.M ? m : a.M - 1) * a.ldx;
#pragma unroll
            for (int j = 0; j < 4; ++j) x[m][j].fetch(row, k + 8 * j, a.K);
        }
        // Row by row, so that the first rows' products run while the last ones'
        // weights arrive. Without zero points the scale is read twice and the
        // second value ignored (a load on some paths only would be waited
        // for with all before it).
        i32x4 q[D][RW];
        T s[D][RW], z[D][RW];
#pragma unroll
        for (int r = 0; r < RW; ++r) {
            const int64_t f = f0 + r < a.F ? f0 + r : a.F - 1;
#pragma unroll
            for (int d = 0; d < D; ++d) {
                q[d][r] = load_w32(a.Q[d] + f * a.ldq, at, bytes);
                s[d][r] = ((const T*)a.S[d])[f * a.lds + g];
                z[d][r] = ((const T*)(zeros ? a.Z[d] : a.S[d]))[f * (zeros ? a.ldz : a.lds) + g];
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        LaneX<T> lx[MR];
#pragma unroll
        for (int m = 0; m < MR; ++m) {
#pragma unroll
            for (int j = 0; j < 4; ++j) x[m][j].place(k + 8 * j, a.K);
            lx[m].set(x[m]);
        }
#pragma unroll
        for (int r = 0; r < RW; ++r) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                const i32x4 w32 = RAGGED ? place_w32(q[d][r], at, bytes) : q[d][r];
                const float zp = zeros ? (float)z[d][r] : 8.0f;
#pragma unroll
                for (int m = 0; m < MR; ++m) {
                    float& o = acc[(d * RW + r) * MR + m];
                    o = __builtin_fmaf((float)s[d][r], lx[m].times(unpack, w32, zp), o);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float v = wave_sums(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        if ((lane & 15) == 0) red[w][i + (lane >> 4)] = v;
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < sets * RW * MR) {
        const int m = t % MR, r = (t / MR) % RW, st = t / (MR * RW);
        const int f = (blockIdx.x * sets + st) * RW + r;
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int d = 0; d < D; ++d)
            for (int i = 0; i < kw; ++i) v[d] += red[st * kw + i][(d * RW + r) * MR + m];
        if (m < a.M && f < a.F)
            ((T*)a.Y)[(int64_t)m * a.ldy + f] = (T)(DUAL ? act_value<sizeof(T) == 4>(a.act, v[0]) * v[1] : v[0]);
    }
}

template <class T, bool DUAL, int MR>
static hipError_t launch_few(const W4Args& a, const W4Groups& gr, hipStream_t s) {
    const int64_t need = cdiv(a.K, 2048);
    const int kw = need < 1 ? 1 : need > 8 ? 8 : (int)need;
    const int sets = kw >= 4 ? 1 : 4 / kw;
    const dim3 grid((unsigned)cdiv(a.F, sets * (DUAL ? 4 : 8)));
    if (a.K % 32 != 0)
        hipLaunchKernelGGL((k_w4_few<T, DUAL, MR, true>), grid, dim3(64 * kw * sets), 0, s, a, gr, kw);
    else
        hipLaunchKernelGGL((k_w4_few<T, DUAL, MR, false>), grid, dim3(64 * kw * sets), 0, s, a, gr, kw);
    return hipGetLastError();
}

// ---------------------------------------------------------------------------
// More rows: matrix cores.
//
// A workgroup's NW waves are STREAMS streams of 16 NB weight rows (at the least 32
// features, or the two matrices' rows of 16 features) by NW / STREAMS runs of 128 k,
// which one pass of its loop covers. X's part of a pass is staged in LDS once for all streams,
// already paired (and split, for FP32), as 16-byte units [part][k / 8][row],
// the operand of lane (k / 8 % 4, row) of the 16x16x32 matrix instruction.
// Memory is read along the rows, consecutive lanes on consecutive 16 bytes, and
// rearranged through LDS: read in operand order, where neighbouring
// lanes take different rows, each load instruction touched 16 lines and took
// four times as long. A weight row's words reach their step's lanes by a 4 x 4
// transpose between words and quarters of the wave, which puts 32
// consecutive k in each step, so any group of whole steps is scaled apart: PER
// steps of a run share their scales. Bound by issue: unpacking, and for FP32
// splitting X, on eight or sixteen waves a compute unit; with many rows by the loads
// of X, once for each workgroup's features, and their staging. 8192 x 8192 from
// HBM: 16 rows bf16 16.2 us, FP32 (groups of 64, zero points) 28; 64 rows bf16 35, FP32
// 54; 256 rows 71 and 162.
// ---------------------------------------------------------------------------

// The 4 x 4 transpose between a lane's four words and the four quarters of
// the wave: word j of quarter q and word q of quarter j change places.
__device__ __forceinline__ void transpose4(i32x4& d) {
    const auto a = __builtin_amdgcn_permlane32_swap(d.x, d.z, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(d.y, d.w, false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d = i32x4{(int)c[0], (int)c[1], (int)e[0], (int)e[1]};
}

// SHORT: K < 32, rows too short for whole loads.
template <class T, bool DUAL, int MB, int PER, int NW, int NB, int STREAMS, bool SHORT>
__global__ __launch_bounds__(NW * 64) void k_w4_rows(W4Args a, W4Groups gr) {
    using C = W4Type<T>;
    constexpr int RUNS = NW / STREAMS, PASS = 128 * RUNS, STEPS = PASS / 32;
    constexpr int ROWS = 16 * MB, UNITS = PASS / 8 * ROWS;   // 16-byte units of a part's pass
    constexpr int XI = UNITS / (NW * 64);                    // units per thread
    constexpr int WROWS = 16 * NB * STREAMS, HALF = WROWS / 2;     // weight rows; DUAL: of a matrix
    constexpr int OUTS = DUAL ? HALF : WROWS;
    // Two stages of X, or one where two do not fit: the next pass is then
    // stored behind a barrier of its own.
    constexpr int STAGES = 2 * C::PARTS * UNITS * 16 <= 128 * 1024 ? 2 : 1;
    constexpr int SUMS = NW * NB * MB * 4 * 68 / 4;   // units of the sums at the end
    __shared__ i32x4 xs[STAGES * C::PARTS * UNITS > SUMS ? STAGES * C::PARTS * UNITS : SUMS];
    __shared__ i32x4 ws[NW][64];
    __shared__ float sc[2][2][WROWS][STEPS + 1];   // [stage][scale, 16 + zero point][row][step]
    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63;
    const int q = lane >> 4, c = lane & 15;
    const int stream = w % STREAMS, run = w / STREAMS;
    const int f0 = blockIdx.x * OUTS, m0 = blockIdx.y * ROWS;
    const int bytes = (a.K + 1) / 2, passes = (a.K + PASS - 1) / PASS;
    const bool zeros = a.Z[0] != nullptr;

    // What this thread loads: its weight rows (of its stream), its scales' rows
    // and its rows of X. Rows past the last repeat it; their results are not stored.
    auto feature = [&](int r) {   // of weight row r
        const int f = DUAL ? f0 + r % HALF : f0 + r;
        return (int64_t)(f < a.F ? f : a.F - 1);
    };
    const uint8_t* wrow[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
        wrow[b] = a.Q[DUAL ? stream / (STREAMS / 2) : 0] + feature(16 * (NB * stream + b) + (lane >> 2)) * a.ldq;
    const int sr = t / STEPS, ss = t % STEPS;   // (and 16 STREAMS rows further for each b)
    const T *srow[NB], *zrow[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int r = sr + 16 * STREAMS * b, m = DUAL ? r / HALF : 0;
        srow[b] = (const T*)(m ? a.S[1] : a.S[0]) + feature(r) * a.lds;
        // (without zero points the scale is read again and ignored)
        zrow[b] = zeros ? (const T*)(m ? a.Z[1] : a.Z[0]) + feature(r) * a.ldz : srow[b];
    }
    const int last_step = (a.K - 1) >> 5;

    struct Ahead {   // one pass's weights and scales, on their way
        i32x4 w[NB];
        T s[NB], z[NB];
    };
    auto load_ahead = [&](int p, Ahead& r) {
        const int at = PASS / 2 * p + 64 * run + 16 * (lane & 3);
        const int st = STEPS * p + ss, g = gr.of(st < last_step ? st : last_step);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            if constexpr (!SHORT) {
                r.w[b] = load_w32(wrow[b], at, bytes);
            } else {
                unsigned __int128 x = 0;
                for (int i = 0; at + i < bytes; ++i) x |= (unsigned __int128)wrow[b][at + i] << (8 * i);
                r.w[b] = __builtin_bit_cast(i32x4, x);
            }
            r.s[b] = srow[b][g];
            r.z[b] = zrow[b][g];
        }
    };
    // The row and place of this thread's unit i of X (the row is one a wave where
    // a row has at least 64 units).
    constexpr int LINE = PASS / 8;
    auto x_row = [&](int i) { return LINE >= 64 ? (w + NW * i) / (LINE / 64 > 0 ? LINE / 64 : 1) : (t + NW * 64 * i) / LINE; };
    auto x_k8 = [&](int i) { return (t + NW * 64 * i) % LINE; };
    struct XPass {
        XRaw<T> r[XI];
    };
    auto load_x = [&](int p, XPass& x) {
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int m = m0 + x_row(i), k = PASS * p + 8 * x_k8(i);
            const T* row = (const T*)a.X + (int64_t)(m < a.M ? m : a.M - 1) * a.ldx;
            if constexpr (SHORT)
                x.r[i].fetch_short(row, k, a.K);
            else
                x.r[i].fetch(row, k, a.K);
        }
    };
    auto store_x = [&](int p, XPass& x) {
        i32x4* st = xs + p % STAGES * (C::PARTS * UNITS);
#pragma unroll
        for (int i = 0; i < XI; ++i) {
            const int r = x_row(i), k8 = x_k8(i);
            const int k = PASS * p + 8 * k8;
            if (!SHORT && PASS * p + PASS > a.K) x.r[i].place(k, a.K);
            i32x4 parts[C::PARTS];
            pair_up(x.r[i], parts);
#pragma unroll
            for (int e = 0; e < C::PARTS; ++e) st[e * UNITS + k8 * ROWS + (r ^ (k8 & 15))] = parts[e];
        }
    };
    auto store_scales = [&](int p, const Ahead& r) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            sc[p & 1][0][sr + 16 * STREAMS * b][ss] = (float)r.s[b];
            sc[p & 1][1][sr + 16 * STREAMS * b][ss] = 16.0f + (zeros ? (float)r.z[b] : 8.0f);
        }
    };

    const Unpack<T> unpack;
    const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
    const i32x4 ones = {(int)C::ONES, (int)C::ONES, (int)C::ONES, (int)C::ONES};
    f32x4 acc[NB][MB];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MB; ++i) acc[b][i] = none;

    auto compute = [&](int p, const Ahead& r) {
        const int k0 = PASS * p + 128 * run;
        if (k0 >= a.K) return;
        i32x4 d[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            d[b] = r.w[b];
            if (!SHORT && k0 + 128 > a.K) d[b] = place_w32(d[b], (k0 >> 1) + 16 * (lane & 3), bytes);
            // Rows to operand order: unit (row, chunk) at chunk ^ (row / 2 % 4) of
            // its row, so that both accesses spread over all banks. A wave's
            // own units only: no barrier.
            const int wl = lane >> 2;
            ws[w][wl * 4 + ((lane & 3) ^ ((wl >> 1) & 3))] = d[b];
            d[b] = ws[w][c * 4 + (q ^ ((c >> 1) & 3))];
            transpose4(d[b]);
        }
        const i32x4* st = xs + p % STAGES * (C::PARTS * UNITS);
        // FP32: the sums of X's leading parts apart from those of the others. Leading
        // parts have 8 bits and numbers 5, so their sums over a group lose almost nothing
        // before the zero point is taken off; the others' are 2^-8 of them.
        constexpr int KINDS = C::PARTS > 1 ? 2 : 1;
        f32x4 part[KINDS][NB][MB], sx[KINDS][MB];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (k0 + 32 * j >= a.K) break;
            i32x4 u[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) u[b] = unpack((uint32_t)d[b][j]);
            const int k8 = 16 * run + 4 * j + q;
#pragma unroll
            for (int i = 0; i < MB; ++i) {
                if (j % PER == 0) {
#pragma unroll
                    for (int kind = 0; kind < KINDS; ++kind) {
                        sx[kind][i] = none;
#pragma unroll
                        for (int b = 0; b < NB; ++b) part[kind][b][i] = none;
                    }
                }
#pragma unroll
                for (int e = 0; e < C::PARTS; ++e) {
                    const i32x4 x = st[e * UNITS + k8 * ROWS + ((16 * i + c) ^ (k8 & 15))];
#pragma unroll
                    for (int b = 0; b < NB; ++b) part[e > 0][b][i] = C::mma(x, u[b], part[e > 0][b][i]);
                    sx[e > 0][i] = C::mma(x, ones, sx[e > 0][i]);
                }
            }
            if ((j + 1) % PER == 0 || k0 + 32 * (j + 1) >= a.K) {
                const int at = 4 * run + j / PER * PER;
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int row = 16 * (NB * stream + b) + c;
                    const float s = sc[p & 1][0][row][at], z = sc[p & 1][1][row][at];
#pragma unroll
                    for (int i = 0; i < MB; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float v = __builtin_fmaf(-z, sx[0][i][e], part[0][b][i][e]);
                            if constexpr (KINDS == 2) v += __builtin_fmaf(-z, sx[1][i][e], part[1][b][i][e]);
                            acc[b][i][e] = __builtin_fmaf(s, v, acc[b][i][e]);
                        }
                }
            }
        }
    };

    if (passes > 0) {
        // Each register set is refilled as soon as it is used, so weights are
        // two passes ahead and X nearly two, or, where registers run out, nearly one;
        // the barrier waits for LDS only.
        constexpr bool DEEP = MB * NB < 8 || STREAMS > 2;
        Ahead r0, r1;
        XPass x0, x1;
        load_x(0, x0);
        load_ahead(0, r0);
        if constexpr (DEEP) load_x(1, x1);
        load_ahead(1, r1);
        store_x(0, x0);
        store_scales(0, r0);
        load_x(DEEP ? 2 : 1, x0);
        ring_barrier<63>();
        auto pass = [&](int p, Ahead& now, const Ahead& next, XPass& x) {
            compute(p, now);
            load_ahead(p + 2, now);
            if constexpr (STAGES == 1) ring_barrier<63>();
            store_x(p + 1, x);
            store_scales(p + 1, next);
            load_x(p + (DEEP ? 3 : 2), x);
            ring_barrier<63>();
        };
        for (int p = 0; p < passes; p += 2) {
            pass(p, r0, r1, DEEP ? x1 : x0);
            if (p + 1 < passes) pass(p + 1, r1, r0, x0);
        }
    }

    // Sums over the runs in their order, through the space of X.
    float* red = (float*)xs;
    auto slot = [](int wave, int b, int i, int e) { return (((wave * NB + b) * MB + i) * 4 + e) * 68; };
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < MB; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[slot(w, b, i, e) + lane] = acc[b][i][e];
    __syncthreads();
    for (int o = t; o < ROWS * OUTS; o += NW * 64) {
        const int f = o % OUTS, row = (o / OUTS) & 15, i = o / OUTS / 16;
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int d = 0; d < (DUAL ? 2 : 1); ++d) {
            const int wt = (HALF * d + f) / 16;   // the 16 weight rows of this sum
#pragma unroll
            for (int rn = 0; rn < RUNS; ++rn)
                v[d] += red[slot(STREAMS * rn + wt / NB, wt % NB, i, row & 3) + (row >> 2) * 16 + (f & 15)];
        }
        const int m = m0 + 16 * i + row;
        if (m < a.M && f0 + f < a.F)
            ((T*)a.Y)[(int64_t)m * a.ldy + f0 + f] = (T)(DUAL ? act_value<sizeof(T) == 4>(a.act, v[0]) * v[1] : v[0]);
    }
}

int check_w4(const W4Args& a, bool) {
    return cdiv(a.M, 16) <= 65535 && cdiv(a.F, 4) <= max_workgroups(512) ? 0 : SGEMM_F32_ERR_TOO_LARGE;
}

template <class T, bool DUAL, int MB, int PER, int NW = 8, int NB = 1, int STREAMS = 2, bool SHORT = false>
static hipError_t launch_rows(const W4Args& a, const W4Groups& gr, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(a.F, (DUAL ? 8 : 16) * NB * STREAMS), (unsigned)cdiv(a.M, 16 * MB));
    hipLaunchKernelGGL((k_w4_rows<T, DUAL, MB, PER, NW, NB, STREAMS, SHORT>), grid, dim3(NW * 64), 0, s, a, gr);
    return hipGetLastError();
}

template <class T, bool DUAL, int PER>
static hipError_t launch_any(const W4Args& a, const W4Groups& gr, hipStream_t s) {
    // Up to two rows the vector units keep up with the weights (8192 x 8192, one
    // row 10.5 us against 21 on the matrix cores, two 13.4 against 21; four
    // would be level).
    if (a.M <= 2)
        return a.M <= 1 ? launch_few<T, DUAL, 1>(a, gr, s) : launch_few<T, DUAL, 2>(a, gr, s);
    // As few workgroups of up to 64 rows (FP32, whose X takes three parts of
    // LDS: 32) as hold X, of equal height.
    constexpr int MOST = sizeof(T) == 4 ? 32 : 64;
    const int64_t blocks = cdiv(a.M, MOST);
    const int height = (int)cdiv(a.M, 16 * blocks);
    // 32, 64 or 128 weight rows a workgroup: X is staged and its fragments are read
    // once for all of them, but fewer workgroups run. A round of 256 over 8192 k
    // takes 36, 46 or 71 us (64 rows of X, 16-bit), 47, 55 or 80 (32 rows, FP32),
    // so by those and the rounds (8192 x 8192, 256 rows: bf16 122, 80, 71, FP32
    // 322, 195, 162; 4096 rows bf16 1746, 1179, 979).
    auto rounds = [&](int rows) { return (double)cdiv(cdiv(a.F, DUAL ? rows / 2 : rows) * blocks, 256); };
    constexpr bool F32 = sizeof(T) == 4;
    const double by32 = rounds(32) * (F32 ? 47 : 36), by64 = rounds(64) * (F32 ? 55 : 46),
                 by128 = rounds(128) * (F32 ? 80 : 71);
    auto many = [&](auto mb) {
        constexpr int MB = decltype(mb)::value;
        if (by32 <= by64 && by32 <= by128) return launch_rows<T, DUAL, MB, PER>(a, gr, s);
        return by64 <= by128 ? launch_rows<T, DUAL, MB, PER, 8, 2>(a, gr, s)
                             : launch_rows<T, DUAL, MB, PER, 8, 2, 4>(a, gr, s);
    };
    if (height == 2) return many(std::integral_constant<int, 2>{});
    if constexpr (sizeof(T) == 2) {
        if (height == 3) return many(std::integral_constant<int, 3>{});
        if (height == 4) return many(std::integral_constant<int, 4>{});
        // Sixteen waves where a unit holds one workgroup and the rows are long (16
        // rows bf16: 8192 x 8192 17.9 -> 16.2 us, 4096 x 14336 26.2 -> 21.6;
        // with two workgroups, gated 8192 x 4096, 14.1 -> 17.7; 3000 k 7.6 -> 7.9).
        // FP32's X then fits one stage only: level.
        if (a.K >= 8192 && cdiv(a.F, DUAL ? 16 : 32) <= 256) return launch_rows<T, DUAL, 1, PER, 16>(a, gr, s);
    }
    return launch_rows<T, DUAL, 1, PER>(a, gr, s);
}

hipError_t launch_w4(int dtype, const W4Args& a, bool dual, hipStream_t s) {
    W4Groups gr = {a.group / 32, -1};
    if ((gr.steps & (gr.steps - 1)) == 0) gr.shift = __builtin_ctz(gr.steps);
    return with_dtype(dtype, [&](auto tag) {
        using T = typename decltype(tag)::type;
        auto go = [&](auto d) {
            constexpr bool D = decltype(d)::value;
            if (a.K < 32) return launch_rows<T, D, 1, 1, 8, 1, 2, true>(a, gr, s);
            if (gr.steps % 4 == 0) return launch_any<T, D, 4>(a, gr, s);
            if (gr.steps % 2 == 0) return launch_any<T, D, 2>(a, gr, s);
            return launch_any<T, D, 1>(a, gr, s);
        };
        return dual ? go(std::true_type{}) : go(std::false_type{});
    });
}

}  // namespace sgemm

// The matrix-core tile of the gated block's products, for FP32, bfloat16 and
// half operands with FP32 sums.
//
// All types share one tile geometry counted in 16-byte chunks: an operand's
// part of a K slice is ROWS rows of 128 bytes (SLICE = 32 FP32 or 64 16-bit
// k). The k index is only a summation index, so lane half h (lanes 32h ..
// 32h + 31) walks its own half of the slice, chunk 4h + v at part v: one
// 16-byte fragment feeds four v_mfma_f32_32x32x2_f32, or one
// v_mfma_f32_32x32x16_{bf16,f16}, whose 8 k of a lane are 16 bytes.
//
// An operand whose k runs along memory rows (KC) is stored [row][k] in LDS, chunk
// q of row r at q ^ swz32(r) (common.hpp), so fragment reads and fills are free
// of bank conflicts. A 16-bit operand whose rows run along memory rows (RC: dG
// and dU as the left factor of dW, X as its right one, W in dX) is stored
// [k][row], and ds_read_b64_tr_b16 hands each lane the four k of its row: in
// a group of 16 lanes, lane i addresses 4 rows' chunk i % 4 of k line i / 4
// and receives row i of all four lines.
#pragma once

#include "ffn.hpp"

namespace sgemm {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// 16 bytes at an address aligned to its element only.
typedef i32x4 i32x4_u2 __attribute__((aligned(2)));

template <class T>
struct Elem {
    static constexpr int EPC = 16 / sizeof(T);   // elements per 16-byte chunk
    static constexpr int SLICE = 8 * EPC;        // k per slice (128 bytes)
};

__device__ __forceinline__ void mma_chunk(float, const i32x4& a, const i32x4& b, f32x16& c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], c, 0, 0, 0);
}
__device__ __forceinline__ void mma_chunk(bf16, const i32x4& a, const i32x4& b, f32x16& c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ void mma_chunk(f16, const i32x4& a, const i32x4& b, f32x16& c) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                               __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// One lane's fragment of a transposed read: 8 k of one row, from two b64 reads.
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4_ptr;
__device__ __forceinline__ i32x4 read_tr(const char* lo, const char* hi) {
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(lo));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_ptr)(hi));
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    const i32x2 x = __builtin_bit_cast(i32x2, a), y = __builtin_bit_cast(i32x2, b);
    return i32x4{x.x, x.y, y.x, y.y};
}

// Where an operand's elements are: lines of `ld` elements from `p`, of which
// `lines` exist, each with `extent` elements along it. A KC operand's lines
// are its rows and k runs along them; an RC operand's lines are k.
template <class T>
struct Lines {
    const T* p;
    int64_t ld;
    int lines, extent;
};

// The chunk of EPC elements of a line from `at`: elements past the extent, and
// lines that do not exist, are zero. Nothing outside the line is read.
template <class T>
__device__ __forceinline__ i32x4 load_chunk(const Lines<T>& s, int line, int at) {
    constexpr int EPC = Elem<T>::EPC;
    i32x4 v = {0, 0, 0, 0};
    if (line < s.lines && at < s.extent) {
        const T* p = s.p + (int64_t)line * s.ld + at;
        if (at + EPC <= s.extent) {
            v = *(const i32x4_u2*)p;
        } else {
            typedef T Vec __attribute__((ext_vector_type(EPC)));
            Vec x = __builtin_bit_cast(Vec, v);
#pragma unroll
            for (int e = 0; e < EPC; ++e)
                if (at + e < s.extent) x[e] = p[e];
            v = __builtin_bit_cast(i32x4, x);
        }
    }
    return v;
}

// LDS placement of an RC operand's 16-byte chunk (k line, chunk of 8 rows):
// the four k lines that one transposed read takes (kline & 3) lie in distinct
// 64-byte quarters of the 256 bytes that the banks span.
template <int ROWS>
__device__ __forceinline__ int rc_chunk(int kline, int c) {
    return c ^ (ROWS >= 128 ? (kline & 3) << 2 : ((kline >> 1) & 1) << 2);
}

// Register-staged fill of one operand's part of a slice: NT threads, CH
// chunks each.
template <class T, int ROWS, int NT, bool RC>
struct RegFill {
    static constexpr int EPC = Elem<T>::EPC;
    static constexpr int CHUNKS = ROWS * 8;
    static_assert(CHUNKS % NT == 0, "tile/threads mismatch");
    static constexpr int CH = CHUNKS / NT;
    static constexpr int CPL = ROWS / EPC;   // chunks per k line (RC)
    i32x4 v[CH];

    // Slice of k0 .. k0 + SLICE - 1, tile rows from r0. A KC operand may be
    // two matrices whose rows alternate in blocks of 32 (PAIR: block b of the tile
    // is block b / 2 of matrix b % 2, both from row r0).
    template <bool PAIR>
    __device__ __forceinline__ void load(const Lines<T>* s, int r0, int k0, int t) {
#pragma unroll
        for (int p = 0; p < CH; ++p) {
            const int slot = t + NT * p;
            if constexpr (RC) {
                v[p] = load_chunk(s[0], k0 + slot / CPL, r0 + (slot % CPL) * EPC);
            } else {
                const int row = slot / 8, at = k0 + (slot % 8) * EPC;
                if constexpr (PAIR) {
                    const bool u = (row >> 5) & 1;
                    const Lines<T> q = {u ? s[1].p : s[0].p, u ? s[1].ld : s[0].ld, s[0].lines, s[0].extent};
                    v[p] = load_chunk(q, r0 + (row >> 6) * 32 + (row & 31), at);
                }
                else
                    v[p] = load_chunk(s[0], r0 + row, at);
            }
        }
    }
    __device__ __forceinline__ void store(char* lds, int t) const {
#pragma unroll
        for (int p = 0; p < CH; ++p) {
            const int slot = t + NT * p;
            int at;
            if constexpr (RC) {
                const int k = slot / CPL;
                at = k * CPL + rc_chunk<ROWS>(k, slot % CPL);
            } else {
                const int row = slot / 8;
                at = row * 8 + ((slot % 8) ^ swz_chunk<32>(row));
            }
            *(i32x4*)(lds + at * 16) = v[p];
        }
    }
};

// A lane's fragment addresses for one operand: 32-row block `blk` of the
// tile, part v of the slice.
template <class T, int ROWS, bool RC>
__device__ __forceinline__ i32x4 read_frag(const char* lds, int row0, int lane, int v) {
    const int h = lane >> 5;
    if constexpr (RC) {
        const int i = lane & 15, row = row0 + (lane & 16) + 4 * (i & 3);
        const int k = 32 * h + 8 * v + (i >> 2);
        constexpr int PITCH = ROWS * 2;
        const char* lo = lds + k * PITCH + rc_chunk<ROWS>(k, row >> 3) * 16 + (row & 7) * 2;
        const char* hi = lds + (k + 4) * PITCH + rc_chunk<ROWS>(k + 4, row >> 3) * 16 + (row & 7) * 2;
        return read_tr(lo, hi);
    } else {
        const int row = row0 + (lane & 31);
        return *(const i32x4*)(lds + row * 128 + (((4 * h + v) ^ swz_chunk<32>(row)) << 4));
    }
}

// The product of one tile: BM x BN outputs, waves of WM x WN, both operands
// through registers into two LDS stages. `nslices` slices; slice s takes its
// operands from sources src(s, A sources, B sources) -> first k.
template <class T, int BM, int BN, int WM, int WN, bool ARC, bool BRC, bool PAIR>
struct TileCore {
    static constexpr int WAVES_N = BN / WN;
    static constexpr int NT = (BM / WM) * WAVES_N * 64;
    static constexpr int BI = WM / 32, BJ = WN / 32;
    static constexpr int STAGE = (BM + BN) * 128;

    template <class Src>
    __device__ __forceinline__ static void run(char* lds, int m0, int n0, int nslices, Src&& src,
                                               f32x16 (&acc)[BI][BJ]) {
        const int t = threadIdx.x, lane = t & 63, w = t >> 6;
        const int wm = (w / WAVES_N) * WM, wn = (w % WAVES_N) * WN;
#pragma unroll
        for (int i = 0; i < BI; ++i)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
        if (nslices <= 0) return;
        RegFill<T, BM, NT, ARC> fa;
        RegFill<T, BN, NT, BRC> fb;
        auto load = [&](int s) {
            Lines<T> la, lb[2];
            const int k0 = src(s, la, lb);
            fa.template load<false>(&la, m0, k0, t);
            fb.template load<PAIR>(lb, n0, k0, t);
        };
        auto store = [&](int s) {
            char* st = lds + (s & 1) * STAGE;
            fa.store(st, t);
            fb.store(st + BM * 128, t);
        };
        load(0);
        store(0);
        __syncthreads();
        for (int s = 0; s < nslices; ++s) {
            if (s + 1 < nslices) load(s + 1);
            const char* A = lds + (s & 1) * STAGE;
            const char* B = A + BM * 128;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                i32x4 a[BI], b[BJ];
#pragma unroll
                for (int i = 0; i < BI; ++i) a[i] = read_frag<T, BM, ARC>(A, wm + 32 * i, lane, v);
#pragma unroll
                for (int j = 0; j < BJ; ++j) b[j] = read_frag<T, BN, BRC>(B, wn + 32 * j, lane, v);
#pragma unroll
                for (int i = 0; i < BI; ++i)
#pragma unroll
                    for (int j = 0; j < BJ; ++j) mma_chunk(T{}, a[i], b[j], acc[i][j]);
            }
            // The other stage was last read before the previous barrier.
            if (s + 1 < nslices) store(s + 1);
            __syncthreads();
        }
    }

    // f(i, j, register values of block (bi, bj) at tile row i, tile column j).
    template <class Fn>
    __device__ __forceinline__ static void each(Fn&& f) {
        const int t = threadIdx.x, lane = t & 63, w = t >> 6;
        const int wm = (w / WAVES_N) * WM, wn = (w % WAVES_N) * WN;
#pragma unroll
        for (int bi = 0; bi < BI; ++bi)
#pragma unroll
            for (int bj = 0; bj < BJ; ++bj)
#pragma unroll
                for (int r = 0; r < 16; ++r)
                    f(bi, bj, r, wm + 32 * bi + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3),
                      wn + 32 * bj + (lane & 31));
    }
};

}  // namespace sgemm

// The matrix-core tile of the gated block's products, for FP32, bfloat16 and
// half operands with FP32 sums, and for int8 operands with int32 sums.
//
// All types share one tile geometry counted in 16-byte chunks: an operand's
// part of a K slice is ROWS rows of 128 bytes (SLICE = 32 FP32, 64 16-bit or 128
// int8 k). The k index is only a summation index, so lane half h (lanes 32h ..
// 32h + 31) walks its own half of the slice, chunk 4h + v at part v: one
// 16-byte fragment feeds four v_mfma_f32_32x32x2_f32, or one
// v_mfma_f32_32x32x16_{bf16,f16}, whose 8 k of a lane are 16 bytes, or one
// v_mfma_i32_32x32x32_i8, whose 16 are.
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
#include "mfma_pipecore.hpp"   // ring_barrier

namespace sgemm {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

typedef int i32x16 __attribute__((ext_vector_type(16)));

// 16 bytes at an address aligned to its element only.
typedef i32x4 i32x4_u1 __attribute__((aligned(1)));
typedef i32x4 i32x4_u2 __attribute__((aligned(2)));

template <class T>
struct Elem {
    static constexpr int EPC = 16 / sizeof(T);   // elements per 16-byte chunk
    static constexpr int SLICE = 8 * EPC;        // k per slice (128 bytes)
    using Unaligned = std::conditional_t<sizeof(T) == 1, i32x4_u1, i32x4_u2>;
    using Sum = std::conditional_t<sizeof(T) == 1, int, float>;         // of products, and a block's sums
    using Sums = std::conditional_t<sizeof(T) == 1, i32x16, f32x16>;
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

__device__ __forceinline__ void mma_chunk(int8_t, const i32x4& a, const i32x4& b, i32x16& c) {
    c = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
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

// The chunk of EPC elements of a line from `at`, in two steps, so that a tile's
// loads are all in flight at once (a load in a divergent branch would be
// waited for there). load_chunk reads EPC elements of the line without a
// branch: the line's last ones where the chunk would reach past its end, the last
// line where the line does not exist. place_chunk moves the chunk's elements
// into place, zeros behind them. Lines shorter than a chunk (SHORT) are read
// element by element. Nothing outside the lines is read.
template <bool SHORT, class T>
__device__ __forceinline__ i32x4 load_chunk(const Lines<T>& s, int line, int at) {
    constexpr int EPC = Elem<T>::EPC;
    const T* p = s.p + (int64_t)(line < s.lines ? line : s.lines - 1) * s.ld;
    if constexpr (!SHORT) return *(const typename Elem<T>::Unaligned*)(p + (at < s.extent - EPC ? at : s.extent - EPC));
    typedef T Vec __attribute__((ext_vector_type(EPC)));
    Vec x = __builtin_bit_cast(Vec, i32x4{0, 0, 0, 0});
#pragma unroll
    for (int e = 0; e < EPC; ++e) {
        const T y = p[at + e < s.extent ? at + e : s.extent - 1];
        x[e] = at + e < s.extent ? y : (T)0.0f;
    }
    return __builtin_bit_cast(i32x4, x);
}
template <bool SHORT, class T>
__device__ __forceinline__ i32x4 place_chunk(const i32x4& v, const Lines<T>& s, int line, int at) {
    constexpr int EPC = Elem<T>::EPC;
    const int past = SHORT ? 0 : at - (s.extent - EPC);   // elements to drop
    const unsigned __int128 x = __builtin_bit_cast(unsigned __int128, v);
    const bool none = line >= s.lines || past >= EPC;
    return __builtin_bit_cast(i32x4, none ? (unsigned __int128)0 : x >> (past > 0 ? 8 * (int)sizeof(T) * past : 0));
}

// LDS placement of an RC operand's 16-byte chunk (k line, chunk of 8 rows):
// the four k lines that one transposed read takes (kline & 3) lie in distinct
// 64-byte quarters of the 256 bytes that the banks span.
// FP32 fragments are read as single words, a row's four k from four lines, and
// need no placement.
template <class T, int ROWS>
__device__ __forceinline__ int rc_chunk(int kline, int c) {
    if (sizeof(T) == 4) return c;
    return c ^ (ROWS >= 128 ? (kline & 3) << 2 : ((kline >> 1) & 1) << 2);
}

// Register-staged fill of one operand's part of a slice: NT threads, CH
// chunks each.
template <class T, int ROWS, int NT, bool RC, bool SHORT>
struct RegFill {
    static constexpr int EPC = Elem<T>::EPC;
    static constexpr int CHUNKS = ROWS * 8;
    static_assert(CHUNKS % NT == 0, "tile/threads mismatch");
    static constexpr int CH = CHUNKS / NT;
    static constexpr int CPL = ROWS / EPC;   // chunks per k line (RC)
    i32x4 v[CH];

    // The chunk of slot `slot`: its line and its place along it. Slice of k0 ..
    // k0 + SLICE - 1, tile rows from r0. A KC operand may be two matrices whose
    // rows alternate in blocks of 32 (PAIR: block b of the tile is block b / 2
    // of matrix b % 2, both from row r0).
    template <bool PAIR>
    __device__ __forceinline__ static void where(int slot, int r0, int k0, int& line, int& at) {
        if constexpr (RC) {
            line = k0 + slot / CPL;
            at = r0 + (slot % CPL) * EPC;
        } else {
            const int row = slot / 8;
            line = r0 + (PAIR ? (row >> 6) * 32 + (row & 31) : row);
            at = k0 + (slot % 8) * EPC;
        }
    }
    template <bool PAIR>
    __device__ __forceinline__ void load(const Lines<T>* s, int r0, int k0, int t) {
#pragma unroll
        for (int p = 0; p < CH; ++p) {
            const int slot = t + NT * p;
            int line, at;
            where<PAIR>(slot, r0, k0, line, at);
            const bool u = PAIR && ((slot / 8 >> 5) & 1);
            v[p] = load_chunk<SHORT>(Lines<T>{u ? s[1].p : s[0].p, u ? s[1].ld : s[0].ld, s[0].lines, s[0].extent}, line, at);
        }
    }
    template <bool PAIR>
    __device__ __forceinline__ void store(char* lds, const Lines<T>* s, int r0, int k0, int t) const {
        // A slice wholly inside its operand needs no placing.
        constexpr int SLICE = Elem<T>::SLICE, TR = PAIR ? ROWS / 2 : ROWS;
        const bool whole = RC ? k0 + SLICE <= s[0].lines && r0 + TR <= s[0].extent
                              : k0 + SLICE <= s[0].extent && r0 + TR <= s[0].lines;
#pragma unroll
        for (int p = 0; p < CH; ++p) {
            const int slot = t + NT * p;
            int at;
            if constexpr (RC) {
                const int k = slot / CPL;
                at = k * CPL + rc_chunk<T, ROWS>(k, slot % CPL);
            } else {
                const int row = slot / 8;
                at = row * 8 + ((slot % 8) ^ swz_chunk<32>(row));
            }
            i32x4 x = v[p];
            if (!whole) {
                int line, place;
                where<PAIR>(slot, r0, k0, line, place);
                x = place_chunk<SHORT>(x, s[0], line, place);
            }
            *(i32x4*)(lds + at * 16) = x;
        }
    }
};

// A lane's fragment addresses for one operand: 32-row block `blk` of the
// tile, part v of the slice.
template <class T, int ROWS, bool RC>
__device__ __forceinline__ i32x4 read_frag(const char* lds, int row0, int lane, int v) {
    const int h = lane >> 5;
    if constexpr (RC && sizeof(T) == 4) {
        const int* p = (const int*)lds + (16 * h + 4 * v) * ROWS + row0 + (lane & 31);
        return i32x4{p[0], p[ROWS], p[2 * ROWS], p[3 * ROWS]};
    } else if constexpr (RC) {
        const int i = lane & 15, row = row0 + (lane & 16) + 4 * (i & 3);
        const int k = 32 * h + 8 * v + (i >> 2);
        constexpr int PITCH = ROWS * 2;
        const char* lo = lds + k * PITCH + rc_chunk<T, ROWS>(k, row >> 3) * 16 + (row & 7) * 2;
        const char* hi = lds + (k + 4) * PITCH + rc_chunk<T, ROWS>(k + 4, row >> 3) * 16 + (row & 7) * 2;
        return read_tr(lo, hi);
    } else {
        const int row = row0 + (lane & 31);
        return *(const i32x4*)(lds + row * 128 + (((4 * h + v) ^ swz_chunk<32>(row)) << 4));
    }
}

// The product of one tile: BM x BN outputs, waves of WM x WN, both operands
// through registers into two LDS stages. src(s, A, B[2]) gives slice s's
// operands and returns its first k; slices s_begin .. s_end - 1 are summed. Two
// register sets keep the loads of the next two slices in flight (a slice's
// products are shorter than a load's way from memory), and the barrier waits for
// LDS only.
//
// KS = 2: two waves share each wave tile and take half of every slice each, so that
// a small tile has four waves; exchange() adds their sums, each wave then
// holding half of the rows of each block (registers 0 .. 7).
template <int BM, int BN, int WM, int WN, int KS>
struct WaveMap {
    static constexpr int WAVES_N = BN / WN, WAVES = (BM / WM) * WAVES_N;
    static constexpr int BI = WM / 32, BJ = WN / 32, REGS = 16 / KS;
    int wm, wn, kk, lane, w;
    __device__ __forceinline__ WaveMap() {
        const int t = threadIdx.x;
        lane = t & 63;
        w = t >> 6;
        kk = KS == 1 ? 0 : w / WAVES;
        const int mn = KS == 1 ? w : w - kk * WAVES;
        wm = (mn / WAVES_N) * WM;
        wn = (mn % WAVES_N) * WN;
    }
    // `space`: 64 lanes x BI BJ 16 words for each wave, free to be written.
    template <class T>
    __device__ __forceinline__ void exchange(typename Elem<T>::Sum* const* space, typename Elem<T>::Sums (&acc)[BI][BJ]) const {
        if constexpr (KS > 1) {
#pragma unroll
            for (int i = 0; i < BI; ++i)
#pragma unroll
                for (int j = 0; j < BJ; ++j)
#pragma unroll
                    for (int r = 0; r < 16; ++r) space[w][((i * BJ + j) * 16 + r) * 64 + lane] = acc[i][j][r];
            __syncthreads();
            const int mn = w - kk * WAVES;
#pragma unroll
            for (int i = 0; i < BI; ++i)
#pragma unroll
                for (int j = 0; j < BJ; ++j)
#pragma unroll
                    for (int r = 0; r < REGS; ++r) {
                        typename Elem<T>::Sum v = 0;
#pragma unroll
                        for (int g = 0; g < KS; ++g)
                            v += space[mn + g * WAVES][((i * BJ + j) * 16 + kk * REGS + r) * 64 + lane];
                        acc[i][j][r] = v;
                    }
            __syncthreads();   // the space is free again
        }
    }
};

template <class T, int BM, int BN, int WM, int WN, bool ARC, bool BRC, bool PAIR, int KS = 1, bool SHORT = false>
struct TileCore {
    using Map = WaveMap<BM, BN, WM, WN, KS>;
    static constexpr int NT = Map::WAVES * KS * 64;
    static constexpr int BI = WM / 32, BJ = WN / 32;
    using Sums = typename Elem<T>::Sums;
    static constexpr int STAGE = (BM + BN) * 128;
    static constexpr int PER_WAVE = 2 * STAGE / (Map::WAVES * KS);   // LDS of a wave's own, the product done

    template <class Src>
    __device__ __forceinline__ static void run(char* lds, int m0, int n0, int s_begin, int s_end, Src&& src,
                                               typename Elem<T>::Sums (&acc)[BI][BJ]) {
        const Map map;
        const int t = threadIdx.x, lane = map.lane, wm = map.wm, wn = map.wn;
#pragma unroll
        for (int i = 0; i < BI; ++i)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
        if (s_begin >= s_end) return;
        struct Set {
            RegFill<T, BM, NT, ARC, SHORT> a;
            RegFill<T, BN, NT, BRC, SHORT> b;
        };
        // Past the last slice the last one is loaded (and stored) again.
        auto load = [&](int s, Set& r) {
            Lines<T> la, lb[2];
            const int k0 = src(s < s_end ? s : s_end - 1, la, lb);
            r.a.template load<false>(&la, m0, k0, t);
            r.b.template load<PAIR>(lb, n0, k0, t);
        };
        auto store = [&](int s, const Set& r, char* st) {
            Lines<T> la, lb[2];
            const int k0 = src(s < s_end ? s : s_end - 1, la, lb);
            r.a.template store<false>(st, &la, m0, k0, t);
            r.b.template store<PAIR>(st + BM * 128, lb, n0, k0, t);
        };
        auto compute = [&](const char* A) {
            const char* B = A + BM * 128;
#pragma unroll
            for (int p = 0; p < 4 / KS; ++p) {
                const int v = map.kk * (4 / KS) + p;
                i32x4 a[BI], b[BJ];
#pragma unroll
                for (int i = 0; i < BI; ++i) a[i] = read_frag<T, BM, ARC>(A, wm + 32 * i, lane, v);
#pragma unroll
                for (int j = 0; j < BJ; ++j) b[j] = read_frag<T, BN, BRC>(B, wn + 32 * j, lane, v);
#pragma unroll
                for (int i = 0; i < BI; ++i)
#pragma unroll
                    for (int j = 0; j < BJ; ++j) mma_chunk(T{}, b[j], a[i], acc[i][j]);
            }
        };
        Set r0, r1;
        load(s_begin, r0);
        load(s_begin + 1, r1);
        store(s_begin, r0, lds);
        load(s_begin + 2, r0);
        ring_barrier<63>();
        // The stage written was last read before the previous barrier.
        auto slice = [&](int s, char* now, char* next, Set& r) {
            compute(now);
            __builtin_amdgcn_sched_barrier(0);
            store(s + 1, r, next);
            load(s + 3, r);
            ring_barrier<63>();
        };
        int s = s_begin;
        for (; s + 2 <= s_end; s += 2) {
            slice(s, lds, lds + STAGE, r1);
            slice(s + 1, lds + STAGE, lds, r0);
        }
        if (s < s_end) {
            compute(lds);
            ring_barrier<63>();
        }
        if constexpr (KS > 1) {
            using Sum = typename Elem<T>::Sum;
            Sum* const space[4] = {(Sum*)lds, (Sum*)(lds + STAGE / 2), (Sum*)(lds + STAGE),
                                   (Sum*)(lds + STAGE + STAGE / 2)};
            static_assert(Map::WAVES * KS == 4 && BI * BJ * 16 * 64 * 4 <= STAGE / 2, "a wave's sums fit");
            map.template exchange<T>(space, acc);
        }
    }
};

// ---------------------------------------------------------------------------
// The same tile filled by buffer-to-LDS loads and software-pipelined, for
// operands whose lines are whole 16-byte chunks.
//
// One workgroup per compute unit: two LDS stages of (BM + BN) x 128 bytes. A
// slice is four parts; each part's matrix instructions run while the fragments of
// the next part are read into the other register set. The barrier sits before the
// last part: every wave has then read the whole stage and its own loads of
// the next slice have landed, so after it the stage is refilled (the slice
// after next) and the next slice's first fragments are read, both under the last
// part's matrix instructions.
// ---------------------------------------------------------------------------
constexpr uint32_t kRange = 0x80000000u;   // byte offsets of an operand's tile stay below

// Buffer-to-LDS fill of one operand's part of a slice.
template <class T, int ROWS, int NT, bool RC>
struct DmaFill {
    static constexpr int EPC = Elem<T>::EPC, SLICE = Elem<T>::SLICE;
    static constexpr int W = NT / 64, PIECES = ROWS / 8;   // of 64 chunks
    static_assert(PIECES % W == 0, "whole pieces per wave");
    static constexpr int G = PIECES / W;                   // loads per wave
    static constexpr int CPL = ROWS / EPC;
    uint32_t off[G];   // byte offset from the tile's first line, OOB where the line does not exist
    int q[G];          // KC: first k of the chunk

    // PAIR: which of the two matrices piece p of wave w (8 rows) belongs to.
    static_assert(W == 1 || W == 2 || W == 4 || W % 8 == 0, "a piece's matrix depends on the wave or on p alone");
    __device__ __forceinline__ static int matrix(int w, int p) {
        return W <= 4 ? (W * p >> 2) & 1 : (w >> 2) & 1;
    }

    // A KC tile's rows start at line r0 (PAIR: of both matrices, as in
    // RegFill), an RC tile's chunks at element r0 of each line.
    template <bool PAIR>
    __device__ __forceinline__ void init(const Lines<T>* s, int r0, int t) {
        const int w = __builtin_amdgcn_readfirstlane(t >> 6), lane = t & 63;
        const int lines = s[0].lines, extent = s[0].extent;
#pragma unroll
        for (int p = 0; p < G; ++p) {
            const int slot = (w + W * p) * 64 + lane;
            const int64_t ld = PAIR && matrix(w, p) ? s[1].ld : s[0].ld;
            if constexpr (RC) {
                const int k = slot / CPL, c = rc_chunk<T, ROWS>(k, slot % CPL);
                off[p] = r0 + c * EPC < extent ? (uint32_t)((k * (int)ld + c * EPC) * (int)sizeof(T)) : OOB;
            } else {
                const int row = slot / 8, src = PAIR ? (row >> 6) * 32 + (row & 31) : row;
                q[p] = ((slot % 8) ^ swz_chunk<32>(row)) * EPC;
                off[p] = r0 + src < lines ? (uint32_t)((src * (int)ld + q[p]) * (int)sizeof(T)) : OOB;
            }
        }
    }
    // The slice at k0 of s, whose tile starts at row r0. Past the last k
    // everything reads as zero.
    template <bool PAIR>
    __device__ __forceinline__ void issue(const Lines<T>* both, int r0, int k0, int t, char* lds) const {
        const int w = __builtin_amdgcn_readfirstlane(t >> 6);
        const Lines<T>& s = both[0];
        const int left = (RC ? s.lines : s.extent) - k0;
        const int kk = __builtin_amdgcn_readfirstlane(left <= 0 ? 0 : left < SLICE ? left : SLICE);
        const T* base = RC ? s.p + (int64_t)k0 * s.ld + r0 : s.p + (int64_t)r0 * s.ld + k0;
        // RC: k lines past the last are past the resource's end. KC: rows
        // that do not exist have the offset OOB, k past the last is masked below.
        const uint32_t bytes = kk == 0 ? 0u
                               : RC ? (uint32_t)(((int64_t)(kk - 1) * s.ld + (s.extent - r0)) * (int64_t)sizeof(T))
                                    : kRange;
        const __amdgpu_buffer_rsrc_t r = make_rsrc((const float*)base, bytes);
        __amdgpu_buffer_rsrc_t r1 = r;
        if constexpr (PAIR) r1 = make_rsrc((const float*)(both[1].p + (int64_t)r0 * both[1].ld + k0), bytes);
        const bool mask = !RC && kk < SLICE;
#pragma unroll
        for (int p = 0; p < G; ++p) {
            const uint32_t o = mask && q[p] >= kk ? OOB : off[p];
            if (PAIR && matrix(w, p))
                buf_load_lds16(r1, (const float*)(lds + (w + W * p) * 1024), o);
            else
                buf_load_lds16(r, (const float*)(lds + (w + W * p) * 1024), o);
        }
    }
};

template <class T, int BM, int BN, int WM, int WN, bool ARC, bool BRC, bool PAIR, int KS = 1>
struct DmaCore {
    using Map = WaveMap<BM, BN, WM, WN, KS>;
    static constexpr int NT = Map::WAVES * KS * 64;
    static constexpr int BI = WM / 32, BJ = WN / 32;
    using Sums = typename Elem<T>::Sums;
    static constexpr int LDS_A = BM * 128, LDS_B = BN * 128;
    // LDS of a wave's own once the product is done.
    static constexpr int WAVES = Map::WAVES * KS, PER_WAVE = 2 * (LDS_A + LDS_B) / WAVES;
    static_assert(LDS_A == LDS_B && WAVES % 4 == 0, "four equal objects, whole waves in each");
    __device__ __forceinline__ static char* own(char* a0, char* b0, char* a1, char* b1) {
        const int w = threadIdx.x >> 6, o = w / (WAVES / 4);
        return (o == 0 ? a0 : o == 1 ? b0 : o == 2 ? a1 : b1) + w % (WAVES / 4) * PER_WAVE;
    }
    using FA = DmaFill<T, BM, NT, ARC>;
    using FB = DmaFill<T, BN, NT, BRC>;

    struct Frag {
        i32x4 a[BI], b[BJ];
    };

    // Order of one region's instructions: MFMAS matrix instructions, the reads
    // of the next part early among them and the fill's loads behind those.
    template <int LOADS>
    __device__ __forceinline__ static void weave() {
        constexpr int MFMA = 0x008, VMEM_READ = 0x020, DS_READ = 0x100;
        constexpr int MFMAS = BI * BJ * (sizeof(T) == 4 ? 4 : 1);
        constexpr int RC_READS = sizeof(T) == 4 ? 4 : 2;
        constexpr int READS = BI * (ARC ? RC_READS : 1) + BJ * (BRC ? RC_READS : 1);
        constexpr int RN = MFMAS > 2 ? MFMAS - 2 : 1, RS = (READS + RN - 1) / RN;   // reads after each of the first RN
        constexpr int LS = LOADS == 0 ? 1 : (LOADS + MFMAS - 2) / (MFMAS - 1);
#pragma unroll
        for (int i = 0; i < MFMAS; ++i) {
            __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
            if (i * RS < READS) __builtin_amdgcn_sched_group_barrier(DS_READ, RS, 0);
            if (i * LS < LOADS) __builtin_amdgcn_sched_group_barrier(VMEM_READ, LS, 0);
        }
    }

    // src(s, A, B[2]) -> first k of slice s, with the operands' lines.
    template <class Src>
    __device__ __forceinline__ static void run(char* a0, char* b0, char* a1, char* b1, int m0, int n0,
                                               int s_begin, int s_end, Src&& src, typename Elem<T>::Sums (&acc)[BI][BJ]) {
        const Map map;
        const int t = threadIdx.x, lane = map.lane, wm = map.wm, wn = map.wn;
#pragma unroll
        for (int i = 0; i < BI; ++i)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
        if (s_begin >= s_end) return;
        FA fa;
        FB fb;
        {
            Lines<T> la, lb[2];
            src(s_begin, la, lb);
            fa.template init<false>(&la, m0, t);
            fb.template init<PAIR>(lb, n0, t);
        }
        auto issue = [&](int s, char* A, char* B) {
            Lines<T> la, lb[2];
            const int k0 = src(s, la, lb);
            fa.template issue<false>(&la, m0, k0, t, A);
            fb.template issue<PAIR>(lb, n0, k0, t, B);
        };
        auto read = [&](Frag& f, const char* A, const char* B, int v) {
#pragma unroll
            for (int i = 0; i < BI; ++i) f.a[i] = read_frag<T, BM, ARC>(A, wm + 32 * i, lane, v);
#pragma unroll
            for (int j = 0; j < BJ; ++j) f.b[j] = read_frag<T, BN, BRC>(B, wn + 32 * j, lane, v);
        };
        auto mma = [&](const Frag& f) {
#pragma unroll
            for (int i = 0; i < BI; ++i)
#pragma unroll
                for (int j = 0; j < BJ; ++j) mma_chunk(T{}, f.b[j], f.a[i], acc[i][j]);
        };
        Frag f0, f1;
        issue(s_begin, a0, b0);
        issue(s_begin + 1, a1, b1);   // past the last slice: never used
        ring_barrier<FA::G + FB::G>();
        constexpr int PARTS = 4 / KS;
        const int v0 = map.kk * PARTS;
        read(f0, a0, b0, v0);
        auto slice = [&](int s, char* A, char* B, char* An, char* Bn) {
#pragma unroll
            for (int p = 0; p + 1 < PARTS; ++p) {
                read(p & 1 ? f0 : f1, A, B, v0 + p + 1);
                mma(p & 1 ? f1 : f0);
                weave<0>();
                __builtin_amdgcn_sched_barrier(0);
            }
            ring_barrier<0>();
            read(f0, An, Bn, v0);
            mma(f1);
            issue(s + 2, A, B);
            weave<FA::G + FB::G>();
            __builtin_amdgcn_sched_barrier(0);
        };
        int s = s_begin;
        for (; s + 2 <= s_end; s += 2) {
            slice(s, a0, b0, a1, b1);
            slice(s + 1, a1, b1, a0, b0);
        }
        if (s < s_end) slice(s, a0, b0, a1, b1);
        ring_barrier<0>();   // the loads past the last slice land before LDS is given up
        if constexpr (KS > 1) {
            using Sum = typename Elem<T>::Sum;
            Sum* const space[4] = {(Sum*)a0, (Sum*)b0, (Sum*)a1, (Sum*)b1};
            static_assert(Map::WAVES * KS == 4 && BI * BJ * 16 * 64 * 4 <= (LDS_A < LDS_B ? LDS_A : LDS_B),
                          "a wave's sums fit");
            map.template exchange<T>(space, acc);
        }
    }
};

// Waits until this wave's LDS reads are done; nothing moves across. Before a
// stage that they read is filled again.
__device__ __forceinline__ void lds_wait() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));
    asm volatile("" ::: "memory");
}
// Waits until at most VMCNT of this wave's vector-memory operations are
// outstanding (their LDS writes included); nothing moves across.
template <int VMCNT>
__device__ __forceinline__ void wave_wait() {
    static_assert(VMCNT >= 0 && VMCNT < 64, "vmcnt field is 6 bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((VMCNT & 15) | ((VMCNT >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("" ::: "memory");
}

// Between a wave's lanes writing LDS of the wave's own and other lanes of it reading that, and before it is written
// again. The hardware keeps a wave's LDS instructions in their order, so nothing is waited for; the
// compiler, which sees each lane's addresses by themselves, may not move one across.
__device__ __forceinline__ void lanes_meet() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// One block row of a wave's results on its way out: 32 rows of COLS columns of
// type O, through LDS of the wave's own (no barrier), so that a store
// instruction writes whole runs of rows, 16 bytes a lane. The matrix instructions take
// the column operand first, so a lane's registers run along a row: lane l holds
// row l % 32, register group r of a block its columns 8 r + 4 (l / 32) + 0..3.
// (Stored from the registers, those 16 or 8 bytes of each of 32 rows a time, the
// FP32 pre-activations of 4096 x 8192 outputs cost 140 us more.)
template <class O, int COLS>
struct RowsOut {
    static constexpr int PITCH = COLS * (int)sizeof(O) + 16;   // bytes; rows 16 bytes apart in the banks
    static constexpr int BYTES = 32 * PITCH;
    static constexpr int EPC = 16 / (int)sizeof(O), LPR = COLS / EPC;   // lanes per row
    typedef O O4 __attribute__((ext_vector_type(4)));
    char* lds;
    int lane;

    __device__ __forceinline__ void put(int col, float a, float b, float c, float d) const {
        *(O4*)(lds + (lane & 31) * PITCH + (col + 4 * (lane >> 5)) * (int)sizeof(O)) = O4{(O)a, (O)b, (O)c, (O)d};
    }
    // To rows row0 .. of a matrix whose first column here is `out`'s; `rows` and
    // `cols` of them exist.
    __device__ __forceinline__ void flush(O* out, int64_t ld, int row0, int rows, int cols) const {
        lanes_meet();
        typedef O E __attribute__((ext_vector_type(EPC)));
        typedef E Eu __attribute__((aligned(sizeof(O))));
#pragma unroll
        for (int i = 0; i < 32 * LPR / 64; ++i) {
            const int at = i * 64 + lane, row = at / LPR, col = at % LPR * EPC;
            const E v = *(const E*)(lds + row * PITCH + col * (int)sizeof(O));
            O* p = out + (int64_t)(row0 + row) * ld + col;
            if (row0 + row < rows && col < cols) {
                if (col + EPC <= cols) {
                    *(Eu*)p = v;
                } else {
#pragma unroll
                    for (int k = 0; k < EPC - 1; ++k)
                        if (col + k < cols) p[k] = v[k];
                }
            }
        }
        lanes_meet();
    }
};

constexpr int GLU_GROUP_M = 4;

// A core's product in LDS of its own: two stages for each operand, as objects
// apart so that the compiler can tell the stage being filled from the one
// being read.
// Returns LDS of the wave's own for the results.
template <class Core, bool DMA, class Src>
__device__ __forceinline__ char* product(int m0, int n0, int s_begin, int s_end, Src&& src,
                                        typename Core::Sums (&acc)[Core::BI][Core::BJ]) {
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
    static constexpr bool ALONE = false;
    using Map = WaveMap<BM_, BN_, WM_, WN_, KS_>;
    template <class T, bool ARC, bool BRC, bool PAIR>
    using Core = std::conditional_t<DMA_, DmaCore<T, BM_, BN_, WM_, WN_, ARC, BRC, PAIR, KS_>,
                                    TileCore<T, BM_, BN_, WM_, WN_, ARC, BRC, PAIR, KS_, SHORT_>>;
};

// Whether an operand of e-byte elements can be filled by buffer-to-LDS loads:
// whole 16-byte chunks, and a tile's span within 31-bit byte offsets.
static inline bool dma_ok(int64_t e, const void* p, int64_t ld, int64_t extent, int64_t tile_lines) {
    const int64_t chunk = 16 / e;
    // (ld by itself first: a single line's may be anything)
    return aligned16(p) && ld % chunk == 0 && extent % chunk == 0 && ld < (int64_t)kRange &&
           ((tile_lines - 1) * ld + extent) * e < (int64_t)kRange;
}

using TileReg = Tile<128, 128, 64, 64, 1, false>;
using TileReg64 = Tile<64, 64, 32, 64, 2, false>;
using TileDma64 = Tile<64, 64, 32, 64, 2, true>;
using TileShort = Tile<128, 128, 64, 64, 1, false, true>;
using TileMid = Tile<128, 128, 64, 64, 1, true>;
using TileBig = Tile<256, 256, 128, 64, 1, true>;

// Times that the choice of a tile goes by, in microseconds, measured on MI355X
// (products of 300 x 1000 x 511 to 4096 x 8192 x 4096): a call takes about
//     fixed + n max(alone, tiles per compute unit * busy)
// for n slices, with `alone` a slice of a lone tile and `busy` a slice's share of a
// unit that holds several.
struct TileCost {
    double fixed, alone, busy;
    double of(int64_t tiles, int64_t slices) const {
        const double per_unit = (double)((tiles + 255) / 256), b = per_unit * busy;
        return fixed + (double)slices * (b > alone ? b : alone);
    }
};
}  // namespace sgemm

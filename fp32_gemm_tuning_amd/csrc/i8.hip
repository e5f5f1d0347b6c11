// Products of matrices in 8 bits: Y = X W^T (i8) and the gated block over two such
// weights (i8_glu). The matrix cores sum the stored numbers exactly in 32 bits; the
// scales of a token and of a feature multiply each sum once, at the end.
#include "glu_core.hpp"
#include "norm_core.hpp"

namespace sgemm {

// A scale as mantissa and exponent: sum * (Sx * Sw) then leaves FP32's range, or its
// normal numbers, only where the result does (Sx = 2^-100, Sw = 2^90 and the other
// way round are ordinary). Of scales that are `plain` the product of the FP32 numbers
// has the same bits, for two instructions less.
struct Scale {
    float m;
    int e;
    Scale() = default;
    __device__ __forceinline__ explicit Scale(float s)
        : m(__builtin_amdgcn_frexp_mantf(s)), e(__builtin_amdgcn_frexp_expf(s)) {}
};
__device__ __forceinline__ float scaled(int sum, const Scale& x, const Scale& w) {
    return __builtin_amdgcn_ldexpf((float)sum * (x.m * w.m), x.e + w.e);
}
__device__ __forceinline__ bool plain(float s) {
    const float a = fabsf(s);
    return a == 0.0f || (a >= 0x1p-60f && a <= 0x1p60f);
}
template <bool PLAIN>
__device__ __forceinline__ float scaled(int sum, float x, float w) {
    if constexpr (PLAIN) return (float)sum * (x * w);
    return scaled(sum, Scale(x), Scale(w));
}

// LDS that a wave's results go out through (put_i8): 32 rows of 64 FP32 values, and their scales.
constexpr int STAGING = RowsOut<float, 64>::BYTES + 256;

// g = act(g) * u, for N results with one branch on the activation: a branch for each result keeps their
// instructions apart (4096 x 8192 x 4096 gated 250 us, and 264 with both that and mantissas for all scales).
// 16-bit results take the hardware's exponential.
template <class O, int N>
__device__ __forceinline__ void gate(int act, float (&g)[N], const float (&u)[N]) {
    auto all = [&](auto kind) {
#pragma unroll
        for (int e = 0; e < N; ++e) g[e] = as_f32(act_value<sizeof(O) == 4>(decltype(kind)::value, g[e]) * u[e]);
    };
    using std::integral_constant;
    switch (act) {
        case SGEMM_F32_ACT_SILU: all(integral_constant<int, SGEMM_F32_ACT_SILU>{}); break;
        case SGEMM_F32_ACT_GELU: all(integral_constant<int, SGEMM_F32_ACT_GELU>{}); break;
        case SGEMM_F32_ACT_GELU_TANH: all(integral_constant<int, SGEMM_F32_ACT_GELU_TANH>{}); break;
        default: all(integral_constant<int, SGEMM_F32_ACT_RELU>{});
    }
}

// A tile's results: blocks of 32 rows of 32 (KS = 2: 16) features, or, without a gate, of all the
// wave's features together where they are next to each other. The scales of the wave's 64 columns,
// one a lane, go through LDS of its own too: read from memory by the lanes that use them, four
// features each, they took a third more registers than the product.
template <class O, class Tl, class Core, bool DUAL>
__device__ __forceinline__ void put_i8(const I8Args& a, char* own, int m0, int n0,
                                       const i32x16 (&acc)[Core::BI][Core::BJ]) {
    const typename Tl::Map map;
    constexpr int REGS = Tl::Map::REGS, KS = 16 / REGS, STEP = DUAL ? 2 : KS == 1 ? Core::BJ : 1;
    constexpr int TOGETHER = DUAL ? 1 : STEP, COLS = 2 * REGS * TOGETHER;
    static_assert(Core::BJ == 2, "64 columns a wave");
    const RowsOut<O, COLS> o = {own, map.lane};
    static_assert(RowsOut<O, COLS>::BYTES + 256 <= Core::PER_WAVE && Core::PER_WAVE % 16 == 0, "staging");
    float* const scales = (float*)(own + Core::PER_WAVE - 256);
    const int f0 = n0 + (DUAL ? map.wn >> 1 : map.wn);
    bool all_plain;
    {
        const int c = f0 + (DUAL ? map.lane & 31 : map.lane);
        const float* sw = DUAL && map.lane >= 32 ? a.Sw[1] : a.Sw[0];
        const float mine = sw[c < a.F ? c : a.F - 1];
        scales[map.lane] = mine;
        all_plain = __builtin_amdgcn_ballot_w64(!plain(mine)) == 0;
    }
    lanes_meet();
    const int half = 4 * (map.lane >> 5);
#pragma unroll
    for (int bi = 0; bi < Core::BI; ++bi) {
        const int row = m0 + map.wm + 32 * bi, mine = row + (map.lane & 31);
        const float sx = a.Sx[mine < a.M ? mine : a.M - 1];
        auto blocks = [&](auto is_plain) {
            constexpr bool PLAIN = decltype(is_plain)::value;
#pragma unroll
            for (int bj = 0; bj < Core::BJ; bj += STEP) {
                const int col = (DUAL ? 0 : 32 * bj) + 2 * REGS * map.kk;   // of the wave's
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j) {
                    float g[REGS], u[REGS];
#pragma unroll
                    for (int r = 0; r < REGS; r += 4) {
                        const int at = col + 32 * j + 2 * r + half;
                        const f32x4 sg = *(const f32x4*)(scales + at);
#pragma unroll
                        for (int e = 0; e < 4; ++e) g[r + e] = scaled<PLAIN>(acc[bi][bj + j][r + e], sx, sg[e]);
                        if constexpr (DUAL) {
                            const f32x4 su = *(const f32x4*)(scales + 32 + at);
#pragma unroll
                            for (int e = 0; e < 4; ++e) u[r + e] = scaled<PLAIN>(acc[bi][bj + 1][r + e], sx, su[e]);
                        }
                    }
                    if constexpr (DUAL) gate<O>(a.act, g, u);
#pragma unroll
                    for (int r = 0; r < REGS; r += 4) o.put(32 * j + 2 * r, g[r], g[r + 1], g[r + 2], g[r + 3]);
                }
                o.flush((O*)a.Y + f0 + col, a.ldy, row, a.M, a.F - f0 - col);
            }
        };
        if (all_plain && __builtin_amdgcn_ballot_w64(!plain(sx)) == 0)
            blocks(std::true_type{});
        else
            blocks(std::false_type{});
    }
}

// Fill of an operand's part of a slice through registers, for rows that are not whole 16-byte chunks: NT
// threads, CH chunks each. A lane's chunks are all at the same place along the slice, in rows NT / 8 apart, so their
// addresses are one offset for each row, kept in 32 bits, and a place along K; rows past the last one
// are the last one again (their results are not kept). Where a chunk would reach past K, the row's last
// 16 bytes are read and moved down in `store`, zeros behind.
template <int ROWS, int NT, bool PAIR>
struct FlatFill {
    static constexpr int CH = ROWS * 8 / NT, STEP = NT / 8;   // rows apart
    static_assert(ROWS * 8 % NT == 0 && STEP <= 64, "a chunk's matrix depends on it or on the wave alone");
    // PAIR: rows alternate between two matrices in blocks of 32: chunk p's row is of the second where this
    // says so, or, where a step of rows is two blocks, all of a wave's are of one.
    static constexpr bool BY_CHUNK = PAIR && STEP <= 32;
    __device__ __forceinline__ static bool second(int p) { return BY_CHUNK && (STEP * p >> 5) & 1; }
    const int8_t *base, *other;
    uint32_t off[CH];
    int q;   // the lane's place along a slice, in chunks

    __device__ __forceinline__ void init(const Lines<int8_t>* s, int r0, int t) {
        q = t & 7;
        uint32_t ld = (uint32_t)s[0].ld, ld1 = (uint32_t)s[PAIR].ld;
        base = s[0].p + (int64_t)r0 * s[0].ld;
        other = s[PAIR].p + (int64_t)r0 * s[PAIR].ld;
        if (PAIR && !BY_CHUNK && (__builtin_amdgcn_readfirstlane(t >> 8) & 1)) {
            base = other;
            ld = ld1;
        }
#pragma unroll
        for (int p = 0; p < CH; ++p) {
            const int row = (t >> 3) + STEP * p, src = PAIR ? (row >> 6) * 32 + (row & 31) : row;
            const int last = s[0].lines - 1 - r0;
            off[p] = (uint32_t)(src < last ? src : last) * (second(p) ? ld1 : ld);
        }
    }
    __device__ __forceinline__ void load(i32x4 (&v)[CH], int k0, int K) const {
        const int at = k0 + 16 * q, place = at < K - 16 ? at : K - 16;
#pragma unroll
        for (int p = 0; p < CH; ++p) v[p] = *(const i32x4_u1*)((second(p) ? other : base) + (off[p] + (uint32_t)place));
    }
    __device__ __forceinline__ void store(const i32x4 (&v)[CH], char* lds, int k0, int K, int t) const {
#pragma unroll
        for (int p = 0; p < CH; ++p) {
            const int row = (t >> 3) + STEP * p;
            i32x4 x = v[p];
            if (k0 + 128 > K) {
                const int past = k0 + 16 * q - (K - 16);
                const unsigned __int128 w = __builtin_bit_cast(unsigned __int128, x);
                x = __builtin_bit_cast(i32x4, past >= 16 ? (unsigned __int128)0 : w >> (past > 0 ? 8 * past : 0));
            }
            *(i32x4*)(lds + row * 128 + ((q ^ swz_chunk<32>(row)) << 4)) = x;
        }
    }
};

// The tile filled that way: two LDS stages, and SETS slices under way in registers behind the one being
// multiplied (rows that are not whole chunks cannot be loaded past the registers). A second set helps the smallest
// tile where it is alone on its unit (128 x 4091 x 4091 20.4 -> 17.5 us); larger tiles are level, or lose
// the registers' room for a second workgroup (1000 x 4091 x 4091 on 64 x 64 tiles 60 -> 62).
template <int BM, int BN, int WM, int WN, bool PAIR, int KS, int SETS>
struct FlatCore {
    using T = int8_t;
    using Map = WaveMap<BM, BN, WM, WN, KS>;
    using Sums = i32x16;
    static constexpr int STAGES = 2, NT = Map::WAVES * KS * 64, BI = WM / 32, BJ = WN / 32;
    static constexpr int STAGE = (BM + BN) * 128, WAVES = Map::WAVES * KS;
    static constexpr int PER_WAVE = STAGES * STAGE / WAVES > STAGING ? STAGES * STAGE / WAVES / 16 * 16 : STAGING;
    static constexpr int LDS = WAVES * PER_WAVE > STAGES * STAGE ? WAVES * PER_WAVE : STAGES * STAGE;
    using FA = FlatFill<BM, NT, false>;
    using FB = FlatFill<BN, NT, PAIR>;

    template <class Src>
    __device__ __forceinline__ static void run(char* lds, int m0, int n0, int slices, Src&& src, i32x16 (&acc)[BI][BJ]) {
        const Map map;
        const int t = threadIdx.x, lane = map.lane;
#pragma unroll
        for (int i = 0; i < BI; ++i)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
        FA fa;
        FB fb;
        Lines<T> la, lb[2];
        src(0, la, lb);
        fa.init(&la, m0, t);
        fb.init(lb, n0, t);
        const int K = la.extent;
        i32x4 a[SETS][FA::CH], b[SETS][FB::CH];   // slice s: set s % SETS
        // Past the last slice the last one is loaded (and stored) again.
        auto load = [&](int s, int set) {
            const int k0 = (s < slices ? s : slices - 1) * 128;
            fa.load(a[set], k0, K);
            fb.load(b[set], k0, K);
        };
        auto store = [&](int s, int set, char* st) {
            const int k0 = (s < slices ? s : slices - 1) * 128;
            fa.store(a[set], st, k0, K, t);
            fb.store(b[set], st + BM * 128, k0, K, t);
        };
        auto compute = [&](const char* st) {
#pragma unroll
            for (int p = 0; p < 4 / KS; ++p) {
                const int v = map.kk * (4 / KS) + p;
                i32x4 x[BI], w[BJ];
#pragma unroll
                for (int i = 0; i < BI; ++i) x[i] = read_frag<T, BM, false>(st, map.wm + 32 * i, lane, v);
#pragma unroll
                for (int j = 0; j < BJ; ++j) w[j] = read_frag<T, BN, false>(st + BM * 128, map.wn + 32 * j, lane, v);
#pragma unroll
                for (int i = 0; i < BI; ++i)
#pragma unroll
                    for (int j = 0; j < BJ; ++j) mma_chunk(T{}, w[j], x[i], acc[i][j]);
            }
        };
        static_assert(SETS == 1 || SETS == 2, "a slice's set is known");
#pragma unroll
        for (int i = 0; i < SETS; ++i) load(i, i);
        store(0, 0, lds);
        load(SETS, 0);
        ring_barrier<63>();
        // The stage written was last read before the previous barrier.
        auto slice = [&](int s, int set, char* now, char* next) {   // set: of slice s + 1
            compute(now);
            __builtin_amdgcn_sched_barrier(0);
            store(s + 1, set, next);
            load(s + 1 + SETS, set);
            ring_barrier<63>();
        };
        int s = 0;
        for (; s + 2 <= slices; s += 2) {
            slice(s, 1 % SETS, lds, lds + STAGE);
            slice(s + 1, 0, lds + STAGE, lds);
        }
        if (s < slices) {
            compute(lds);
            ring_barrier<63>();
        }
        if constexpr (KS > 1) {
            int* space[Map::WAVES * KS];
#pragma unroll
            for (int w = 0; w < Map::WAVES * KS; ++w) space[w] = (int*)(lds + w * PER_WAVE);
            static_assert(BI * BJ * 16 * 64 * 4 <= PER_WAVE, "a wave's sums fit");
            map.template exchange<T>(space, acc);
        }
    }
};
template <int BM_, int BN_, int WM_, int WN_, int KS_ = 1, int SETS_ = 1>
struct Flat {
    static constexpr int BM = BM_, BN = BN_, NT = (BM_ / WM_) * (BN_ / WN_) * KS_ * 64;
    static constexpr bool ALONE = true;   // its LDS is the core's
    using Map = WaveMap<BM_, BN_, WM_, WN_, KS_>;
    template <class T, bool, bool, bool PAIR>
    using Core = FlatCore<BM_, BN_, WM_, WN_, PAIR, KS_, SETS_>;
};

// A tile for products whose tiles fill the chip once or twice, where a slice's way from memory
// takes longer than its products: STAGES slices in LDS, all but the one being multiplied under way. As in
// DmaCore, the barrier sits before a slice's last part, after which the slice's stage is filled again. 1024 x 4096
// x 4096 23.5 us (two stages, DmaCore: 26.7), 256 x 8192 x 8192 32.8 (41).
template <int BM, int BN, int WM, int WN, bool PAIR, int STAGES_>
struct RingCore {
    using T = int8_t;
    using Map = WaveMap<BM, BN, WM, WN, 1>;
    using Sums = i32x16;
    static constexpr int STAGES = STAGES_, NT = Map::WAVES * 64, BI = WM / 32, BJ = WN / 32;
    static constexpr int STAGE = (BM + BN) * 128, LDS = STAGES * STAGE, PER_WAVE = LDS / Map::WAVES / 16 * 16;
    using FA = DmaFill<T, BM, NT, false>;
    using FB = DmaFill<T, BN, NT, false>;
    static constexpr int G = FA::G + FB::G;
    static_assert((STAGES - 1) * G < 64, "vmcnt counts them");

    template <class Src>
    __device__ __forceinline__ static void run(char* lds, int m0, int n0, int slices, Src&& src, i32x16 (&acc)[BI][BJ]) {
        const Map map;
        const int t = threadIdx.x, lane = map.lane;
#pragma unroll
        for (int i = 0; i < BI; ++i)
#pragma unroll
            for (int j = 0; j < BJ; ++j)
#pragma unroll
                for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
        FA fa;
        FB fb;
        {
            Lines<T> la, lb[2];
            src(0, la, lb);
            fa.template init<false>(&la, m0, t);
            fb.template init<PAIR>(lb, n0, t);
        }
        auto issue = [&](int s, char* st) {   // past the last slice: zeros, never used
            Lines<T> la, lb[2];
            const int k0 = src(s, la, lb);
            fa.template issue<false>(&la, m0, k0, t, st);
            fb.template issue<PAIR>(lb, n0, k0, t, st + BM * 128);
        };
        struct Frag {
            i32x4 a[BI], b[BJ];
        };
        auto read = [&](Frag& f, const char* st, int v) {
#pragma unroll
            for (int i = 0; i < BI; ++i) f.a[i] = read_frag<T, BM, false>(st, map.wm + 32 * i, lane, v);
#pragma unroll
            for (int j = 0; j < BJ; ++j) f.b[j] = read_frag<T, BN, false>(st + BM * 128, map.wn + 32 * j, lane, v);
        };
        auto mma = [&](const Frag& f) {
#pragma unroll
            for (int i = 0; i < BI; ++i)
#pragma unroll
                for (int j = 0; j < BJ; ++j) mma_chunk(T{}, f.b[j], f.a[i], acc[i][j]);
        };
        // Reads early among a part's matrix instructions, and a fill's loads behind those.
        auto weave = [&](auto loads) {
            constexpr int MFMA = 0x008, VMEM_READ = 0x020, DS_READ = 0x100, LOADS = decltype(loads)::value;
            constexpr int MFMAS = BI * BJ, READS = BI + BJ, RN = MFMAS > 2 ? MFMAS - 2 : 1, RS = (READS + RN - 1) / RN;
            constexpr int LS = LOADS == 0 ? 1 : MFMAS > 1 ? (LOADS + MFMAS - 2) / (MFMAS - 1) : LOADS;
#pragma unroll
            for (int i = 0; i < MFMAS; ++i) {
                __builtin_amdgcn_sched_group_barrier(MFMA, 1, 0);
                if (i * RS < READS) __builtin_amdgcn_sched_group_barrier(DS_READ, RS, 0);
                if (i * LS < LOADS) __builtin_amdgcn_sched_group_barrier(VMEM_READ, LS, 0);
            }
        };
#pragma unroll
        for (int i = 0; i < STAGES; ++i) issue(i, lds + i * STAGE);
        Frag f[2];
        ring_barrier<(STAGES - 1) * G>();
        read(f[0], lds, 0);
        int at = 0;
        for (int s = 0; s < slices; ++s) {
            char* const now = lds + at * STAGE;
            at = at == STAGES - 1 ? 0 : at + 1;
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                read(f[(p + 1) & 1], now, p + 1);
                mma(f[p & 1]);
                weave(std::integral_constant<int, 0>{});
                __builtin_amdgcn_sched_barrier(0);
            }
            ring_barrier<(STAGES - 2) * G>();
            read(f[0], lds + at * STAGE, 0);
            mma(f[1]);
            issue(s + STAGES, now);
            weave(std::integral_constant<int, G>{});
            __builtin_amdgcn_sched_barrier(0);
        }
        ring_barrier<0>();   // the loads past the last slice land before LDS is given up
    }
};
template <int BM_, int BN_, int WM_, int WN_, int STAGES_>
struct Ring {
    static constexpr int BM = BM_, BN = BN_, NT = (BM_ / WM_) * (BN_ / WN_) * 64;
    static constexpr bool ALONE = true;   // its LDS is the core's
    using Map = WaveMap<BM_, BN_, WM_, WN_, 1>;
    template <class T, bool, bool, bool PAIR>
    using Core = RingCore<BM_, BN_, WM_, WN_, PAIR, STAGES_>;
};

// Y or H, tile by tile, in an order that keeps a die's tiles next to each other. With tiles for every unit it is
// bound by the matrix cores: gated 4096 x 8192 x 4096 250 us (2.2 POP/s; counters show the cores busy for 62% of the units'
// cycles, at the 1.6 to 1.7 GHz the card holds under them), 8192^3 450 us (2.44 POP/s); through registers, 4000
// x 8001 x 4001 178 us (1.44 POP/s). With fewer, by the bytes of a lone tile's slices (RingCore).
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
    const int slices = (a.K + Elem<int8_t>::SLICE - 1) / Elem<int8_t>::SLICE;
    char* own;
    if constexpr (Tl::ALONE) {
        __shared__ __attribute__((aligned(16))) char lds[Core::LDS];
        Core::run(lds, m0, n0, slices, src, acc);
        own = lds + (threadIdx.x >> 6) * Core::PER_WAVE;
    } else {
        own = product<Core, Tl::DMA>(m0, n0, 0, slices, src, acc);
    }
    with_out(a, [&](auto* o) { put_i8<std::remove_pointer_t<decltype(o)>, Tl, Core, DUAL>(a, own, m0, n0, acc); });
}

// f(a null pointer of the type of the call's results).
template <class Fn>
__device__ __forceinline__ void with_out(const I8Args& a, Fn&& f) {
    if (a.dtype == SGEMM_F32_DTYPE_F32)
        f((float*)nullptr);
    else if (a.dtype == SGEMM_F32_DTYPE_BF16)
        f((bf16*)nullptr);
    else
        f((f16*)nullptr);
}

// Sums over the wave's 64 lanes, of four values at a time: lane 16 r + x ends with value r's.
__device__ __forceinline__ int lane_sums(int a, int b, int c, int d) {
    const auto ac = __builtin_amdgcn_permlane32_swap((uint32_t)a, (uint32_t)c, false, false);
    const auto bd = __builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)d, false, false);
    const auto r = __builtin_amdgcn_permlane16_swap(ac[0] + ac[1], bd[0] + bd[1], false, false);
    int v = (int)(r[0] + r[1]);
    v += moved<0xB1>(v);
    v += moved<0x4E>(v);
    v += moved<0x141>(v);
    return v + moved<0x140>(v);
}

// Very few rows, on the vector units (v_dot4_i32_i8): a workgroup takes FW features (FW weight rows, or
// 2 FW of two matrices) and up to MR rows of X, and its four waves take K's kibibytes of each in turn. Bound by
// the weights' bytes: one row of 8192 x 8192 11.4 us (67 MB, 5.9 TB/s, partly cached).
template <int MR, bool DUAL>
__global__ __launch_bounds__(256) void k_i8_few(I8Args a) {
    constexpr int FW = DUAL ? 2 : 4, STEP = 64 * 16;
    __shared__ int red[4][MR][4];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int f0 = blockIdx.x * FW, m0 = blockIdx.y * MR;
    const Lines<int8_t> lx = {a.X, a.ldx, a.M, a.K};
    const Lines<int8_t> lw[2] = {{a.W[0], a.ldw[0], a.F, a.K}, {a.W[1], a.ldw[1], a.F, a.K}};
    int acc[MR][4] = {};   // [row][weight row: DUAL 2 matrix + feature]
    for (int k0 = w * STEP; k0 < a.K; k0 += 4 * STEP) {
        const int at = k0 + lane * 16;
        i32x4 v[4], x[MR];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load_chunk<false>(lw[DUAL ? i >> 1 : 0], f0 + (DUAL ? i & 1 : i), at);
#pragma unroll
        for (int m = 0; m < MR; ++m) x[m] = load_chunk<false>(lx, m0 + m, at);
        // (what lies past K is zero in X; W's rows past F are another row's, and not kept)
        if (k0 + STEP > a.K) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = place_chunk<false>(v[i], lw[DUAL ? i >> 1 : 0], f0 + (DUAL ? i & 1 : i), at);
#pragma unroll
            for (int m = 0; m < MR; ++m) x[m] = place_chunk<false>(x[m], lx, m0 + m, at);
        }
#pragma unroll
        for (int m = 0; m < MR; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][i] = __builtin_amdgcn_sdot4(x[m][e], v[i][e], acc[m][i], false);
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        const int v = lane_sums(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
        if ((lane & 15) == 0) red[w][m][lane >> 4] = v;
    }
    __syncthreads();
    const int m = threadIdx.x / FW, f = threadIdx.x % FW;
    if (m < MR && m0 + m < a.M && f0 + f < a.F) {
        auto sum = [&](int i) { return red[0][m][i] + red[1][m][i] + red[2][m][i] + red[3][m][i]; };
        const Scale sx(a.Sx[m0 + m]);
        float g[1] = {scaled(sum(f), sx, Scale(a.Sw[0][f0 + f]))};
        const float u[1] = {DUAL ? scaled(sum(2 + f), sx, Scale(a.Sw[1][f0 + f])) : 0.0f};
        with_out(a, [&](auto* o) {
            using O = std::remove_pointer_t<decltype(o)>;
            if constexpr (DUAL) gate<O>(a.act, g, u);
            ((O*)a.Y)[(int64_t)(m0 + m) * a.ldy + f0 + f] = (O)g[0];
        });
    }
}

// Few rows: the weights' bytes are the work. A workgroup takes BM rows of X and BN weight rows (DUAL: of two
// matrices in blocks of 32); its KW waves take K's slices in turn, each with a ring of LDS stages of its own, so
// no wave waits for another before the sums are added. Bound by the weights' way to the units: 16 rows of 8192 x
// 8192 17.7 us (3.8 TB/s) cached and 18.2 from memory, where rows a power of two apart meet in the same few
// channels: with 128 bytes more between them 14.8 and 15.5; 64 of 4096 x 4096 6.8 and 8.8. Through registers, gated
// 33 of 4091 x 4092, 12.7.
constexpr int KW = 4;
template <int BM, int BN, bool DUAL, bool DMA>
__global__ __launch_bounds__(KW * 64) void k_i8_rows(I8Args a) {
    using T = int8_t;
    constexpr int BI = BM / 32, BJ = BN / 32, STAGE = (BM + BN) * 128;
    // Through registers one LDS stage a wave is enough: its own loads and reads of LDS stay in their order.
    constexpr int FIT = DMA ? 160 * 1024 / (KW * STAGE) : 1, SUMS = (BI * BJ * 16 * 64 * 4 + STAGE - 1) / STAGE;
    constexpr int STAGES = FIT > SUMS ? FIT : SUMS;
    static_assert(STAGES * STAGE >= BI * BJ * 16 * 64 * 4, "the sums fit in the rings");
    __shared__ __attribute__((aligned(16))) char lds[KW * STAGES * STAGE];
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int f0 = blockIdx.x * (DUAL ? BN / 2 : BN), m0 = blockIdx.y * BM;
    const int nslices = (a.K + Elem<T>::SLICE - 1) / Elem<T>::SLICE;
    const int count = nslices > w ? (nslices - w + KW - 1) / KW : 0;
    char* const ring = lds + w * (STAGES * STAGE);
    const Lines<T> x = {a.X, a.ldx, a.M, a.K};
    const Lines<T> wgt[2] = {{a.W[0], a.ldw[0], a.F, a.K}, {a.W[1], a.ldw[1], a.F, a.K}};
    i32x16 acc[BI][BJ];
#pragma unroll
    for (int i = 0; i < BI; ++i)
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
    auto compute = [&](const char* A) {
        const char* B = A + BM * 128;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            i32x4 b[BJ];
#pragma unroll
            for (int j = 0; j < BJ; ++j) b[j] = read_frag<T, BN, false>(B, 32 * j, lane, v);
#pragma unroll
            for (int i = 0; i < BI; ++i) {
                const i32x4 xv = read_frag<T, BM, false>(A, 32 * i, lane, v);
#pragma unroll
                for (int j = 0; j < BJ; ++j) mma_chunk(T{}, xv, b[j], acc[i][j]);
            }
        }
    };
    auto k_of = [&](int i) { return (w + KW * i) * Elem<T>::SLICE; };
    if constexpr (DMA) {
        DmaFill<T, BM, 64, false> fa;
        DmaFill<T, BN, 64, false> fb;
        fa.template init<false>(&x, m0, lane);
        fb.template init<DUAL>(wgt, f0, lane);
        auto issue = [&](int i, char* st) {   // slices past K read as zeros
            fa.template issue<false>(&x, m0, k_of(i), lane, st);
            fb.template issue<DUAL>(wgt, f0, k_of(i), lane, st + BM * 128);
        };
        constexpr int LOADS = (STAGES - 1) * (decltype(fa)::G + decltype(fb)::G);
        static_assert(LOADS < 64, "vmcnt counts them");
        if (count > 0) {
#pragma unroll
            for (int i = 0; i < STAGES - 1; ++i) issue(i, ring + i * STAGE);
            int at = 0;
            for (int i = 0; i < count; ++i) {
                const int to = at == 0 ? STAGES - 1 : at - 1;   // the stage read one slice ago
                lds_wait();
                issue(i + STAGES - 1, ring + to * STAGE);
                wave_wait<LOADS>();
                compute(ring + at * STAGE);
                at = at == STAGES - 1 ? 0 : at + 1;
            }
            wave_wait<0>();
        }
    } else if (count > 0) {
        FlatFill<BM, 64, false> fa;
        FlatFill<BN, 64, DUAL> fb;
        fa.init(&x, m0, lane);
        fb.init(wgt, f0, lane);
        i32x4 av[decltype(fa)::CH], bv[decltype(fb)::CH];
        fa.load(av, k_of(0), a.K);
        fb.load(bv, k_of(0), a.K);
        for (int i = 0; i < count; ++i) {
            fa.store(av, ring, k_of(i), a.K, lane);
            fb.store(bv, ring + BM * 128, k_of(i), a.K, lane);
            lanes_meet();
            const int next = k_of(i + 1 < count ? i + 1 : i);
            fa.load(av, next, a.K);
            fb.load(bv, next, a.K);
            compute(ring);
            lanes_meet();
        }
    }
    __syncthreads();
    int* const red = (int*)lds;
    constexpr int PER_WAVE = STAGES * STAGE / 4, OUTS = DUAL ? BJ / 2 : BJ;
#pragma unroll
    for (int i = 0; i < BI; ++i)
#pragma unroll
        for (int j = 0; j < BJ; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) red[w * PER_WAVE + ((i * BJ + j) * 16 + r) * 64 + lane] = acc[i][j][r];
    __syncthreads();
    // Each wave a share of the registers: lane l holds feature l % 32 of rows 8 (r / 4) + 4 (l / 32) + r % 4.
    constexpr int MINE = BI * 16 / KW;
    float g[MINE * OUTS], u[MINE * OUTS];
    auto row_of = [&](int o) {
        const int ir = w * MINE + o, r = ir & 15;
        return m0 + 32 * (ir >> 4) + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3);
    };
    Scale sw[DUAL ? 2 : 1][OUTS] = {};
#pragma unroll
    for (int j = 0; j < OUTS; ++j) {
        const int f = f0 + 32 * j + (lane & 31), at = f < a.F ? f : a.F - 1;
#pragma unroll
        for (int d = 0; d < (DUAL ? 2 : 1); ++d) sw[d][j] = Scale(a.Sw[d][at]);
    }
#pragma unroll
    for (int o = 0; o < MINE; ++o) {
        const int ir = w * MINE + o, i = ir >> 4, r = ir & 15, row = row_of(o);
        const Scale sx(a.Sx[row < a.M ? row : a.M - 1]);
        auto sum = [&](int j) {
            int v = 0;
#pragma unroll
            for (int ww = 0; ww < KW; ++ww) v += red[ww * PER_WAVE + ((i * BJ + j) * 16 + r) * 64 + lane];
            return v;
        };
#pragma unroll
        for (int j = 0; j < OUTS; ++j) {
            g[o * OUTS + j] = scaled(sum(DUAL ? 2 * j : j), sx, sw[0][j]);
            if (DUAL) u[o * OUTS + j] = scaled(sum(2 * j + 1), sx, sw[DUAL ? 1 : 0][j]);
        }
    }
    with_out(a, [&](auto* out) {
        using O = std::remove_pointer_t<decltype(out)>;
        if constexpr (DUAL) gate<O>(a.act, g, u);
#pragma unroll
        for (int o = 0; o < MINE; ++o)
#pragma unroll
            for (int j = 0; j < OUTS; ++j) {
                const int row = row_of(o), f = f0 + 32 * j + (lane & 31);
                if (row < a.M && f < a.F) ((O*)a.Y)[(int64_t)row * a.ldy + f] = (O)g[o * OUTS + j];
            }
    });
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

// Times that the choice of a kernel goes by, in microseconds, measured on MI355X with operands in the caches
// (products of 16 to 4096 rows, 300 to 8192 features and 777 to 8192 k): a call takes about
//     fixed + rounds * each + slices max(alone, rounds * busy)
// for `rounds` tiles on a compute unit, with `alone` a slice of 128 k where tiles are few and `busy` a tile's share
// of a unit's slice where every unit has one or more; a workgroup of the rows' kernel has its unit to itself, and its
// start and its sums (`each`) with it. What bounds a lone tile's slice is its bytes: a unit takes some 70
// GB/s from the caches, whatever is under way (two to eight slices a workgroup were level). Predictions are off
// by 15% on the average, and 10% short with weights from memory (22% up to 32 rows); of 104 products of random
// sizes the choice took 1.9% longer than the best kernel on the average with weights in the caches (at worst 32%)
// and 1.5% with weights from memory (24%).
struct Cost {
    double fixed, each, alone, busy;
    double of(int64_t tiles, int64_t slices) const {
        const double rounds = (double)((tiles + 255) / 256), b = rounds * busy;
        return fixed + rounds * each + (double)slices * (b > alone ? b : alone);
    }
};
// [filled through registers]
static const Cost kRows32[2] = {{1.0, 3.0, 0.12, 0.12}, {1.0, 2.5, 0.21, 0.22}};       // 32 x 32
static const Cost kRows64[2] = {{1.0, 3.0, 0.16, 0.165}, {1.0, 2.5, 0.32, 0.33}};      // 32 x 64
static const Cost kRows64x64 = {1.0, 3.0, 0.235, 0.235};                               // buffer-to-LDS
static const Cost kTile64 = {5.0, 0.0, 0.38, 0.42};                                    // 64 x 64, through registers
static const Cost kTile64x128[2] = {{5.0, 0.0, 0.33, 0.35}, {5.0, 0.0, 0.68, 0.70}};
static const Cost kTile128[2] = {{5.0, 0.0, 0.42, 0.60}, {5.0, 0.0, 0.85, 1.0}};
static const Cost kTileMid = {5.0, 0.0, 0.68, 0.55};                                   // 128 x 128, two workgroups a unit
static const Cost kTile256x128 = {6.0, 0.0, 1.45, 1.62};                               // through registers
static const Cost kTile256[2] = {{5.0, 0.0, 1.3, 1.95}, {7.0, 0.0, 2.2, 2.9}};

template <int MR, bool DUAL>
static hipError_t launch_few(const I8Args& a, hipStream_t s) {
    hipLaunchKernelGGL((k_i8_few<MR, DUAL>), dim3((unsigned)cdiv(a.F, DUAL ? 2 : 4), (unsigned)cdiv(a.M, MR)), dim3(256),
                       0, s, a);
    return hipGetLastError();
}
template <int BM, int BN, bool DUAL>
static hipError_t launch_rows(const I8Args& a, bool dma, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(a.F, DUAL ? BN / 2 : BN), (unsigned)cdiv(a.M, BM));
    if constexpr (BM == 32)
        if (!dma) {
            hipLaunchKernelGGL((k_i8_rows<BM, BN, DUAL, false>), grid, dim3(KW * 64), 0, s, a);
            return hipGetLastError();
        }
    hipLaunchKernelGGL((k_i8_rows<BM, BN, DUAL, true>), grid, dim3(KW * 64), 0, s, a);
    return hipGetLastError();
}

// The kernel of a call, and whether it is filled by buffer-to-LDS loads.
enum I8Kernel { FEW1, FEW2, FEW4, FEW8, ROWS32, ROWS64, ROWS64X64, TILE64, TILE64X128, TILE128, TILE_MID, TILE256X128,
                TILE256, TILE_SHORT, TILE_FAR };
struct I8Choice {
    I8Kernel kernel;
    bool dma;
};

static I8Choice choose(const I8Args& a, bool dual) {
    const bool dma = dma_ok(1, a.X, a.ldx, a.K, 256) && dma_ok(1, a.W[0], a.ldw[0], a.K, 256) &&
                     (!dual || dma_ok(1, a.W[1], a.ldw[1], a.K, 256));
    if (a.K < Elem<int8_t>::EPC) return {TILE_SHORT, false};
    const int64_t slices = cdiv(a.K, Elem<int8_t>::SLICE), cols = (dual ? 2 : 1) * (int64_t)a.F;
    // Very few rows, or few features: the vector units (in us, here against the rows' kernel: one row of
    // 8192 x 8192 12.3 and 16.7, eight 18.4 and 17.8, gated four 26.6 and 27.8, eight 33 and 27; 16
    // rows of 300 x 4096 3.6 and 5.7, of 1000 x 4096 5.0 and 5.9, 32 rows 6.4 and 6.2).
    if (cdiv(a.F, 2) <= max_workgroups(256) &&
        (a.M <= (dual ? 4 : 8) || (a.M <= 32 && cdiv(a.M, 8) * cols <= 4096)))
        return {a.M <= 1 ? FEW1 : a.M <= 2 ? FEW2 : a.M <= 4 ? FEW4 : FEW8, false};
    // Rows too far apart for offsets of 32 bits within a tile: 64-bit addresses.
    const int64_t far = (int64_t)kRange / 256;
    if (a.ldx >= far || a.ldw[0] >= far || (dual && a.ldw[1] >= far)) return {TILE_FAR, false};
    I8Kernel best = TILE256;
    double least = -1.0;
    auto offer = [&](I8Kernel id, const Cost& c, int64_t bm, int64_t bn) {
        const double t = c.of(cdiv(a.M, bm) * cdiv(cols, bn), slices);
        if (least < 0.0 || t < least) {
            best = id;
            least = t;
        }
    };
    const int reg = !dma;
    if (cdiv(a.M, 32) <= 65535) {   // their blocks of rows are the grid's second extent
        if (!dual) offer(ROWS32, kRows32[reg], 32, 32);
        offer(ROWS64, kRows64[reg], 32, 64);
        if (dma) offer(ROWS64X64, kRows64x64, 64, 64);
    }
    if (!dma) offer(TILE64, kTile64, 64, 64);
    offer(TILE64X128, kTile64x128[reg], 64, 128);
    offer(TILE128, kTile128[reg], 128, 128);
    if (dma) offer(TILE_MID, kTileMid, 128, 128);
    if (!dma) offer(TILE256X128, kTile256x128, 256, 128);
    offer(TILE256, kTile256[reg], 256, 256);
    return {best, dma};
}

const char* i8_kernel_name(const I8Args& a, bool dual) {
    if (a.K == 0) return "zero";
    const I8Choice c = choose(a, dual);
    switch (c.kernel) {
        case FEW1: return "few 1";
        case FEW2: return "few 2";
        case FEW4: return "few 4";
        case FEW8: return "few 8";
        case ROWS32: return c.dma ? "rows 32x32" : "rows 32x32 through registers";
        case ROWS64: return c.dma ? "rows 32x64" : "rows 32x64 through registers";
        case ROWS64X64: return "rows 64x64";
        case TILE64: return "flat 64x64";
        case TILE64X128: return c.dma ? "ring 64x128" : "flat 64x128";
        case TILE128: return c.dma ? "ring 128x128" : "flat 128x128";
        case TILE_MID: return "tile 128x128";
        case TILE256X128: return "flat 256x128";
        case TILE256: return c.dma ? "tile 256x256" : "flat 256x256";
        case TILE_SHORT: return "tile 128x128 of short rows";
        default: return "tile 64x64 of far rows";
    }
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
    const auto [kernel, dma] = choose(a, DUAL);
    switch (kernel) {
        case FEW1: return launch_few<1, DUAL>(a, s);
        case FEW2: return launch_few<2, DUAL>(a, s);
        case FEW4: return launch_few<4, DUAL>(a, s);
        case FEW8: return launch_few<8, DUAL>(a, s);
        case ROWS32:
            if constexpr (!DUAL) return launch_rows<32, 32, DUAL>(a, dma, s);
        case ROWS64: return launch_rows<32, 64, DUAL>(a, dma, s);
        case ROWS64X64: return launch_rows<64, 64, DUAL>(a, dma, s);
        case TILE64: return go(TypeTag<Flat<64, 64, 32, 64, 2, 2>>{});
        case TILE64X128: return dma ? go(TypeTag<Ring<64, 128, 32, 64, 3>>{}) : go(TypeTag<Flat<64, 128, 32, 64>>{});
        case TILE128: return dma ? go(TypeTag<Ring<128, 128, 32, 64, 4>>{}) : go(TypeTag<Flat<128, 128, 32, 64>>{});
        case TILE_MID: return go(TypeTag<TileMid>{});
        case TILE256X128: return go(TypeTag<Flat<256, 128, 64, 64>>{});
        case TILE256: return dma ? go(TypeTag<TileBig>{}) : go(TypeTag<Flat<256, 256, 128, 64>>{});
        case TILE_SHORT: return go(TypeTag<TileShort>{});
        default: return go(TypeTag<TileReg64>{});
    }
}

hipError_t launch_i8(const I8Args& a, bool dual, hipStream_t s) {
    if (a.K == 0) {
        hipLaunchKernelGGL(k_i8_zero, dim3((unsigned)cdiv((int64_t)a.M * a.F, 256)), dim3(256), 0, s, a);
        return hipGetLastError();
    }
    return dual ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace sgemm

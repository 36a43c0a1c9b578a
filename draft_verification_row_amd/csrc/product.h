// product.h -- the tiled matrix product under the operators that train a head:
// out[m][n] = sum_k X[m][k] W[n][k], finished by an epilogue of the operator's
// own.  Either operand may lie with k along its rows ("by rows": X[m][k]) or
// down them ("by k": X[k][m]), so that no gradient needs a turned copy.
#ifndef SPEC_PRODUCT_H
#define SPEC_PRODUCT_H

#include "tiles.h"

namespace {

struct Product {
    const void *x[2], *w[2];  // [1]: of a second sum over k, a second product, or a pair's other matrix
    int64_t ldx, ldw;         // elements from row to row, or from k to k
    int M, N, K;
    int K2;                   // length of a second sum that is added to the first, or 0
    const int *live_m, *live_k;  // on the device: the count that stands for M, or for K, or null
    int products;             // 1, or 2: x[0] and x[1] with the same w
    int splits;               // of the sum over k
    int more;                 // with live_m: splits where few rows are in use, or 0
};
// The splits where `tiles` of a workgroup each are in use: enough of them for a
// compute unit each, as far as there is room for their sums.
__host__ __device__ inline int splits_in_use(int splits, int more, unsigned tiles) {
    const int want = tiles ? (int)(256 / tiles) : 1;
    return want <= splits ? splits : want < more ? want : more > splits ? more : splits;
}

// One tile's shape.  XK, WK: the operand lies by k.  PAIR: w[0] and w[1] are
// multiplied side by side, BN / 2 rows of each, every wave with the same rows of
// both.  DIRECT: 16-byte aligned rows, loaded straight to LDS.  ONCE: W is read
// once and not to be kept in the caches.
template <typename T_, int BM_, int BN_, int WM_, int WN_, int STAGES_, bool XK_, bool WK_, bool PAIR_, bool DIRECT_, bool ONCE_ = false>
struct Tile {
    using T = T_;
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_;
    static constexpr bool XK = XK_, WK = WK_, PAIR = PAIR_, DIRECT = DIRECT_, ONCE = ONCE_;
    static constexpr int kElems = 16 / (int)sizeof(T), kStep = 8 * kElems;  // k of a stage: 128 bytes of a row
    // a block of the result and of the matrix instructions: kB x kB
    static constexpr int kB = BM == 256 && sizeof(T) == 2 ? 16 : 32, kV = kB * kB / 64;
    using Acc = std::conditional_t<kB == 16, f32x4, f32x16>;  // a lane's kV values of one
    static constexpr int FM = WM / kB, FN = WN / kB, kWavesM = BM / WM, kWavesN = BN / WN;
    static constexpr int kColsN = PAIR ? BN / 2 : BN;  // columns of the result
    static constexpr int kWaveN = PAIR ? WN / 2 : WN;
    static constexpr int kStageBytes = (BM + BN) * 128;
    static_assert(kWavesM * kWavesN == kThreads / 64, "four waves");
    static_assert(!PAIR || (WN >= 64 && !WK), "whole blocks of each of a pair");
};

// How an operand of B rows lies in a stage: 128 bytes of k of each row, or k
// after k of B elements.  A load is 1 KiB, lane after lane 16 bytes.  Chunks
// are exchanged within their row so that the reads of an instruction's operand
// use each bank once: by rows, sixteen rows are read at one chunk; by k in
// bf16, four k of 64 neighbouring bytes at once, or (SIXTEEN) four and four k
// that are eight apart of 32 bytes; in fp32, 128 bytes of two k that are four
// apart.
template <typename T, int B, bool K, bool SIXTEEN = false>
struct Lies {
    static constexpr int kRowBytes = K ? B * (int)sizeof(T) : 128, kRowChunks = kRowBytes / 16;
    static constexpr int kRows = 64 / kRowChunks, kLoads = B / 32;
    static_assert(kRows * kRowChunks == 64, "whole rows a load");
    __device__ static int row(int i, int w, int lane) { return (i * 4 + w) * kRows + lane / kRowChunks; }
    __device__ static int swizzle(int r) {
        if constexpr (!K) return r >> 1 & 7;
        else if constexpr (sizeof(T) == 2) return SIXTEEN ? ((r & 3) | (r >> 3 & 1) << 2) << 1 : kRowBytes >= 256 ? (r & 3) << 2 : kRowBytes == 128 ? (r >> 1 & 1) << 2 : 0;
        else return kRowBytes >= 256 ? (r >> 2 & 1) << 3 : 0;
    }
    __device__ static int chunk(int i, int w, int lane) { return lane % kRowChunks ^ swizzle(row(i, w, lane)); }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// The chunk pair's operand of 32 rows from r0 on: lane l has row r0 + l % 32 and
// chunk 2 pair + l / 32.  A stage that lies by k is read turned: in bf16 by the
// LDS's own transposing reads, four k of sixteen rows to a group of lanes.
template <typename T, int B, bool K>
__device__ inline u32x4 operand(const char* at, int pair, int r0, int lane) {
    using L = Lies<T, B, K>;
    const int l = lane & 31, h = lane >> 5;
    if constexpr (!K) {
        return *reinterpret_cast<const u32x4*>(at + (r0 + l) * 128 + ((2 * pair + h) ^ L::swizzle(l)) * 16);
    } else if constexpr (sizeof(T) == 2) {
        const int k = (lane & 15) >> 2;
        const char* p = at + ((2 * pair + h) * 8 + k) * L::kRowBytes + (r0 * 2 ^ L::swizzle(k) * 16) + (lane >> 4 & 1) * 32 + (lane & 3) * 8;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + 4 * L::kRowBytes));
        const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
        return (u32x4){x[0], x[1], y[0], y[1]};
    } else {
        const char* p = at + (2 * pair + h) * 4 * L::kRowBytes + ((r0 + l) * 4 ^ L::swizzle(4 * h) * 16);
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const uint32_t*>(p + i * L::kRowBytes);
        return q;
    }
}

// The same of 16 rows, for a bf16 instruction of 32 k: lane l has row r0 + l % 16
// and chunk 4 step + l / 16.
template <int B, bool K>
__device__ inline u32x4 operand16(const char* at, int step, int r0, int lane) {
    using L = Lies<bf16, B, K, true>;
    const int l = lane & 15, h = lane >> 4;
    if constexpr (!K) {
        return *reinterpret_cast<const u32x4*>(at + (r0 + l) * 128 + ((4 * step + h) ^ L::swizzle(l)) * 16);
    } else {
        const int k = h * 8 + (l >> 2);
        const char* p = at + (step * 32 + k) * L::kRowBytes + (r0 * 2 ^ L::swizzle(k) * 16) + (l & 3) * 8;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + 4 * L::kRowBytes));
        const u32x2 x = __builtin_bit_cast(u32x2, a), y = __builtin_bit_cast(u32x2, b);
        return (u32x4){x[0], x[1], y[0], y[1]};
    }
}

// Where a wave's part of the result lies.
struct Part {
    int m0, n0;       // its first row and column
    int M, N;         // of the whole result
    int lane, w;      // of the workgroup's waves
    int tm, tn;       // the workgroup's tile
    int split, product;
    char* lds;        // the workgroup's, free to use
};

// What the wave's lanes wrote to the LDS is there for all of them.  The barrier
// emits nothing, but keeps the lanes together: without it the compiler may let
// those that skip the reads run ahead to the next writes.
__device__ __attribute__((always_inline)) inline void settle() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// A wave's blocks of the j-th 32 rows of m, laid in its own part of the LDS so
// that neighbouring lanes may take neighbouring n: row r at rows + r * (WN + 4).
template <class C>
__device__ inline float* rows_of(const Part& p) {
    static_assert(4 * 32 * (C::WN + 4) * 4 <= C::STAGES * C::kStageBytes, "the rows fit");
    return reinterpret_cast<float*>(p.lds) + p.w * 32 * (C::WN + 4);
}
template <class C, class J>
__device__ __attribute__((always_inline)) inline void lay(const Part& p, typename C::Acc (&acc)[C::FN][C::FM], J j) {
    constexpr int kFours = C::kV / 4, kBlocks = 32 / C::kB;
    float* rows = rows_of<C>(p) + p.lane % C::kB * (C::WN + 4) + p.lane / C::kB * 4;
    each(std::make_integer_sequence<int, kBlocks * C::FN * kFours>(), [&](auto u) __attribute__((always_inline)) {
        constexpr int k = u / (C::FN * kFours), i = u / kFours % C::FN, q = u % kFours, jj = j * kBlocks + k;
        *reinterpret_cast<f32x4*>(rows + k * C::kB * (C::WN + 4) + i * C::kB + q * 8) =
            (f32x4){acc[i][jj][4 * q], acc[i][jj][4 * q + 1], acc[i][jj][4 * q + 2], acc[i][jj][4 * q + 3]};
    });
    settle();
}
// All of them in turn: f(j, rows).
template <class C, typename F>
__device__ __attribute__((always_inline)) inline void turned(const Part& p, typename C::Acc (&acc)[C::FN][C::FM], F f) {
    each(std::make_integer_sequence<int, C::WM / 32>(), [&](auto j) __attribute__((always_inline)) {
        lay<C>(p, acc, j);
        f(j, rows_of<C>(p));
        settle();
    });
}

// The product.  E::start<C>(part, acc) may set what the sums start from, and
// E::finish<C>(part, acc) takes each wave's sums: acc[i][j] is a block of kB x kB,
// lane l with row l % kB of m, value 4 q + r with column 8 q + 4 (l / kB) + r of
// n.
template <class C, class E>
__global__ __launch_bounds__(kThreads, C::kStageBytes * C::STAGES <= 80 * 1024 ? 2 : 1) void k_product(Product g, E e) {
    using T = typename C::T;
    using LX = Lies<T, C::BM, C::XK>;
    using LW = Lies<T, C::BN, C::WK>;
    constexpr int BM = C::BM, BN = C::BN, FM = C::FM, FN = C::FN, STAGES = C::STAGES;
    constexpr int kElems = C::kElems, kStep = C::kStep, kLoadsW = LW::kLoads, kLoads = kLoadsW + LX::kLoads;
    constexpr int kStageBytes = C::kStageBytes;
    __shared__ __attribute__((aligned(1024))) char lds[STAGES][kStageBytes];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int M = g.live_m ? __builtin_amdgcn_readfirstlane(*g.live_m) : g.M;
    const int K = g.live_k ? __builtin_amdgcn_readfirstlane(*g.live_k) : g.K;
    const unsigned tiles_m = (M + BM - 1) / BM, tiles_n = (g.N + C::kColsN - 1) / C::kColsN, tiles = tiles_m * tiles_n;
    const int splits = splits_in_use(g.splits, g.more, tiles);
    if (blockIdx.x >= tiles * (unsigned)(splits * g.products)) return;
    const int turn = blockIdx.x / tiles, split = turn % splits, product = turn / splits;
    int tm, tn;
    tile_of(blockIdx.x % tiles, tiles, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * C::kColsN;
    const int wm = w / C::kWavesN * C::WM, wn = w % C::kWavesN * C::WN;

    // The order of the sum's steps: the whole ones of both sums, then what is
    // left of each.  This split's are [begin, end).
    const int whole1 = K / kStep, whole = whole1 + g.K2 / kStep;
    const int rest1 = K % kStep != 0, steps = whole + rest1 + (g.K2 % kStep != 0);
    const int per = (steps + splits - 1) / splits, begin = split * per, end = min(steps, begin + per);
    auto second = [&](int s) { return s < whole ? s >= whole1 : s >= whole + rest1; };
    auto k_of = [&](int s) {
        if (s < whole) return (s < whole1 ? s : s - whole1) * kStep;
        return (second(s) ? g.K2 : K) / kStep * kStep;
    };
    // row r of W's part of a stage: which matrix of a pair, and its column n
    auto pair_of = [](int r) { return C::PAIR && r % C::WN >= C::kWaveN; };
    auto col_of = [](int r) { return C::PAIR ? r / C::WN * C::kWaveN + r % C::kWaveN : r; };
    // both sums' operands from this tile's first row and column on
    const int64_t xm = C::XK ? m0 : m0 * g.ldx, wn0 = C::WK ? n0 : n0 * g.ldw;
    const T* const x1 = static_cast<const T*>(product ? g.x[1] : g.x[0]) + xm;
    const T* const x2 = static_cast<const T*>(g.x[1]) + xm;
    const T* const w1 = static_cast<const T*>(g.w[0]) + wn0;
    const T* const w2 = static_cast<const T*>(g.w[1]) + wn0;
    auto x_at = [&](int s) { return (second(s) ? x2 : x1) + (C::XK ? k_of(s) * g.ldx : k_of(s)); };
    auto w_at = [&](int s, bool other) { return ((C::PAIR ? other : second(s)) ? w2 : w1) + (C::WK ? k_of(s) * g.ldw : k_of(s)); };

    // offsets of this lane's loads; what lies past the matrix reads a row or
    // column that does not: those sums are dropped
    uint32_t off[C::DIRECT ? kLoads : 1];
    if constexpr (C::DIRECT)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            int64_t at;
            if (i < kLoadsW) {
                const int r = LW::row(i, w, lane), c = LW::chunk(i, w, lane);
                at = C::WK ? r * g.ldw + (c * kElems < g.N - n0 ? c * kElems : 0) : min(col_of(r), g.N - 1 - n0) * g.ldw + c * kElems;
            } else {
                const int r = LX::row(i - kLoadsW, w, lane), c = LX::chunk(i - kLoadsW, w, lane);
                at = C::XK ? r * g.ldx + (c * kElems < M - m0 ? c * kElems : 0) : min(r, M - 1 - m0) * g.ldx + c * kElems;
            }
            off[i] = (uint32_t)(at * (int64_t)sizeof(T));
        }
    // loads [FROM, TO) of a whole step into a stage
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)&lds[0][0] + w * 1024;
    auto rsrc_of = [](const T* p) { return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), (short)0, 0x7fffffff, 0x00020000); };
    auto load_direct = [&](int stage, int s, auto from, auto to) {
        if constexpr (C::DIRECT) {
            const uint32_t base = lds0 + stage * kStageBytes;
            const __amdgpu_buffer_rsrc_t rx = rsrc_of(x_at(s)), rw = rsrc_of(w_at(s, false)), rp = rsrc_of(w_at(s, C::PAIR));
            each(std::make_integer_sequence<int, kLoads>(), [&](auto i) {
                if constexpr (i >= from && i < to) {
                    if constexpr (i >= kLoadsW)
                        to_lds<i * 4096, false>(rx, base, off[i], 0);
                    else if constexpr (C::PAIR && i * 32 % C::WN >= C::kWaveN)
                        to_lds<i * 4096, C::ONCE>(rp, base, off[i], 0);
                    else
                        to_lds<i * 4096, C::ONCE>(rw, base, off[i], 0);
                }
            });
        }
    };
    using Zero = std::integral_constant<int, 0>;
    using All = std::integral_constant<int, kLoads>;
    // any step through registers, at any alignment, zero past the sum's end
    auto fetch = [&](int s, u32x4 (&q)[kLoads]) {
        const int left = (second(s) ? g.K2 : K) - k_of(s);
        const T *px = x_at(s), *pw[2] = {w_at(s, false), w_at(s, C::PAIR)};
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const bool x = i >= kLoadsW;
            const int r = x ? LX::row(i - kLoadsW, w, lane) : LW::row(i, w, lane);
            const int c = (x ? LX::chunk(i - kLoadsW, w, lane) : LW::chunk(i, w, lane)) * kElems;
            const int64_t ld = x ? g.ldx : g.ldw;
            const int rows = x ? M - m0 : g.N - n0;
            if (x ? C::XK : C::WK) {
                q[i] = (u32x4){0, 0, 0, 0};
                if (r < left) q[i] = chunk_of((x ? px : pw[0]) + r * ld, c, rows);
            } else {
                const T* p = x ? px + min(r, rows - 1) * ld : pw[pair_of(r)] + min(col_of(r), rows - 1) * ld;
                q[i] = chunk_of(p, c, left);
            }
        }
    };
    auto place = [&](int stage, const u32x4 (&q)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) *reinterpret_cast<u32x4*>(&lds[stage][(i * 4 + w) * 1024 + lane * 16]) = q[i];
    };

    const Part part{m0 + wm, n0 + w % C::kWavesN * C::kWaveN, M, g.N, lane, w, tm, tn, split, product, &lds[0][0]};
    typename C::Acc acc[FN][FM] = {};
    e.template start<C>(part, acc);
    // Operands of one pair of chunks, read from LDS a pair ahead of their use.
    constexpr int kPairs = 4, kProducts = FN * FM, kReads = FN + FM;
    struct Operands {
        u32x4 a[FN], b[FM];
    };
    Operands f[2];
    auto read = [&](int stage, int pair, int i, Operands& o) {
        const char* at = &lds[0][0] + stage * kStageBytes;
        if (i < FM)
            o.b[i] = operand<T, BM, C::XK>(at + BN * 128, pair, wm + i * 32, lane);
        else
            o.a[i - FM] = operand<T, BN, C::WK>(at, pair, wn + (i - FM) * 32, lane);
    };
    // The products of one pair, with `between` called for each before it: the
    // order is kept, so that reads and loads sit under the products.
    auto multiply = [&](const Operands& o, auto&& between) {
        each(std::make_integer_sequence<int, kProducts>(), [&](auto i) {
            between(i);
            acc[i / FM][i % FM] = mfma32(T(), o.a[i / FM], o.b[i % FM], acc[i / FM][i % FM]);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // the next pair's operands are read under the first products
    auto read_under = [&](auto i, int stage, int pair, Operands& o) {
        constexpr int from = kProducts > kReads ? (i < kReads ? i : kReads) : i * kReads / kProducts;
        constexpr int to = kProducts > kReads ? (i + 1 < kReads ? i + 1 : kReads) : (i + 1) * kReads / kProducts;
#pragma unroll
        for (int r = from; r < to; ++r) read(stage, pair, r, o);
    };

    int s = begin;
    if constexpr (C::DIRECT) {
        const int stop = min(end, whole), full = max(0, stop - begin);
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
            if (i < full) load_direct(i, begin + i, Zero(), All());
        if (full >= STAGES)
            asm volatile("s_waitcnt vmcnt(%0)" :: "n"(kLoads * (STAGES - 1)) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        int slot = 0;
        // All but the last pair of a stage.  LOADS: with the second half of the
        // loads of `step` into the stage that was freed last.
        auto inner = [&](auto loads, int freed, int step) {
            each(std::make_integer_sequence<int, kPairs - 1>(), [&](auto p) {
                multiply(f[p & 1], [&](auto i) {
                    read_under(i, slot, p + 1, f[(p + 1) & 1]);
                    if constexpr (loads && p == 0) {
                        constexpr int h = kLoads / 2, m = kLoads - h;
                        load_direct(freed, step, std::integral_constant<int, h + i * m / kProducts>(),
                                    std::integral_constant<int, h + (i + 1) * m / kProducts>());
                    }
                });
            });
        };
        // A stage's last pair and the next stage's others.  Before it the next
        // stage's loads have arrived, in every wave, and every wave has this
        // stage's last operands, so that it can be filled anew: half of the
        // loads under this pair, half under the next.
        auto advance = [&](auto loads, int step) {
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            const int freed = slot;
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            multiply(f[1], [&](auto i) {
                read_under(i, slot, 0, f[0]);
                if constexpr (loads) {
                    constexpr int h = kLoads / 2;
                    load_direct(freed, step, std::integral_constant<int, i * h / kProducts>(),
                                std::integral_constant<int, (i + 1) * h / kProducts>());
                }
            });
            inner(loads, freed, step);
        };
        if (full > 0) {
#pragma unroll
            for (int i = 0; i < kReads; ++i) read(0, 0, i, f[0]);
            inner(std::false_type(), 0, 0);
            int n = STAGES;
            for (; n < full; ++n) {
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(kLoads * (STAGES - 2)) : "memory");
                advance(std::true_type(), begin + n);
            }
            for (n = n - STAGES + 1; n < full; ++n) {
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                advance(std::false_type(), 0);
            }
            multiply(f[1], [](auto) {});
            s = stop;
        }
    }
    // what is no whole step, or not aligned: the next step's loads are on
    // their way while one is worked on
    if (s < end) {
        u32x4 q[kLoads];
        fetch(s, q);
        for (; s < end; ++s) {
            __syncthreads();
            place(0, q);
            __syncthreads();
            if (s + 1 < end) fetch(s + 1, q);
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
#pragma unroll
                for (int i = 0; i < kReads; ++i) read(0, p, i, f[0]);
                multiply(f[0], [](auto) {});
            }
        }
    }
    __syncthreads();
    e.template finish<C>(part, acc);
}

// ------------------------------------------------------------- the large tile
// 256 x 256 outputs of four waves, 128 x 128 each, one wave a SIMD: nothing but
// its own order hides what a wave waits for.  A stage is four quarters of 128
// rows each, the first and the second halves of every wave's rows of X (A0, A1)
// and of W (B0, B1); in a pair, B0 is the one matrix and B1 the other.  A stage's
// products go by quadrants, A0 B0, A0 B1, A1 B1, A1 B0, each quarter read to
// registers once, under the quadrant before its first: so a quarter's place in
// LDS is free half a stage or more before the stage ends, its next loads go out
// evenly over the whole of the stage, and each has at least a stage's time
// (2048 cycles) to arrive.  On zeros 8192 x 32768 x 8192 bf16 so reaches 1988
// TFLOP/s with 32x32x16 instructions, where one stage after the other reached
// 1676.  On normal values power bounds the clock, and instructions of 16x16x32,
// which move half the accumulators for the same products, are faster: 1680 ->
// 1625 us for 8192 x 32768 x 4096, and 1% more with the order below.
template <class C, class E>
__global__ __launch_bounds__(kThreads, 1) void k_wide(Product g, E e) {
    using T = typename C::T;
    static_assert(C::BM == 256 && C::BN == 256 && C::WM == 128 && C::WN == 128 && C::DIRECT, "the large tile");
    using LX = Lies<T, 128, C::XK, C::kB == 16>;
    using LW = Lies<T, 128, C::WK, C::kB == 16>;
    constexpr int kElems = C::kElems, kStep = C::kStep, kQuarter = 128 * 128, kLoads = 16;
    enum { A0, B0, B1, A1 };  // in the order of their loads
    __shared__ __attribute__((aligned(1024))) char lds[2][4 * kQuarter];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int M = g.live_m ? __builtin_amdgcn_readfirstlane(*g.live_m) : g.M;
    const int K = g.live_k ? __builtin_amdgcn_readfirstlane(*g.live_k) : g.K;
    const unsigned tiles_m = (M + 255) / 256, tiles_n = (g.N + C::kColsN - 1) / C::kColsN, tiles = tiles_m * tiles_n;
    const int splits = splits_in_use(g.splits, g.more, tiles);
    if (blockIdx.x >= tiles * (unsigned)(splits * g.products)) return;
    const int turn = blockIdx.x / tiles, split = turn % splits, product = turn / splits;
    int tm, tn;
    tile_of(blockIdx.x % tiles, tiles, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * 256, n0 = tn * C::kColsN;

    // the order of the sum's steps, as in k_product
    const int whole1 = K / kStep, whole = whole1 + g.K2 / kStep;
    const int rest1 = K % kStep != 0, steps = whole + rest1 + (g.K2 % kStep != 0);
    const int per = (steps + splits - 1) / splits, begin = split * per, end = min(steps, begin + per);
    auto second = [&](int s) { return s < whole ? s >= whole1 : s >= whole + rest1; };
    auto k_of = [&](int s) {
        if (s < whole) return (s < whole1 ? s : s - whole1) * kStep;
        return (second(s) ? g.K2 : K) / kStep * kStep;
    };
    // row r of a quarter of X or W among the tile's rows
    auto row_x = [](int q, int r) { return r / 64 * 128 + (q == A1) * 64 + r % 64; };
    auto row_w = [](int q, int r) { return C::PAIR ? r : r / 64 * 128 + (q == B1) * 64 + r % 64; };
    const int64_t xm = C::XK ? m0 : m0 * g.ldx, wn = C::WK ? n0 : n0 * g.ldw;
    const T* const x1 = static_cast<const T*>(product ? g.x[1] : g.x[0]) + xm;
    const T* const x2 = static_cast<const T*>(g.x[1]) + xm;
    const T* const w1 = static_cast<const T*>(g.w[0]) + wn;
    const T* const w2 = static_cast<const T*>(g.w[1]) + wn;
    auto from = [&](int q, int s) -> const T* {
        if (q == A0 || q == A1) return (second(s) ? x2 : x1) + (C::XK ? k_of(s) * g.ldx : k_of(s));
        return ((C::PAIR ? q == B1 : second(s)) ? w2 : w1) + (C::WK ? k_of(s) * g.ldw : k_of(s));
    };

    // offsets of this lane's loads, four a quarter; what lies past the matrix
    // reads a row or column that does not: those sums are dropped
    uint32_t off[kLoads];
    each(std::make_integer_sequence<int, kLoads>(), [&](auto i) {
        constexpr int q = i / 4, u = i % 4;
        int64_t at;
        if constexpr (q == A0 || q == A1) {
            const int r = LX::row(u, w, lane), c = LX::chunk(u, w, lane) * kElems;
            if constexpr (C::XK)
                at = r * g.ldx + (row_x(q, c) < M - m0 ? row_x(q, c) : 0);
            else
                at = min(row_x(q, r), M - 1 - m0) * g.ldx + c;
        } else {
            const int r = LW::row(u, w, lane), c = LW::chunk(u, w, lane) * kElems;
            if constexpr (C::WK)
                at = r * g.ldw + (row_w(q, c) < g.N - n0 ? row_w(q, c) : 0);
            else
                at = min(row_w(q, r), g.N - 1 - n0) * g.ldw + c;
        }
        off[i] = (uint32_t)(at * (int64_t)sizeof(T));
    });
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)&lds[0][0] + w * 1024;
    const int stop = min(end, whole);
    // a whole step's buffers; past the last step they have no length, and their
    // loads nothing to load
    struct Buffers {
        __amdgpu_buffer_rsrc_t x, w, p;
    };
    auto buffers = [&](int s) -> Buffers {
        const bool sec = s >= whole1;
        const int64_t k = (int64_t)(sec ? s - whole1 : s) * kStep;
        auto rsrc = [&](const T* p) { return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), (short)0, s < stop ? 0x7fffffff : 0, 0x00020000); };
        const int64_t kx = C::XK ? k * g.ldx : k, kw = C::WK ? k * g.ldw : k;
        if constexpr (C::PAIR) return {rsrc(x1 + kx), rsrc(w1 + kw), rsrc(w2 + kw)};
        const __amdgpu_buffer_rsrc_t w = rsrc((sec ? w2 : w1) + kw);
        return {rsrc((sec ? x2 : x1) + kx), w, w};
    };
    auto load = [&](int slot, auto i, const Buffers& f) {
        constexpr int q = i / 4;
        to_lds<i * 4096, false>(q == A0 || q == A1 ? f.x : q == B0 ? f.w : f.p, lds0 + slot * 4 * kQuarter, off[i], 0);
    };

    const Part part{m0 + w / 2 * 128, n0 + w % 2 * C::kWaveN, M, g.N, lane, w, tm, tn, split, product, &lds[0][0]};
    typename C::Acc acc[C::FN][C::FM] = {};
    e.template start<C>(part, acc);
    // A quarter's operands: kHalf blocks, of each the parts of a stage's k.  b2:
    // the next B0, read while b0 is still in use.
    constexpr int kHalf = C::FM / 2, kParts = 8 / kHalf, kProducts = kHalf * kHalf * kParts;
    u32x4 a0[8], a1[8], b0[8], b1[8], b2[8];
    auto read = [&](int slot, int q, int i, u32x4 (&o)[8]) {
        const char* at = &lds[slot][q * kQuarter];
        const bool x = q == A0 || q == A1;
        const int r0 = (x ? w / 2 : w % 2) * 64 + i % kHalf * C::kB;
        if constexpr (C::kB == 16)
            o[i] = x ? operand16<128, C::XK>(at, i / kHalf, r0, lane) : operand16<128, C::WK>(at, i / kHalf, r0, lane);
        else
            o[i] = x ? operand<T, 128, C::XK>(at, i / kHalf, r0, lane) : operand<T, 128, C::WK>(at, i / kHalf, r0, lane);
    };
    // A quadrant's products, each with an operand of the one before; `between` is
    // called before every sixteenth of them.
    auto quadrant = [&](auto i0, auto j0, const u32x4 (&wq)[8], const u32x4 (&xq)[8], auto&& between) {
        each(std::make_integer_sequence<int, kProducts>(), [&](auto u) {
            constexpr int p = u / (kHalf * kHalf), i = i0 * kHalf + u / kHalf % kHalf, j = j0 * kHalf + (u / kHalf % 2 ? kHalf - 1 - u % kHalf : u % kHalf), each16 = kProducts / 16;
            if constexpr (u % each16 == 0) between(std::integral_constant<int, u / each16>());
            const u32x4 &a = wq[p * kHalf + i % kHalf], &b = xq[p * kHalf + j % kHalf];
            if constexpr (C::kB == 16)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc[i][j], 0, 0, 0);
            else
                acc[i][j] = mfma32(T(), a, b, acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    using Zero = std::integral_constant<int, 0>;
    using One = std::integral_constant<int, 1>;
    auto arrived = [&](auto left) {  // all but the last `left` loads, in every wave; and every wave has read what it asked for
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"((int)left) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // The sums stay where they are, whatever comes before or after would rather
    // have: else the compiler moves some of them about in the loop.
    auto pin = [&] {
        each(std::make_integer_sequence<int, C::FN * C::FM>(), [&](auto i) {
            auto& v = acc[i / C::FM][i % C::FM];
            asm volatile("" : "+a"(v));
        });
    };
    int s = begin;
    if (s < stop) {
        pin();
        each(std::make_integer_sequence<int, kLoads>(), [&](auto i) { load(0, i, buffers(s)); });
        each(std::make_integer_sequence<int, kLoads>(), [&](auto i) { load(1, i, buffers(s + 1)); });
        arrived(std::integral_constant<int, 24>());
#pragma unroll
        for (int i = 0; i < 8; ++i) read(0, A0, i, a0), read(0, B0, i, b2);
        int slot = 0;
        // a stage: step s + 2 is loaded into its place, a load every fourth product
        do {
            using Left = std::integral_constant<int, kLoads>;
            const Buffers f = buffers(s + 2);
            arrived(Left());
            quadrant(Zero(), Zero(), b2, a0, [&](auto u) {
                if constexpr (u % 2 == 0) read(slot, B1, u / 2, b1);
                if constexpr (u % 2 == 1) b0[u / 2] = b2[u / 2];
                if constexpr (u % 4 == 1) load(slot, std::integral_constant<int, u / 4>(), f);
            });
            quadrant(One(), Zero(), b1, a0, [&](auto u) {
                if constexpr (u < 8) read(slot, A1, u, a1);
                if constexpr (u % 4 == 1) load(slot, std::integral_constant<int, 4 + u / 4>(), f);
            });
            arrived(Left());
            const int other = 1 - slot;
            quadrant(One(), One(), b1, a1, [&](auto u) {
                if constexpr (u % 2 == 0) read(other, A0, u / 2, a0);
                if constexpr (u % 4 == 1) load(slot, std::integral_constant<int, 8 + u / 4>(), f);
            });
            quadrant(Zero(), One(), b0, a1, [&](auto u) {
                if constexpr (u < 8) read(other, B0, u, b2);
                if constexpr (u % 4 == 1) load(slot, std::integral_constant<int, 12 + u / 4>(), f);
            });
            slot = other;
        } while (++s < stop);
        // and the last products' results are there
        asm volatile("s_waitcnt vmcnt(0)\n\ts_nop 15\n\ts_nop 15" ::: "memory");
        pin();
    }
    // what is no whole step, through registers, zero past the sum's end
    for (; s < end; ++s) {
        const int left = (second(s) ? g.K2 : K) - k_of(s);
        u32x4 v[kLoads];
        each(std::make_integer_sequence<int, kLoads>(), [&](auto i) {
            constexpr int q = i / 4, u = i % 4;
            constexpr bool x = q == A0 || q == A1;
            const int r = x ? LX::row(u, w, lane) : LW::row(u, w, lane), c = (x ? LX::chunk(u, w, lane) : LW::chunk(u, w, lane)) * kElems;
            const int64_t ld = x ? g.ldx : g.ldw;
            const int rows = x ? M - m0 : g.N - n0;
            const T* p = from(q, s);
            v[i] = (u32x4){0, 0, 0, 0};
            if (x ? C::XK : C::WK) {
                if (r < left) v[i] = chunk_of(p + r * ld, x ? row_x(q, c) : row_w(q, c), rows);
            } else {
                v[i] = chunk_of(p + min(x ? row_x(q, r) : row_w(q, r), rows - 1) * ld, c, left);
            }
        });
        __syncthreads();
        each(std::make_integer_sequence<int, kLoads>(), [&](auto i) { *reinterpret_cast<u32x4*>(&lds[0][i * 4096 + w * 1024 + lane * 16]) = v[i]; });
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) read(0, A0, i, a0), read(0, B0, i, b0), read(0, B1, i, b1), read(0, A1, i, a1);
        quadrant(Zero(), Zero(), b0, a0, [](auto) {});
        quadrant(One(), Zero(), b1, a0, [](auto) {});
        quadrant(One(), One(), b1, a1, [](auto) {});
        quadrant(Zero(), One(), b0, a1, [](auto) {});
    }
    __syncthreads();
    e.template finish<C>(part, acc);
}

// ------------------------------------------------------------- plain epilogue
struct FromZero {
    template <class C>
    __device__ void start(const Part&, typename C::Acc (&)[C::FN][C::FM]) const {}
};
// The sums as they are: rounded to O, or added to (ADD) or set as fp32 parts
// [split][M][ld].
template <typename O>
struct Store : FromZero {
    O* out[2];       // of each product
    int64_t ld;      // from row to row
    int64_t splits;  // from split to split
    bool add, whole;  // whole: four at once
    template <class C>
    __device__ __attribute__((always_inline)) void finish(const Part& p, typename C::Acc (&acc)[C::FN][C::FM]) const {
        static_assert(!C::PAIR, "one matrix");
        constexpr int kLanes = C::WN / 4, kAtOnce = 64 / kLanes, kPitch = C::WN + 4;
        const int c = p.lane % kLanes * 4, n = p.n0 + c;
        O* to0 = out[p.product] + p.split * splits + n;
        turned<C>(p, acc, [&](int j, float* rows) __attribute__((always_inline)) {
            if (n >= p.N) return;
#pragma unroll 4
            for (int r = p.lane / kLanes; r < 32; r += kAtOnce) {
                const int m = p.m0 + j * 32 + r;
                if (m >= p.M) break;
                const f32x4 q = *reinterpret_cast<const f32x4*>(rows + r * kPitch + c);
                float v[4] = {q[0], q[1], q[2], q[3]};
                O* to = to0 + m * ld;
                if (whole) {
                    if (add) {
                        float o[4];
                        get4(to, o);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] += o[i];
                    }
                    put4(to, v);
                } else {
                    for (int i = 0; i < 4 && n + i < p.N; ++i) put(to + i, add ? to_f(to[i]) + v[i] : v[i]);
                }
            }
        });
    }
};
inline bool fours(const void* p, int64_t ld, size_t elem_bytes) { return ld % 4 == 0 && (uintptr_t)p % (4 * elem_bytes) == 0; }

// Adds the splits' sums [splits][rows][N] in their order and rounds them.  row:
// where each row of the result stands among the summed ones, -1 for a row of
// zeros; null: in place.  live: the rows that were in use, in tiles of `tile`.
// Four columns a thread.
struct Live {
    const int* count;
    int tile, more;
};
template <typename T>
__global__ __launch_bounds__(kThreads) void k_join(const float* part, int splits, int64_t stride, const int* row, Live live, int M, int N, T* out, bool whole) {
    if (live.count) splits = splits_in_use(splits, live.more, (unsigned)((*live.count + live.tile - 1) / live.tile) * (unsigned)((N + live.tile - 1) / live.tile));
    const int across = (N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int m = (int)(i / across), n = (int)(i % across) * 4;
    if (m >= M) return;
    const int from = row ? row[m] : m;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    T* to = out + (int64_t)m * N + n;
    if (whole) {
        if (from >= 0)
#pragma unroll 8
            for (int s = 0; s < splits; ++s) {
                float p[4];
                get4(part + s * stride + (int64_t)from * N + n, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] += p[j];
            }
        put4(to, v);
        return;
    }
    if (from >= 0)
        for (int s = 0; s < splits; ++s) {
            const float* p = part + s * stride + (int64_t)from * N + n;
            for (int j = 0; j < 4; ++j)
                if (n + j < N) v[j] += p[j];
        }
    for (int j = 0; j < 4; ++j)
        if (n + j < N) put(to + j, v[j]);
}

// ---------------------------------------------------------------- host side
inline unsigned four_blocks(long long M, long long N) { return (unsigned)((M * ((N + 3) / 4) + kThreads - 1) / kThreads); }

// The tile of a product and the splits of its sum over k: those of the least time
// by a plain count, of rounds of workgroups, steps in each, and the bytes of the
// splits' sums.  Microseconds: a tile's step (128 bytes of k; two tiles of 64 share
// a compute unit), and what a workgroup takes beside its steps.  kTile192 is 192
// rows by 128 columns, only where `tall`: products of up to that many rows read W
// once (192 x 14336 x 4096, a pair: 49 us, 65 with tiles of 64); the count takes it
// for others as well.  `room`: the bytes that the splits' sums may take.
constexpr int kMaxSplits = 32;
constexpr long long kNoSums = 0, kAnySums = 1ll << 62;
enum Size { kTile256, kTile128, kTile64, kTile192 };
struct Plan {
    Size size;
    int splits;
};
inline long long step_of(spec_dtype d) { return 128 / (long long)elem(d); }
inline Plan plan_of(spec_dtype d, long long M, long long N, long long K, int products, long long room, bool tall) {
    static const double kStepTime[2][4] = {{7.2, 1.85, 0.95, 2.8}, {1.4, 0.6, 0.5, 0.5}}, kBeside[4] = {12, 7, 5, 7};
    static const int kRows[4] = {256, 128, 64, 192}, kColumns[4] = {256, 128, 64, 128};
    const long long steps = (K + step_of(d) - 1) / step_of(d);
    Plan best{kTile64, 1};
    double least = 1e30;
    for (int z = 0; z < (tall ? 4 : 3); ++z) {
        const long long slots = z == kTile64 ? 512 : 256;
        const long long tiles = ((M + kRows[z] - 1) / kRows[z]) * ((N + kColumns[z] - 1) / kColumns[z]) * products;
        for (int s = 1; s <= kMaxSplits && s <= steps && (s == 1 || s * M * N * products * 4 <= room); ++s) {
            const long long per = (steps + s - 1) / s, rounds = (tiles * s + slots - 1) / slots;
            double us = rounds * (per * kStepTime[d == SPEC_BF16][z] + kBeside[z]);
            if (s > 1) us += 4 + (double)(s * M * N * products) * 8 / 4e6;
            if (us < least) least = us, best = {(Size)z, (int)((steps + per - 1) / per)};
        }
    }
    return best;
}

template <typename T>
void join(const float* part, int splits, const int* row, Live live, int M, int N, T* out, hipStream_t st) {
    const bool whole = fours(part, N, 4) && fours(out, N, sizeof(T));
    k_join<T><<<four_blocks(M, N), kThreads, 0, st>>>(part, splits, (int64_t)M * N, row, live, M, N, out, whole);
}

template <class C, class E>
void launch_tile(const Product& g, const E& e, hipStream_t st) {
    const unsigned grid = (unsigned)((g.M + C::BM - 1) / C::BM) * (unsigned)((g.N + C::kColsN - 1) / C::kColsN) *
                          (unsigned)((g.more > g.splits ? g.more : g.splits) * g.products);
    if constexpr (C::BM == 256)
        k_wide<C, E><<<grid, kThreads, 0, st>>>(g, e);
    else
        k_product<C, E><<<grid, kThreads, 0, st>>>(g, e);
}
inline bool aligned(const Product& g, size_t e) {
    uintptr_t a = (uintptr_t)g.x[0] | (uintptr_t)g.w[0] | (uintptr_t)g.x[1] | (uintptr_t)g.w[1];
    return a % 16 == 0 && g.ldx * e % 16 == 0 && g.ldw * e % 16 == 0;
}
// What is not aligned takes tiles of 64 through registers, with the same splits.
template <typename T, bool XK, bool WK, class E>
void launch_product(const Product& g, const E& e, Size size, hipStream_t st) {
    if (!aligned(g, sizeof(T)))
        launch_tile<Tile<T, 64, 64, 32, 32, 2, XK, WK, false, false>>(g, e, st);
    else if (size == kTile256)
        launch_tile<Tile<T, 256, 256, 128, 128, 2, XK, WK, false, true>>(g, e, st);
    else if (size == kTile128)
        launch_tile<Tile<T, 128, 128, 64, 64, 4, XK, WK, false, true>>(g, e, st);
    else
        launch_tile<Tile<T, 64, 64, 32, 32, 4, XK, WK, false, true>>(g, e, st);
}

}  // namespace

#endif  // SPEC_PRODUCT_H

// linear.hip -- the matrix product that a draft head is made of, for gfx950
// (MI355X): y = residual + act(x W^T + bias) and its gradients.
//
//   z = x W^T + bias        x [M][K], W [N][K], bias [N]
//   y = residual + act(z)   residual, y, z [M][N]
//   dz = dy act'(z)         dx = dz W, dW = dz^T x, dbias = sum over rows of dz
// Products are summed in fp32; bias, activation and residual are applied to
// the fp32 sum and the result is rounded once.
// With bf16 operands the kept z and dz are bf16: dz is an operand of the matrix
// instructions, and z's half step moves act'(z) by at most 0.8 * 2^-8 |z|,
// about what dz's own rounding does.  The bias gradient sums unrounded dz.
#include "tiles.h"

namespace {

// ------------------------------------------------------------ matrix product
// out[m][n] = residual + act(sum_k X[m][k] W[n][k] + bias[n]).  Rows of X and W
// are `ldx` and `ldw` elements apart.
struct Gemm {
    const void *X, *W;
    int64_t ldx, ldw;
    int M, N, K;
    const void *bias, *residual;
    int act;
    void *out, *preact;
    int tiles_n, splits;  // splits of K, and where there are several
    float* part;          // their sums [splits][M][N]
};

// ------------------------------------------------------------------ epilogue
// Four neighbouring outputs of row m from n on (n % 4 == 0), one by one.
template <typename T, typename O>
__device__ inline void finish4(const Gemm& g, int m, int n, const float (&z)[4]) {
    const size_t at = (size_t)m * g.N + n;
    for (int i = 0; i < 4; ++i) {
        if (n + i >= g.N) break;
        float v = z[i];
        if (g.bias) v += to_f(static_cast<const T*>(g.bias)[n + i]);
        if (g.preact) put(static_cast<T*>(g.preact) + at + i, v);
        v = act_of(v, g.act);
        if (g.residual) v += to_f(static_cast<const O*>(g.residual)[at + i]);
        put(static_cast<O*>(g.out) + at + i, v);
    }
}
// The same at once, bias (or 0) and residual read before.  Where N is a
// multiple of 4 and every array aligned to four elements.
template <typename T, typename O>
__device__ inline void finish4_whole(const Gemm& g, int m, int n, const float (&bias)[4], Raw4<O> res, float (&z)[4]) {
    const size_t at = (size_t)m * g.N + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] += bias[i];
    if (g.preact) put4(static_cast<T*>(g.preact) + at, z);
    if (g.act != SPEC_ACT_NONE)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = act_of(z[i], g.act);
    if (g.residual)
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] += raw4_at(res, i);
    put4(static_cast<O*>(g.out) + at, z);
}
template <typename T, typename O>
__device__ inline bool four_at_once(const Gemm& g) {
    const uintptr_t t = (uintptr_t)g.bias | (uintptr_t)g.preact, o = (uintptr_t)g.residual | (uintptr_t)g.out;
    return g.N % 4 == 0 && t % (4 * sizeof(T)) == 0 && o % (4 * sizeof(O)) == 0;
}

// -------------------------------------------------------------- tiled product
// Bound by the matrix cores: 4096 x 4096 x 8192 bf16 203 us (1354 TFLOP/s), of
// which the instructions themselves are busy about two thirds; fp32 1836 us
// (150 TFLOP/s); 8192 x 4096 x 4096 bf16, with half of the steps to each
// epilogue, 232 us.
// BM x BN outputs per workgroup of four waves; a wave has WM x WN of them in
// 32 x 32 blocks, weights as the instruction's first operand, so that a lane
// ends with four neighbouring n of one m.  The rows'
// next kRowBytes (128: 64 bf16, 32 fp32) are one stage in LDS: chunk c of row r
// lies at place c ^ (r / 2 & 7) of its 128 bytes, or c ^ (r / 4 & 3) of its 64,
// so that sixteen rows read at one chunk use each of the 64 banks once (with
// c ^ (r & 7) a third of the LDS cycles were conflicts).

template <typename T, typename O, int BM, int BN, int WM, int WN, int kRowBytes, int STAGES, bool DIRECT>
__global__ __launch_bounds__(kThreads, (BM + BN) * kRowBytes * STAGES <= 80 * 1024 ? 2 : 1) void k_gemm(Gemm g) {
    static_assert(BM / WM * (BN / WN) == kThreads / 64, "four waves");
    constexpr int kRowChunks = kRowBytes / 16, kElems = 16 / (int)sizeof(T), kStep = kElems * kRowChunks;
    constexpr int kSlab = 1024 / kRowBytes;         // rows of one load
    constexpr int FM = WM / 32, FN = WN / 32;       // 32 x 32 blocks a wave
    constexpr int kWavesN = BN / WN;
    constexpr int kRows = BM + BN;                  // rows of a stage: W's, then X's
    constexpr int kLoads = kRows / kSlab / 4;       // 1 KiB loads a wave and stage
    static_assert(kLoads * kSlab * 4 == kRows && BN % (4 * kSlab) == 0, "whole loads, each of one matrix");
    constexpr int kStageBytes = kRows * kRowBytes;
    __shared__ __attribute__((aligned(1024))) char lds[STAGES][kStageBytes];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    int tm, tn;
    const int tiles_m = (g.M + BM - 1) / BM;
    const int tiles = tiles_m * g.tiles_n, split = blockIdx.x / tiles;
    tile_of(blockIdx.x % tiles, tiles, tiles_m, g.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const T* W = static_cast<const T*>(g.W) + (int64_t)n0 * g.ldw;
    const T* X = static_cast<const T*>(g.X) + (int64_t)m0 * g.ldx;

    // Load i of this wave: kSlab rows, a lane's row and place by its number.
    // swizzle(r): what a row's chunks are exchanged by; the same for r + 16.
    auto swizzle = [](int r) { return kRowBytes == 128 ? r >> 1 & 7 : r >> 2 & 3; };
    auto row_of = [&](int i) { return (i * 4 + w) * kSlab; };
    const int r8 = lane / kRowChunks, c8 = lane % kRowChunks ^ swizzle(w * kSlab + r8);
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(W), (short)0, 0x7fffffff, 0x00020000);
    const __amdgpu_buffer_rsrc_t rx = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(X), (short)0, 0x7fffffff, 0x00020000);
    uint32_t off[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        // rows past the matrix read its last row; their products are dropped
        const int r = row_of(i) + r8;
        const int64_t e = row_of(i) < BN ? min(r, g.N - 1 - n0) * g.ldw : min(r - BN, g.M - 1 - m0) * g.ldx;
        off[i] = (uint32_t)(e * (int64_t)sizeof(T)) + (uint32_t)c8 * 16;
    }
    // this split's steps [begin, end), `full` of them whole and loaded directly
    const int steps = (g.K + kStep - 1) / kStep, per = (steps + g.splits - 1) / g.splits;
    const int begin = split * per, end = min(steps, begin + per);
    const int full = DIRECT ? max(0, min(g.K / kStep, end) - begin) : 0;
    // loads [FROM, TO) of a step into a stage
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)&lds[0][0] + w * 1024;
    auto load_direct = [&](int stage, int step, auto from, auto to) {
        const uint32_t base = lds0 + stage * kStageBytes, k = (uint32_t)(begin + step) * kRowBytes;
        each(std::make_integer_sequence<int, kLoads>(), [&](auto i) {
            if constexpr (i >= from && i < to) to_lds<i * 4096, BM <= 64 && BN == 128 && i * 4 * kSlab < BN>(i * 4 * kSlab < BN ? rw : rx, base, off[i], k);
        });
    };
    using Zero = std::integral_constant<int, 0>;
    using All = std::integral_constant<int, kLoads>;
    auto fetch = [&](int step, u32x4 (&q)[kLoads]) {  // the same through registers, any alignment
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = row_of(i) + r8;
            const T* row = row_of(i) < BN ? W + min(r, g.N - 1 - n0) * g.ldw : X + min(r - BN, g.M - 1 - m0) * g.ldx;
            q[i] = chunk_of(row, step * kStep + c8 * kElems, g.K);
        }
    };
    auto place = [&](int stage, const u32x4 (&q)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<u32x4*>(&lds[stage][row_of(i) * kRowBytes + lane * 16]) = q[i];
    };

    f32x16 acc[FN][FM] = {};
    const int wn = w % kWavesN * WN, wm = w / kWavesN * WM, l = lane & 31, h = lane >> 5;
    // Operands of one pair of chunks, read from LDS a pair ahead of their use.
    constexpr int kPairs = kRowChunks / 2, kProducts = FN * FM, kReads = FN + FM;
    struct Operands {
        u32x4 a[FN], b[FM];
    };
    Operands f[2];
    const char *as = &lds[0][0] + (wn + l) * kRowBytes, *bs = &lds[0][0] + (BN + wm + l) * kRowBytes;
    auto read = [&](int stage, int pair, int i, Operands& o) {
        const int at = stage * kStageBytes + ((2 * pair + h) ^ swizzle(l)) * 16;
        if (i < FM)
            o.b[i] = *reinterpret_cast<const u32x4*>(bs + at + i * 32 * kRowBytes);
        else
            o.a[i - FM] = *reinterpret_cast<const u32x4*>(as + at + (i - FM) * 32 * kRowBytes);
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

    if constexpr (DIRECT) {
        static_assert(kPairs % 2 == 0, "operands alternate");
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (s < full) load_direct(s, s, Zero(), All());
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
        // loads under this pair, half under the next (an instruction takes
        // four cycles of a product's 32, so a product hides seven).
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
            int s = STAGES;
            for (; s < full; ++s) {
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(kLoads * (STAGES - 2)) : "memory");
                advance(std::true_type(), s);
            }
            for (s = s - STAGES + 1; s < full; ++s) {
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                advance(std::false_type(), 0);
            }
            multiply(f[1], [](auto) {});
        }
    }
    auto compute = [&](int stage) {
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
#pragma unroll
            for (int i = 0; i < kReads; ++i) read(stage, p, i, f[0]);
            multiply(f[0], [](auto) {});
        }
    };
    // what is no whole step, or not aligned: the next step's loads are on
    // their way while one is worked on
    if (begin + full < end) {
        u32x4 q[kLoads];
        fetch(begin + full, q);
        for (int s = begin + full; s < end; ++s) {
            __syncthreads();
            place(0, q);
            __syncthreads();
            if (s + 1 < end) fetch(s + 1, q);
            compute(0);
        }
    }

    // Each wave turns its blocks, 32 rows of m at a time, through its own part
    // of the LDS, so that neighbouring lanes have neighbouring n.
    constexpr int kCols = WN, kPitch = kCols + 4;
    static_assert(4 * 32 * kPitch * 4 <= STAGES * kStageBytes, "the epilogue's tiles fit");
    __syncthreads();
    float* turn = reinterpret_cast<float*>(&lds[0][0]) + w * 32 * kPitch;
    const bool whole = four_at_once<T, O>(g);
    constexpr int kLanes = kCols / 4, kAtOnce = 64 / kLanes, kBatch = 32 / kAtOnce < 8 ? 32 / kAtOnce : 8;
    const int n = n0 + wn + lane % kLanes * 4;
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    Raw4<O> ahead[kBatch];
    auto look_ahead = [&](int m) {  // the batch of rows from m on
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            ahead[u] = *reinterpret_cast<const Raw4<O>*>(static_cast<const O*>(g.residual) + (size_t)min(m + u * kAtOnce, g.M - 1) * g.N + n);
    };
    if (whole && n < g.N && g.splits == 1) {
        if (g.bias) get4(static_cast<const T*>(g.bias) + n, bias);
        if (g.residual) look_ahead(m0 + wm + lane / kLanes);
    }
    each(std::make_integer_sequence<int, FM>(), [&](auto j) {
#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *reinterpret_cast<f32x4*>(turn + l * kPitch + i * 32 + q * 8 + h * 4) =
                    (f32x4){acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int top = m0 + wm + j * 32;
        if (g.splits > 1) {
#pragma unroll 1
            for (int r = lane / kLanes; r < 32; r += kAtOnce) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(turn + r * kPitch + lane % kLanes * 4);
                if (top + r >= g.M) break;
                float* to = g.part + ((size_t)split * g.M + top + r) * g.N + n;
                if (g.N % 4 == 0 && n < g.N)
                    *reinterpret_cast<f32x4*>(to) = v;
                else
                    for (int i = 0; i < 4; ++i)
                        if (n + i < g.N) to[i] = v[i];
            }
        } else if (n < g.N && whole) {
#pragma unroll 1
            for (int r0 = lane / kLanes; r0 < 32; r0 += kAtOnce * kBatch) {
                // a batch of rows at once, the next batch's residual on its way
                float z[kBatch][4];
                Raw4<O> res[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    res[u] = ahead[u];
                    const f32x4 v = *reinterpret_cast<const f32x4*>(turn + (r0 + u * kAtOnce) * kPitch + lane % kLanes * 4);
#pragma unroll
                    for (int i = 0; i < 4; ++i) z[u][i] = v[i];
                }
                if (g.residual) look_ahead(top + r0 + kAtOnce * kBatch);
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const int m = top + r0 + u * kAtOnce;
                    if (m < g.M) finish4_whole<T, O>(g, m, n, bias, res[u], z[u]);
                }
            }
        } else if (n < g.N) {
#pragma unroll 1
            for (int r = lane / kLanes; r < 32; r += kAtOnce) {
                const f32x4 v = *reinterpret_cast<const f32x4*>(turn + r * kPitch + lane % kLanes * 4);
                const float z[4] = {v[0], v[1], v[2], v[3]};
                if (top + r < g.M) finish4<T, O>(g, top + r, n, z);
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    });
}

// Adds the splits' sums in their order and finishes them: four outputs a thread.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void k_finish(Gemm g) {
    const int across = (g.N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int m = (int)(i / across), n = (int)(i % across) * 4;
    if (m >= g.M) return;
    float z[4] = {0.f, 0.f, 0.f, 0.f};
    const bool whole = four_at_once<T, O>(g);
    for (int s = 0; s < g.splits; ++s) {
        const float* p = g.part + ((size_t)s * g.M + m) * g.N + n;
        if (whole) {
            const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] += v[j];
        } else {
            for (int j = 0; j < 4; ++j)
                if (n + j < g.N) z[j] += p[j];
        }
    }
    if (!whole) {
        finish4<T, O>(g, m, n, z);
        return;
    }
    float bias[4] = {0.f, 0.f, 0.f, 0.f};
    Raw4<O> res = {};
    if (g.bias) get4(static_cast<const T*>(g.bias) + n, bias);
    if (g.residual) res = *reinterpret_cast<const Raw4<O>*>(static_cast<const O*>(g.residual) + (size_t)m * g.N + n);
    finish4_whole<T, O>(g, m, n, bias, res, z);
}

// -------------------------------------------------------- product of few rows
// M <= 16: bound by reading W once.  A workgroup has 16 rows of W; its four
// waves take every fourth piece of 256 bytes of the rows, W and X
// straight into registers as operands of 16x16 instructions (lane l: row
// l % 16, chunk l / 16), the next piece on its way while one is multiplied.
// The waves' sums are added in LDS.  One row of 4096 x 4096: bf16 11.7 us, of
// which about 5 are the launch, fp32 24 us; one row of 512 x 8192, where 32
// workgroups leave most of the chip idle, 15 and 32 us.
__device__ inline f32x4 mfma16(bf16, u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ inline f32x4 mfma16(float, u32x4 a, u32x4 b, f32x4 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
}

template <typename T, typename O, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void k_few(Gemm g) {
    constexpr int kElems = 16 / (int)sizeof(T), KS = 4, kPiece = KS * 4 * kElems, kPitch = 20;
    __shared__ float sums[4][16][kPitch];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6, r = lane & 15, c = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const T* W = static_cast<const T*>(g.W) + min(n0 + r, g.N - 1) * g.ldw;
    const T* X = static_cast<const T*>(g.X) + min(r, g.M - 1) * g.ldx;
    struct Piece {
        u32x4 a[KS], b[KS];
    };
    auto load = [&](int p, Piece& q) {
        const bool full = ALIGNED && (p + 1) * kPiece <= g.K;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int k = p * kPiece + (s * 4 + c) * kElems;
            q.a[s] = full ? *reinterpret_cast<const u32x4*>(W + k) : chunk_of(W, k, g.K);
            q.b[s] = (u32x4){0, 0, 0, 0};
            if (r < g.M) q.b[s] = full ? *reinterpret_cast<const u32x4*>(X + k) : chunk_of(X, k, g.K);
        }
    };
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    const int pieces = (g.K + kPiece - 1) / kPiece;
    Piece q;
    if (w < pieces) load(w, q);
    for (int p = w; p < pieces; p += 4) {
        Piece next;
        if (p + 4 < pieces) load(p + 4, next);
#pragma unroll
        for (int s = 0; s < KS; ++s) acc = mfma16(T(), q.a[s], q.b[s], acc);
        q = next;
    }
    *reinterpret_cast<f32x4*>(&sums[w][r][c * 4]) = acc;
    __syncthreads();
    const bool whole = four_at_once<T, O>(g);
    if (t < 64) {
        const int m = t / 4, n = t % 4 * 4;
        f32x4 v = *reinterpret_cast<const f32x4*>(&sums[0][m][n]);
#pragma unroll
        for (int k = 1; k < 4; ++k) v += *reinterpret_cast<const f32x4*>(&sums[k][m][n]);
        float z[4] = {v[0], v[1], v[2], v[3]};
        if (m >= g.M || n0 + n >= g.N) return;
        if (whole) {
            float bias[4] = {0.f, 0.f, 0.f, 0.f};
            Raw4<O> res = {};
            if (g.bias) get4(static_cast<const T*>(g.bias) + n0 + n, bias);
            if (g.residual) res = *reinterpret_cast<const Raw4<O>*>(static_cast<const O*>(g.residual) + (size_t)m * g.N + n0 + n);
            finish4_whole<T, O>(g, m, n0 + n, bias, res, z);
        } else {
            finish4<T, O>(g, m, n0 + n, z);
        }
    }
}

// ---------------------------------------------------------- gradients' inputs
// dz = dy act'(z) to dz [M][ld] and, turned, to dzt [N][ldt], rounded, zero up
// to the rows' ends; sums of 64 rows' unrounded dz to part [M/64][N].  Each of
// the three is optional.  The same kernel turns or pads a matrix (dy alone).  Bound by
// memory: a thread reads and writes eight neighbouring elements at once
// (VECTOR: N a multiple of 8 and 16-byte aligned inputs; ld and ldt are whole
// 16-byte chunks always), the turning goes through LDS.  All that an 8192 x
// 4096 x 4096 block's gradients need, 0.45 GB read and written: 90 us (5 TB/s).
struct Slope {
    const void *dy, *preact;
    int act, M, N;
    void *dz, *dzt;
    int64_t ld, ldt;
    float* part;  // or, where there is one part,
    void* sum;    // the bias gradient itself
    bool vector;
};
// Up to three of them in one launch: dz, then W and x turned (jobs 1 and 2 are
// of the operands' type).  A job's 64 x 64 blocks follow the last one's.
struct Slopes {
    Slope job[3];
    unsigned end[3];  // blocks up to the end of each job
};

template <typename I, bool VECTOR>
__device__ inline void get8(const I* p, int left, float (&v)[8]) {
    if constexpr (VECTOR) {
        float a[4], b[4];
        get4(p, a);
        get4(p + 4, b);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = a[i], v[i + 4] = b[i];
    } else if (left >= 8) {  // at any alignment
        struct Any {
            I v[8];
        } __attribute__((packed, aligned(sizeof(I))));
        const Any q = *reinterpret_cast<const Any*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f(q.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? to_f(p[i]) : 0.f;
    }
}
// eight elements to a row of whole chunks, `left` of which are in it
template <typename T>
__device__ inline void put8(T* p, int64_t left, const float (&v)[8]) {
    constexpr int kElems = 16 / (int)sizeof(T);
#pragma unroll
    for (int c = 0; c < 8; c += kElems) {
        u32x4 q;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if constexpr (sizeof(T) == 2)
                q[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            else
                q[i] = __float_as_uint(v[c + i]);
        if (c < left) *reinterpret_cast<u32x4*>(p + c) = q;
    }
}

template <typename I, typename T, bool VECTOR>
__device__ inline void slope_block(const Slope& a, unsigned block, float (&tile)[64][65]) {
    const unsigned across = (unsigned)((a.N + 63) / 64), row = block / across;
    const int n0 = (int)(block % across) * 64, m0 = (int)row * 64, t = threadIdx.x, c = t % 8 * 8;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int r = t / 8 + u * 32, m = m0 + r, n = n0 + c;
        float v[8] = {}, z[8];
        if (m < a.M && n < a.N) {
            const size_t at = (size_t)m * a.N + n;
            get8<I, VECTOR>(static_cast<const I*>(a.dy) + at, a.N - n, v);
            if (a.preact) {
                get8<T, VECTOR>(static_cast<const T*>(a.preact) + at, a.N - n, z);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= act_slope(z[i], a.act);
            }
        }
        if (a.dz && m < a.M && n < a.ld) put8(static_cast<T*>(a.dz) + (size_t)m * a.ld + n, a.ld - n, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) tile[r][c + i] = v[i];
    }
    __syncthreads();
    if (a.dzt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = t / 8 + u * 32, n = n0 + r, m = m0 + c;
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = tile[c + i][r];
            if (n < a.N && m < a.ldt) put8(static_cast<T*>(a.dzt) + (size_t)n * a.ldt + m, a.ldt - m, v);
        }
    if ((a.part || a.sum) && t < 64 && n0 + t < a.N) {
        float s[4] = {};
#pragma unroll
        for (int r = 0; r < 64; ++r) s[r % 4] += tile[r][t];
        const float all = (s[0] + s[1]) + (s[2] + s[3]);
        if (a.sum)
            put(static_cast<T*>(a.sum) + n0 + t, all);
        else
            a.part[(size_t)row * a.N + n0 + t] = all;
    }
}

template <typename I, typename T>
__global__ __launch_bounds__(kThreads) void k_slopes(Slopes a) {
    __shared__ float tile[64][65];
    const unsigned b = blockIdx.x;
    if (b < a.end[0]) {
        if (a.job[0].vector)
            slope_block<I, T, true>(a.job[0], b, tile);
        else
            slope_block<I, T, false>(a.job[0], b, tile);
    } else {
        const bool last = b >= a.end[1];
        const Slope& s = a.job[last ? 2 : 1];
        if (s.vector)
            slope_block<T, T, true>(s, b - a.end[last ? 1 : 0], tile);
        else
            slope_block<T, T, false>(s, b - a.end[last ? 1 : 0], tile);
    }
}

// dbias[n] = the sum of the parts, in a fixed order: 64 columns a workgroup,
// every sixteenth part to a wave
constexpr int kSumWaves = 16;
template <typename T>
__global__ __launch_bounds__(64 * kSumWaves) void k_bias_sum(const float* part, int parts, int N, T* out) {
    __shared__ float sums[kSumWaves][64];
    const int c = threadIdx.x & 63, w = threadIdx.x >> 6, n = blockIdx.x * 64 + c;
    float s = 0.f;
    if (n < N)
        for (int p = w; p < parts; p += kSumWaves) s += part[(size_t)p * N + n];
    sums[w][c] = s;
    __syncthreads();
    if (w == 0 && n < N) {
        for (int i = 1; i < kSumWaves; ++i) s += sums[i][c];
        put(out + n, s);
    }
}

// ---------------------------------------------------------------- host side
constexpr long long kMaxElems = 1ll << 34;  // of a matrix: launches stay below 2^32 threads
inline bool sizes_ok(long long M, long long N, long long K) {
    return M >= 1 && N >= 1 && K >= 1 && M <= SPEC_MAX_LINEAR && N <= SPEC_MAX_LINEAR && K <= SPEC_MAX_LINEAR &&
           M * N < kMaxElems && M * K < kMaxElems && N * K < kMaxElems;
}

// ------------------------------------------------------------ choice of kernel
// A rule on sizes alone.  Up to 16 rows are read against W in registers
// (k_few), but from kWide columns on up to 64 rows take tiles of 32 or 64 rows
// by 128 of W, which keep more of W on its way (us at N 128256, K 4096, bf16:
// one row 155, k_few 199; 32 rows 169, 187 with temporal loads).  Else the
// largest tile that still gives kEnough workgroups: 256 (4096 x 4096 x 8192
// bf16: 219 us beside 259 with 128, timed together), 128 (1024 x 4096 x 4096:
// 37 us), 64; and where 64 leaves compute units idle, K is split over several
// workgroups a tile, of at least four steps each, their fp32 sums added by one
// more launch, where the steps saved outweigh that launch (split / not, us:
// 512 x 512 x 8192 bf16 18.6 / 26.6, fp32 45.8 / 140.8; 192 x 4096 x 4096 bf16
// 19.8 / 15.8).
constexpr int kWide = 16384, kEnough = 200, kSplitGroups = 512, kMaxSplits = 8, kSplitWorth = 50;
enum Choice { kFew, kRows32, kRows64, kTile256, kTile128, kTile64 };
inline long long tiles_of(long long M, long long N, int b) { return ((M + b - 1) / b) * ((N + b - 1) / b); }
inline Choice choose(long long M, long long N) {
    if (M <= 16 && N < kWide) return kFew;
    if (M <= 32 && N >= kWide) return kRows32;
    if (M <= 64 && N >= kWide) return kRows64;
    // a larger tile must not compute more than a quarter more past the edges
    // (100 x 128256 x 4096 bf16: 208 us with 128, 258 with 256)
    auto fits = [&](int b) {
        return tiles_of(M, N, b) >= kEnough && tiles_of(M, N, b) * 16 <= tiles_of(M, N, b / 2) * 5;
    };
    return fits(256) ? kTile256 : fits(128) ? kTile128 : kTile64;
}
inline int splits_of(spec_dtype d, long long M, long long N, long long K) {
    if (choose(M, N) != kTile64) return 1;
    const long long step = 128 / (long long)elem(d), steps = (K + step - 1) / step;
    const long long want = kSplitGroups / tiles_of(M, N, 64);
    long long s = want < steps / 4 ? want : steps / 4;
    s = s < 1 ? 1 : s > kMaxSplits ? kMaxSplits : s;
    const long long per = (steps + s - 1) / s;
    // the second launch costs some 4 us, a step 0.18 us in bf16 and 0.54 in fp32
    if ((steps - per) * (d == SPEC_BF16 ? 1 : 3) < kSplitWorth) return 1;
    return (int)((steps + per - 1) / per);  // no split without steps
}
inline size_t split_bytes(spec_dtype d, long long M, long long N, long long K) {
    const int s = splits_of(d, M, N, K);
    return s > 1 ? align_up((size_t)s * (size_t)(M * N) * 4, 256) : 0;
}

// A K that is no whole number of chunks leaves rows that cannot be loaded
// directly.  For the larger tiles both operands are copied to padded rows
// first, which costs their bytes once; the smaller ones load through registers
// (copied / not, us: 4096 x 4096 x 4095 bf16 156 / 355, fp32 991 / 1222,
// 1500 x 2000 x 777 bf16 20.3 / 20.3).  Two kinds of operands are not copied
// and load through registers whatever the size, into tiles of 64: up to 64
// rows over a wide W of odd K, where the copy would move W twice more (32 x
// 128256 x 4095 bf16 311 us, K 4096 170), and operands off 16-byte alignment,
// which the workspace's size cannot tell (4096 x 4096 x 4096 bf16 119 us, x off
// by an element 330, W too 463; fp32 932 and 1230).
inline bool packs(spec_dtype d, long long M, long long N, long long K) {
    const Choice c = choose(M, N);
    return K * (long long)elem(d) % 16 != 0 && (c == kTile256 || c == kTile128);
}
inline size_t packed_x_bytes(spec_dtype d, long long M, long long K) {
    return align_up((size_t)(M * padded(d, K)) * elem(d), 256);
}

template <typename T, typename O, int BM, int BN, int WM, int WN, int kRowBytes, int STAGES, bool DIRECT>
void launch_tiles(Gemm g, hipStream_t st) {
    g.tiles_n = (g.N + BN - 1) / BN;
    const unsigned grid = (unsigned)((g.M + BM - 1) / BM) * (unsigned)g.tiles_n * (unsigned)g.splits;
    k_gemm<T, O, BM, BN, WM, WN, kRowBytes, STAGES, DIRECT><<<grid, kThreads, 0, st>>>(g);
    if (g.splits > 1) {
        const int64_t four = (int64_t)g.M * ((g.N + 3) / 4);
        k_finish<T, O><<<(unsigned)((four + kThreads - 1) / kThreads), kThreads, 0, st>>>(g);
    }
}
template <typename T, typename O>
void launch_typed(Gemm g, spec_dtype d, hipStream_t st) {
    const uintptr_t a = (uintptr_t)g.X | (uintptr_t)g.W | (uintptr_t)(g.ldx * (int64_t)sizeof(T)) | (uintptr_t)(g.ldw * (int64_t)sizeof(T));
    const bool direct = a % 16 == 0;
    const Choice c = choose(g.M, g.N);
    g.splits = 1;
    if (c == kFew) {
        const unsigned grid = (unsigned)((g.N + 15) / 16);
        if (direct)
            k_few<T, O, true><<<grid, kThreads, 0, st>>>(g);
        else
            k_few<T, O, false><<<grid, kThreads, 0, st>>>(g);
    } else if (!direct) {  // rows that start anywhere: through registers
        g.splits = splits_of(d, g.M, g.N, g.K);
        launch_tiles<T, O, 64, 64, 32, 32, 128, 2, false>(g, st);
    } else if (c == kRows32) {
        launch_tiles<T, O, 32, 128, 32, 32, 128, 4, true>(g, st);
    } else if (c == kRows64) {
        launch_tiles<T, O, 64, 128, 64, 32, 128, 3, true>(g, st);
    } else if (c == kTile256) {
        launch_tiles<T, O, 256, 256, 128, 128, 128, 2, true>(g, st);
    } else if (c == kTile128) {
        launch_tiles<T, O, 128, 128, 64, 64, 128, 4, true>(g, st);
    } else {
        g.splits = splits_of(d, g.M, g.N, g.K);
        launch_tiles<T, O, 64, 64, 32, 32, 128, 4, true>(g, st);
    }
}
void launch_gemm(const Gemm& g, spec_dtype d, spec_dtype o, hipStream_t st) {
    if (d == SPEC_F32)
        launch_typed<float, float>(g, d, st);
    else if (o == SPEC_F32)
        launch_typed<bf16, float>(g, d, st);
    else
        launch_typed<bf16, bf16>(g, d, st);
}

// The gradients' workspace: dz, dz turned, x and W turned, rows padded to whole
// chunks, the bias gradient's parts, and the sums of a split product.
struct GradLayout {
    int64_t np, mp;  // padded N and M
    size_t dz, dzt, xt, wt, part, sums, total;
};
inline GradLayout grad_layout(spec_dtype d, long long M, long long N, long long K) {
    const long long e = (long long)elem(d);
    GradLayout l;
    l.np = padded(d, N);
    l.mp = padded(d, M);
    l.dz = 0;
    l.dzt = align_up(l.dz + (size_t)(M * l.np * e), 256);
    l.xt = align_up(l.dzt + (size_t)(N * l.mp * e), 256);
    l.wt = align_up(l.xt + (size_t)(K * l.mp * e), 256);
    l.part = align_up(l.wt + (size_t)(K * l.np * e), 256);
    l.sums = align_up(l.part + (size_t)((M + 63) / 64 * N * 4), 256);  // of K's splits: one product at a time
    const size_t a = split_bytes(d, M, K, l.np), b = split_bytes(d, N, K, l.mp);
    l.total = l.sums + (a > b ? a : b);
    return l;
}

void launch_slopes(Slopes& a, spec_dtype in, spec_dtype d, hipStream_t st) {
    unsigned blocks = 0;
    for (int i = 0; i < 3; ++i) {
        Slope& s = a.job[i];
        s.vector = s.N % 8 == 0 && ((uintptr_t)s.dy | (uintptr_t)s.preact) % 16 == 0;
        if (s.dz || s.dzt || s.part || s.sum) blocks += (unsigned)((s.N + 63) / 64) * (unsigned)((s.M + 63) / 64);
        a.end[i] = blocks;
    }
    if (blocks == 0) return;
    if (d == SPEC_F32)
        k_slopes<float, float><<<blocks, kThreads, 0, st>>>(a);
    else if (in == SPEC_F32)
        k_slopes<float, bf16><<<blocks, kThreads, 0, st>>>(a);
    else
        k_slopes<bf16, bf16><<<blocks, kThreads, 0, st>>>(a);
}

}  // namespace

extern "C" size_t spec_linear_workspace_bytes(spec_dtype dtype, int M, int N, int K) {
    if (!types_ok(dtype, SPEC_F32) || !sizes_ok(M, N, K)) return 0;
    if (packs(dtype, M, N, K)) return packed_x_bytes(dtype, M, K) + packed_x_bytes(dtype, N, K);
    const size_t n = split_bytes(dtype, M, N, K);
    return n ? n : 256;
}

extern "C" spec_status spec_linear(const void* x, const void* weight, const void* bias, const void* residual,
                                   spec_dtype dtype, spec_dtype out_dtype, spec_activation activation, int M, int N,
                                   int K, void* out, void* out_preact, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    if (!types_ok(dtype, out_dtype)) return SPEC_EDTYPE;
    if (!sizes_ok(M, N, K) || !act_ok(activation) || !x || !weight || !out) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_linear_workspace_bytes(dtype, M, N, K))) return SPEC_EWORKSPACE;
    Gemm g{x, weight, K, K, M, N, K, bias, residual, activation, out, out_preact, 0, 1, static_cast<float*>(workspace)};
    if (packs(dtype, M, N, K)) {
        char *xp = static_cast<char*>(workspace), *wp = xp + packed_x_bytes(dtype, M, K);
        const int64_t ld = padded(dtype, K);
        Slopes s{};
        s.job[1] = {weight, nullptr, 0, N, K, wp, nullptr, ld, 0, nullptr, nullptr, false};
        s.job[2] = {x, nullptr, 0, M, K, xp, nullptr, ld, 0, nullptr, nullptr, false};
        launch_slopes(s, dtype, dtype, static_cast<hipStream_t>(stream));
        g.X = xp;
        g.W = wp;
        g.ldx = g.ldw = ld;
        g.K = (int)ld;  // the padding is zero
    }
    launch_gemm(g, dtype, out_dtype, static_cast<hipStream_t>(stream));
    return launched();
}

extern "C" size_t spec_linear_grad_workspace_bytes(spec_dtype dtype, int M, int N, int K) {
    if (!types_ok(dtype, SPEC_F32) || !sizes_ok(M, N, K)) return 0;
    return grad_layout(dtype, M, N, K).total;
}

extern "C" spec_status spec_linear_grad(const void* x, const void* weight, const void* preact, const void* grad_out,
                                        spec_dtype dtype, spec_dtype out_dtype, spec_activation activation, int M,
                                        int N, int K, void* grad_x, void* grad_weight, void* grad_bias,
                                        void* workspace, size_t workspace_bytes, void* stream) {
    if (!types_ok(dtype, out_dtype)) return SPEC_EDTYPE;
    if (!sizes_ok(M, N, K) || !act_ok(activation) || !grad_out) return SPEC_EINVAL;
    if (activation != SPEC_ACT_NONE && !preact) return SPEC_EINVAL;
    if ((grad_x && !weight) || (grad_weight && !x)) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_linear_grad_workspace_bytes(dtype, M, N, K))) return SPEC_EWORKSPACE;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const GradLayout lay = grad_layout(dtype, M, N, K);
    char* ws = static_cast<char*>(workspace);
    const void* z = activation == SPEC_ACT_NONE ? nullptr : preact;
    // without an activation dy is dz where it has the operands' type and
    // aligned rows
    const bool as_is = !z && dtype == out_dtype && lay.np == N && (uintptr_t)grad_out % 16 == 0;
    float* sums = reinterpret_cast<float*>(ws + lay.sums);
    Slopes s{};
    s.job[0] = {grad_out, z, activation, M, N, grad_x && !as_is ? ws + lay.dz : nullptr,
                grad_weight ? ws + lay.dzt : nullptr, lay.np, lay.mp,
                grad_bias && M > 64 ? reinterpret_cast<float*>(ws + lay.part) : nullptr,
                grad_bias && M <= 64 ? grad_bias : nullptr, false};
    if (grad_x) s.job[1] = {weight, nullptr, 0, N, K, nullptr, ws + lay.wt, 0, lay.np, nullptr, nullptr, false};
    if (grad_weight) s.job[2] = {x, nullptr, 0, M, K, nullptr, ws + lay.xt, 0, lay.mp, nullptr, nullptr, false};
    launch_slopes(s, out_dtype, dtype, st);
    if (s.job[0].part) {
        const float* part = reinterpret_cast<const float*>(ws + lay.part);
        const int parts = (M + 63) / 64;
        if (dtype == SPEC_F32)
            k_bias_sum<float><<<(N + 63) / 64, 64 * kSumWaves, 0, st>>>(part, parts, N, (float*)grad_bias);
        else
            k_bias_sum<bf16><<<(N + 63) / 64, 64 * kSumWaves, 0, st>>>(part, parts, N, (bf16*)grad_bias);
    }
    if (grad_x)
        launch_gemm({as_is ? grad_out : ws + lay.dz, ws + lay.wt, lay.np, lay.np, M, K, (int)lay.np, nullptr, nullptr, 0, grad_x, nullptr, 0, 1, sums},
                    dtype, dtype, st);
    if (grad_weight)
        launch_gemm({ws + lay.dzt, ws + lay.xt, lay.mp, lay.mp, N, K, (int)lay.mp, nullptr, nullptr, 0, grad_weight, nullptr, 0, 1, sums},
                    dtype, dtype, st);
    return launched();
}

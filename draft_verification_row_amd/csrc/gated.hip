// gated.hip -- the gated block of a draft head, for gfx950 (MI355X): two
// projections, an activation and their product, with the gradients.
//
//   g = x G^T, u = x U^T, y = act(g) u      x [M][K], G, U [N][K], y [M][N]
//   dg = dy u act'(g), du = dy act(g)
//   dx = dg G + du U, dG = dg^T x, dU = du^T x
// Products are summed in fp32, y is formed from the fp32 sums and rounded once.
// With bf16 operands the slopes dg and du are rounded to bf16, as operands of the
// matrix instructions.  g and u are kept as the fp32 sums: two more roundings to
// bf16 would put the gradients of 8192 x 14336 x 4096 at 0.0031 from float64
// instead of 0.0024 (0.0017 is the result's own rounding).
#include "product.h"

namespace {

// ------------------------------------------------------------------- forward
// Both matrices side by side in one tile, so that a wave ends with g and u of
// the same outputs, x is loaded once for both and y needs no second pass.  8192 x
// 14336 x 4096 bf16 1.51 to 1.57 ms (1230 to 1270 TFLOP/s), with g and u kept 1.66.
template <typename T>
struct Gate : FromZero {
    T* y;
    float *g, *u;  // kept for the gradient, or null
    int act;
    bool whole;
    template <class C>
    __device__ __attribute__((always_inline)) void finish(const Part& p, typename C::Acc (&acc)[C::FN][C::FM]) const {
        constexpr int kLanes = C::kWaveN / 4, kAtOnce = 64 / kLanes, kPitch = C::WN + 4;
        const int c = p.lane % kLanes * 4, n = p.n0 + c;
        turned<C>(p, acc, [&](int j, float* rows) __attribute__((always_inline)) {
            if (n >= p.N) return;
#pragma unroll 4
            for (int r = p.lane / kLanes; r < 32; r += kAtOnce) {
                const int m = p.m0 + j * 32 + r;
                if (m >= p.M) break;
                const f32x4 a = *reinterpret_cast<const f32x4*>(rows + r * kPitch + c);
                const f32x4 b = *reinterpret_cast<const f32x4*>(rows + r * kPitch + C::kWaveN + c);
                out4(m, n, p.N, a, b);
            }
        });
    }
    __device__ void out4(int m, int n, int N, f32x4 a, f32x4 b) const {
        const float va[4] = {a[0], a[1], a[2], a[3]}, vb[4] = {b[0], b[1], b[2], b[3]};
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = act_of(va[i], act) * vb[i];
        const int64_t at = (int64_t)m * N + n;
        if (whole) {
            if (g) put4(g + at, va), put4(u + at, vb);
            put4(y + at, v);
        } else {
            for (int i = 0; i < 4 && n + i < N; ++i) {
                if (g) put(g + at + i, va[i]), put(u + at + i, vb[i]);
                put(y + at + i, v[i]);
            }
        }
    }
};

// M <= 16: bound by reading G and U once.  A workgroup has 16 rows of each; its
// four waves take every fourth piece of 256 bytes of the rows, straight into
// registers as operands of 16x16 instructions (lane l: row l % 16, chunk l /
// 16), the next piece on its way while one is multiplied.  The waves' sums are
// added in LDS.  One row, 14336 x 4096 bf16: 45 us, 5.2 TB/s (loads past the
// caches 55).
__device__ inline f32x4 mfma16(bf16, u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ inline f32x4 mfma16(float, u32x4 a, u32x4 b, f32x4 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], y[i], c, 0, 0, 0);
    return c;
}

template <typename T, bool ALIGNED>
__global__ __launch_bounds__(kThreads) void k_gated_few(Product g, Gate<T> e) {
    constexpr int kElems = 16 / (int)sizeof(T), KS = 4, kPiece = KS * 4 * kElems, kPitch = 20;
    __shared__ float sums[4][2][16][kPitch];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6, r = lane & 15, c = lane >> 4;
    const int n0 = blockIdx.x * 16;
    const T* G = static_cast<const T*>(g.w[0]) + min(n0 + r, g.N - 1) * g.ldw;
    const T* U = static_cast<const T*>(g.w[1]) + min(n0 + r, g.N - 1) * g.ldw;
    const T* X = static_cast<const T*>(g.x[0]) + min(r, g.M - 1) * g.ldx;
    struct Piece {
        u32x4 a[KS], b[KS], x[KS];
    };
    auto load = [&](int p, Piece& q) {
        const bool full = ALIGNED && (p + 1) * kPiece <= g.K;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int k = p * kPiece + (s * 4 + c) * kElems;
            q.a[s] = full ? *reinterpret_cast<const u32x4*>(G + k) : chunk_of(G, k, g.K);
            q.b[s] = full ? *reinterpret_cast<const u32x4*>(U + k) : chunk_of(U, k, g.K);
            q.x[s] = (u32x4){0, 0, 0, 0};
            if (r < g.M) q.x[s] = full ? *reinterpret_cast<const u32x4*>(X + k) : chunk_of(X, k, g.K);
        }
    };
    f32x4 acc[2] = {};
    const int pieces = (g.K + kPiece - 1) / kPiece;
    Piece q;
    if (w < pieces) load(w, q);
    for (int p = w; p < pieces; p += 4) {
        Piece next;
        if (p + 4 < pieces) load(p + 4, next);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            acc[0] = mfma16(T(), q.a[s], q.x[s], acc[0]);
            acc[1] = mfma16(T(), q.b[s], q.x[s], acc[1]);
        }
        q = next;
    }
    *reinterpret_cast<f32x4*>(&sums[w][0][r][c * 4]) = acc[0];
    *reinterpret_cast<f32x4*>(&sums[w][1][r][c * 4]) = acc[1];
    __syncthreads();
    if (t < 64) {
        const int m = t / 4, n = t % 4 * 4;
        f32x4 v[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            v[i] = *reinterpret_cast<const f32x4*>(&sums[0][i][m][n]);
#pragma unroll
            for (int k = 1; k < 4; ++k) v[i] += *reinterpret_cast<const f32x4*>(&sums[k][i][m][n]);
        }
        if (m < g.M && n0 + n < g.N) e.out4(m, n0 + n, g.N, v[0], v[1]);
    }
}

// The sums of a split of k as they are, part [splits][2][M][N]: g, then u.
struct GateSums : FromZero {
    float* part;
    bool whole;
    template <class C>
    __device__ __attribute__((always_inline)) void finish(const Part& p, typename C::Acc (&acc)[C::FN][C::FM]) const {
        constexpr int kLanes = C::kWaveN / 4, kAtOnce = 64 / kLanes, kPitch = C::WN + 4;
        const int c = p.lane % kLanes * 4, n = p.n0 + c;
        turned<C>(p, acc, [&](int j, float* rows) __attribute__((always_inline)) {
            if (n >= p.N) return;
            for (int r = p.lane / kLanes; r < 32; r += kAtOnce) {
                const int m = p.m0 + j * 32 + r;
                if (m >= p.M) break;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(rows + r * kPitch + k * C::kWaveN + c);
                    float* to = part + ((int64_t)(p.split * 2 + k) * p.M + m) * p.N + n;
                    if (whole)
                        *reinterpret_cast<f32x4*>(to) = v;
                    else
                        for (int i = 0; i < 4 && n + i < p.N; ++i) to[i] = v[i];
                }
            }
        });
    }
};
// They are added and finished.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_gated_join(const float* part, int splits, int M, int N, Gate<T> e) {
    const int across = (N + 3) / 4;
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int m = (int)(i / across), n = (int)(i % across) * 4;
    if (m >= M) return;
    f32x4 v[2] = {};
    for (int s = 0; s < splits; ++s)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float* p = part + ((int64_t)(s * 2 + k) * M + m) * N + n;
            for (int j = 0; j < 4; ++j)
                if (n + j < N) v[k][j] += p[j];
        }
    e.out4(m, n, N, v[0], v[1]);
}

// --------------------------------------------------------------- the slopes
// dg and du from dy, g and u, rows padded to whole chunks.  Bound by memory: 8192
// x 14336 bf16, 1.64 GB read and written, 293 us (5.6 TB/s).
struct GateSlope {
    const void* dy;
    const float *g, *u;
    void *dg, *du;
    int act, M, N;
    int64_t ld;
    bool whole;  // rows of whole fours, aligned
};
template <typename T>
__global__ __launch_bounds__(kThreads) void k_gated_slopes(GateSlope a) {
    const int across = (int)(a.ld / 4);
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int m = (int)(i / across), n = (int)(i % across) * 4;
    if (m >= a.M) return;
    const int64_t at = (int64_t)m * a.N + n;
    const T* dy = static_cast<const T*>(a.dy) + at;
    float v[4] = {}, g[4] = {}, u[4] = {}, dg[4], du[4];
    if (a.whole) {
        if (n < a.N) get4(dy, v), get4(a.g + at, g), get4(a.u + at, u);
    } else {
        for (int j = 0; j < 4 && n + j < a.N; ++j) v[j] = to_f(dy[j]), g[j] = a.g[at + j], u[j] = a.u[at + j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        dg[j] = v[j] * u[j] * act_slope(g[j], a.act);
        du[j] = v[j] * act_of(g[j], a.act);
    }
    put4(static_cast<T*>(a.dg) + m * a.ld + n, dg);
    put4(static_cast<T*>(a.du) + m * a.ld + n, du);
}

// ---------------------------------------------------------------- host side
inline bool gated_ok(const spec_dtype& d, long long M, long long N, long long K) {
    const int t = value_of(d);
    return (t == SPEC_BF16 || t == SPEC_F32) && M >= 1 && N >= 1 && K >= 1 && M <= SPEC_MAX_LINEAR && N <= SPEC_MAX_LINEAR &&
           K <= SPEC_MAX_LINEAR && M * N < (1ll << 33) && M * K < (1ll << 33) && N * K < (1ll << 33);
}

// Rows whose length is no whole number of chunks are copied to padded ones where
// more than 16 rows of x use them, so that tiles are loaded straight to LDS.
inline size_t packed_bytes(spec_dtype d, long long rows, long long k) { return align_up((size_t)(rows * padded(d, k)) * elem(d), 256); }
inline bool packs_pair(spec_dtype d, long long M, long long K) {
    return padded(d, K) != K && M > 16;
}
struct Pads {
    const void* from[3];
    void* to[3];
    int64_t end[3];  // rows up to the end of each
};
template <typename T>
__global__ __launch_bounds__(kThreads) void k_pad_rows(Pads a, int K, int64_t ld, int64_t first) {
    constexpr int kElems = 16 / (int)sizeof(T);
    const int64_t across = ld / kElems, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    int64_t m = first + i / across;
    if (m >= a.end[2]) return;
    const int which = m >= a.end[1] ? 2 : m >= a.end[0], k = (int)(i % across) * kElems;
    if (which) m -= a.end[which - 1];
    *reinterpret_cast<u32x4*>(static_cast<T*>(a.to[which]) + m * ld + k) = chunk_of(static_cast<const T*>(a.from[which]) + m * K, k, K);
}
// x, gate and up, those that are asked for (else null), padded into ws one after
// the other; returns where they are
struct Padded {
    const void *x, *gate, *up;
    int64_t ld;
};
template <typename T>
Padded pad_rows(const void* x, const void* gate, const void* up, spec_dtype d, int M, int N, int K, char* ws, hipStream_t st) {
    const int64_t ld = padded(d, K);
    char *px = ws, *pg = px + packed_bytes(d, M, K), *pu = pg + packed_bytes(d, N, K);
    Pads a{{x, gate, up}, {px, pg, pu}, {}};
    a.end[0] = x ? M : 0;
    a.end[1] = a.end[0] + (gate ? N : 0);
    a.end[2] = a.end[1] + (up ? N : 0);
    // one launch, but its threads are counted in 32 bits
    const int64_t across = ld / (16 / (int64_t)sizeof(T)), most = ((1ll << 32) - kThreads) / across;
    for (int64_t m = 0; m < a.end[2]; m += most) {
        const int64_t rows = a.end[2] - m < most ? a.end[2] - m : most;
        k_pad_rows<T><<<(unsigned)((rows * across + kThreads - 1) / kThreads), kThreads, 0, st>>>(a, K, ld, m);
    }
    return {px, pg, pu, ld};
}

inline Plan gated_plan(spec_dtype d, long long M, long long N, long long K) { return plan_of(d, M, 2 * N, K, 1, kAnySums, true); }
inline size_t gated_packs(spec_dtype d, long long M, long long N, long long K) {
    return packs_pair(d, M, K) ? packed_bytes(d, M, K) + 2 * packed_bytes(d, N, K) : 0;
}
inline size_t gated_bytes(spec_dtype d, long long M, long long N, long long K) {
    const int s = M > 16 ? gated_plan(d, M, N, K).splits : 1;
    return gated_packs(d, M, N, K) + (s > 1 ? align_up((size_t)(2 * s * M * N) * 4, 256) : 0) + 256;
}
template <typename T, class E>
void launch_pair(const Product& g, const E& e, Size size, hipStream_t st) {
    if (!aligned(g, sizeof(T)))
        launch_tile<Tile<T, 64, 128, 32, 64, 2, false, false, true, false>>(g, e, st);
    else if (size == kTile256)
        launch_tile<Tile<T, 256, 256, 128, 128, 2, false, false, true, true>>(g, e, st);
    else if (size == kTile192)
        launch_tile<Tile<T, 192, 128, 96, 64, 3, false, false, true, true>>(g, e, st);
    else if (size == kTile128)
        launch_tile<Tile<T, 128, 128, 64, 64, 4, false, false, true, true>>(g, e, st);
    else
        launch_tile<Tile<T, 64, 128, 32, 64, 3, false, false, true, true>>(g, e, st);
}

template <typename T>
void gated_forward(Product g, const Gate<T>& e, spec_dtype d, char* ws, hipStream_t st) {
    if (g.M <= 16) {
        const unsigned grid = (unsigned)((g.N + 15) / 16);
        if (aligned(g, sizeof(T)))
            k_gated_few<T, true><<<grid, kThreads, 0, st>>>(g, e);
        else
            k_gated_few<T, false><<<grid, kThreads, 0, st>>>(g, e);
        return;
    }
    const int k = g.K;
    const Plan plan = gated_plan(d, g.M, g.N, k);
    if (packs_pair(d, g.M, g.K)) {
        const Padded p = pad_rows<T>(g.x[0], g.w[0], g.w[1], d, g.M, g.N, g.K, ws, st);
        g.x[0] = g.x[1] = p.x, g.w[0] = p.gate, g.w[1] = p.up;
        g.ldx = g.ldw = p.ld;
        g.K = (int)p.ld;  // the padding is zero
    }
    if (plan.splits == 1) {
        launch_pair<T>(g, e, plan.size, st);
        return;
    }
    float* part = reinterpret_cast<float*>(ws + gated_packs(d, g.M, g.N, k));
    g.splits = plan.splits;
    launch_pair<T>(g, GateSums{{}, part, fours(part, g.N, 4)}, plan.size, st);
    k_gated_join<T><<<four_blocks(g.M, g.N), kThreads, 0, st>>>(part, plan.splits, g.M, g.N, e);
}

// The gradients' workspace: dg and du, and the sums of split products.
struct GatedLayout {
    int64_t np;
    size_t dg, du, packed, sums, total;
    Plan x, w;
};
inline GatedLayout gated_layout(spec_dtype d, long long M, long long N, long long K) {
    GatedLayout l;
    l.np = padded(d, N);
    l.dg = 0;
    l.du = align_up((size_t)(M * l.np) * elem(d), 256);
    l.packed = 2 * l.du;
    l.sums = l.packed + (packs_pair(d, M, K) ? packed_bytes(d, M, K) + 2 * packed_bytes(d, N, K) : 0);
    l.x = plan_of(d, M, K, 2 * N, 1, kAnySums, false);
    l.w = plan_of(d, N, K, M, 2, kAnySums, false);
    const size_t a = l.x.splits > 1 ? (size_t)(l.x.splits * M * K) * 4 : 0, b = l.w.splits > 1 ? (size_t)(2 * l.w.splits * N * K) * 4 : 0;
    l.total = l.sums + align_up(a > b ? a : b, 256);
    return l;
}

template <typename T>
void gated_backward(const void* x, const void* gate, const void* up, const float* g, const float* u, const void* dy, int act,
                    int M, int N, int K, void* gx, void* gg, void* gu, spec_dtype d, char* ws, hipStream_t st) {
    const GatedLayout lay = gated_layout(d, M, N, K);
    void *dg = ws + lay.dg, *du = ws + lay.du;
    float* sums = reinterpret_cast<float*>(ws + lay.sums);
    const bool whole = fours(g, N, 4) && fours(u, N, 4) && fours(dy, N, sizeof(T));
    k_gated_slopes<T><<<four_blocks(M, lay.np), kThreads, 0, st>>>({dy, g, u, dg, du, act, M, N, lay.np, whole});
    int64_t ld = K;
    if (packs_pair(d, M, K)) {
        const Padded p = pad_rows<T>(gg || gu ? x : nullptr, gx ? gate : nullptr, gx ? up : nullptr, d, M, N, K, ws + lay.packed, st);
        x = p.x, gate = p.gate, up = p.up, ld = p.ld;
    }
    if (gx) {
        const Product p{{dg, du}, {gate, up}, lay.np, ld, M, K, N, N, nullptr, nullptr, 1, lay.x.splits, 0};
        if (lay.x.splits > 1) {
            launch_product<T, false, true>(p, Store<float>{{}, {sums, sums}, K, (int64_t)M * K, false, fours(sums, K, 4)}, lay.x.size, st);
            join(sums, lay.x.splits, nullptr, {}, M, K, static_cast<T*>(gx), st);
        } else {
            launch_product<T, false, true>(p, Store<T>{{}, {static_cast<T*>(gx), static_cast<T*>(gx)}, K, 0, false, fours(gx, K, sizeof(T))}, lay.x.size, st);
        }
    }
    if (gg || gu) {
        // both in one launch where both are asked for
        const void *a = gg ? dg : du, *b = gu ? du : dg;
        T *oa = static_cast<T*>(gg ? gg : gu), *ob = static_cast<T*>(gu ? gu : gg);
        const int products = gg && gu ? 2 : 1;
        const Product p{{a, b}, {x, x}, lay.np, ld, N, K, M, 0, nullptr, nullptr, products, lay.w.splits, 0};
        if (lay.w.splits > 1) {
            const int64_t one = (int64_t)N * K;
            float* second = sums + lay.w.splits * one;
            launch_product<T, true, true>(p, Store<float>{{}, {sums, second}, K, one, false, fours(sums, K, 4)}, lay.w.size, st);
            join(sums, lay.w.splits, nullptr, {}, N, K, oa, st);
            if (products == 2) join(second, lay.w.splits, nullptr, {}, N, K, ob, st);
        } else {
            const bool four = fours(oa, K, sizeof(T)) && fours(ob, K, sizeof(T));
            launch_product<T, true, true>(p, Store<T>{{}, {oa, ob}, K, 0, false, four}, lay.w.size, st);
        }
    }
}

}  // namespace

extern "C" size_t spec_gated_linear_workspace_bytes(spec_dtype dtype, int M, int N, int K) {
    if (!gated_ok(dtype, M, N, K)) return 0;
    return gated_bytes(dtype, M, N, K);
}

extern "C" spec_status spec_gated_linear(const void* x, const void* gate, const void* up, spec_dtype dtype,
                                         spec_activation activation, int M, int N, int K, void* out, float* out_gate,
                                         float* out_up, void* workspace, size_t workspace_bytes, void* stream) {
    if (!type_ok(dtype)) return SPEC_EDTYPE;
    if (!gated_ok(dtype, M, N, K) || !act_ok(activation) || !x || !gate || !up || !out || !out_gate != !out_up) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_gated_linear_workspace_bytes(dtype, M, N, K))) return SPEC_EWORKSPACE;
    const Product g{{x, x}, {gate, up}, K, K, M, N, K, 0, nullptr, nullptr, 1, 1, 0};
    const bool whole = fours(out, N, elem(dtype)) && fours(out_gate, N, 4) && fours(out_up, N, 4);
    char* ws = static_cast<char*>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (value_of(dtype) == SPEC_BF16)
        gated_forward(g, Gate<bf16>{{}, (bf16*)out, out_gate, out_up, activation, whole}, dtype, ws, st);
    else
        gated_forward(g, Gate<float>{{}, (float*)out, out_gate, out_up, activation, whole}, dtype, ws, st);
    return launched();
}

extern "C" size_t spec_gated_linear_grad_workspace_bytes(spec_dtype dtype, int M, int N, int K) {
    return gated_ok(dtype, M, N, K) ? gated_layout(dtype, M, N, K).total : 0;
}

extern "C" spec_status spec_gated_linear_grad(const void* x, const void* gate, const void* up, const float* gate_preact,
                                              const float* up_preact, const void* grad_out, spec_dtype dtype,
                                              spec_activation activation, int M, int N, int K, void* grad_x, void* grad_gate,
                                              void* grad_up, void* workspace, size_t workspace_bytes, void* stream) {
    if (!type_ok(dtype)) return SPEC_EDTYPE;
    if (!gated_ok(dtype, M, N, K) || !act_ok(activation) || !gate_preact || !up_preact || !grad_out) return SPEC_EINVAL;
    if ((grad_x && (!gate || !up)) || ((grad_gate || grad_up) && !x)) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_gated_linear_grad_workspace_bytes(dtype, M, N, K))) return SPEC_EWORKSPACE;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    if (value_of(dtype) == SPEC_BF16)
        gated_backward<bf16>(x, gate, up, gate_preact, up_preact, grad_out, activation, M, N, K, grad_x, grad_gate, grad_up, dtype, ws, st);
    else
        gated_backward<float>(x, gate, up, gate_preact, up_preact, grad_out, activation, M, N, K, grad_x, grad_gate, grad_up, dtype, ws, st);
    return launched();
}

// cross_entropy.hip -- the cross entropy of given tokens under a draft head's
// output layer, for gfx950 (MI355X), whose logits are never kept.
//
//   z = x W^T + bias                 x [M][K], W [V][K], bias [V]
//   top = max z, S = sum e^(z - top), lse = top + ln S
//   loss = ln S - (z[token] - top)
//   p = e^(z - top) / S, dz = (dloss + dlse) p - dloss [token]
//   dx = dz W, dW = dz^T x, dbias = sum over rows of dz
// Forward, a tile of the product leaves only its rows' maxima and sums, which
// one more launch folds.  Backward, the product is computed once more, a piece
// of the vocabulary after the other, and dz of a piece is used for both
// gradients before the next.  Products, sums and dx over the pieces are fp32;
// with bf16 operands dz is rounded to bf16, as an operand of the matrix
// instructions, and the bias gradient sums unrounded dz.
#include "product.h"

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
__device__ inline float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2e); }

// --------------------------------------------------------------- rows in use
// Rows of padded tokens are left out of the products: live[i] is the i-th row
// in use and place[r] its number i, -1 where row r is not in use.
struct Outputs {
    float *loss, *lse, *stats;
    int32_t* status;
};
// Outputs of a row whose token is x, if it is not in use; returns whether it is.
__device__ inline bool in_use(const Outputs& o, int64_t r, int x, int V) {
    const bool in = x >= 0 && x < V;
    if (o.status) {
        o.status[r] = x < -1 || x >= V;
        if (!in) {
            o.loss[r] = o.lse[r] = 0.f;
            if (o.stats) o.stats[2 * r] = o.stats[2 * r + 1] = 0.f;
        }
    }
    return in;
}
struct Rows {
    const int32_t* tokens;
    int M, V;
    int *live, *place, *count;
    Outputs out;  // forward
};
constexpr int kLiveThreads = 1024;
__global__ __launch_bounds__(kLiveThreads) void k_live(Rows a) {
    __shared__ int waves[kLiveThreads / 64];
    const int t = threadIdx.x, lane = t & 63, w = t >> 6;
    int before = 0;
    for (int r0 = 0; r0 < a.M; r0 += kLiveThreads) {
        const int r = r0 + t;
        const bool in = r < a.M && in_use(a.out, r, a.tokens[r], a.V);
        const uint64_t mask = __ballot(in);
        if (lane == 0) waves[w] = __popcll(mask);
        __syncthreads();
        int at = before;
        for (int i = 0; i < kLiveThreads / 64; ++i) {
            if (i < w) at += waves[i];
            before += waves[i];
        }
        at += __popcll(mask & ((1ull << lane) - 1));
        if (in) a.live[at] = r;
        if (r < a.M) a.place[r] = in ? at : -1;
        __syncthreads();
    }
    if (t == 0) *a.count = before;
}

// The rows in use, packed one after the other, zero up to `ld`; or (live null)
// all rows padded.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_pack(const T* x, const int* live, const int* count, int64_t rows, int K, int64_t ld, T* to) {
    constexpr int kElems = 16 / (int)sizeof(T);
    const int64_t across = ld / kElems, i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t m = i / across;
    if (m >= (live ? (int64_t)*count : rows)) return;
    const int k = (int)(i % across) * kElems;
    *reinterpret_cast<u32x4*>(to + m * ld + k) = chunk_of(x + (live ? (int64_t)live[m] : m) * K, k, K);
}

// ------------------------------------------------------------------- forward
struct MaxSum {
    float top, sum;  // a maximum, and the sum of e^(z - top)
};
__device__ inline MaxSum joined(MaxSum a, MaxSum b) {
    const float top = fmaxf(a.top, b.top);
    // where nothing but -inf was seen, both sums are 0 (or NaN, which stays)
    const float ref = top == -INFINITY ? 0.f : top;
    return {top, a.sum * exp_of(a.top - ref) + b.sum * exp_of(b.top - ref)};
}

// f(value) for a lane's values of the j-th kB rows.
template <class C, class J, typename F>
__device__ __attribute__((always_inline)) inline void values(typename C::Acc (&acc)[C::FN][C::FM], J j, F f) {
    each(std::make_integer_sequence<int, C::FN * C::kV>(), [&](auto u) __attribute__((always_inline)) {
        constexpr int i = u / C::kV, v = u % C::kV;
        acc[i][j][v] = f(acc[i][j][v]);
    });
}
// Logits: their sums start from the bias, and from -inf past the last column.
template <typename T>
struct Logits {
    const T* bias;  // or null
    template <class C>
    __device__ __attribute__((always_inline)) void start(const Part& p, typename C::Acc (&acc)[C::FN][C::FM]) const {
        if (!bias && p.n0 + C::WN <= p.N) return;
        each(std::make_integer_sequence<int, C::FN * C::kV>(), [&](auto u) __attribute__((always_inline)) {
            constexpr int i = u / C::kV, v = u % C::kV;
            const int n = p.n0 + i * C::kB + v / 4 * 8 + p.lane / C::kB * 4 + v % 4;
            const float b = n >= p.N ? -INFINITY : bias ? to_f(bias[n]) : 0.f;
#pragma unroll
            for (int j = 0; j < C::FM; ++j) acc[i][j][v] = b;
        });
    }
};

// Leaves each row's maximum and sum over the tile's columns, part [tile][M],
// and the row's token's logit.  A lane has the columns of one row, so that most
// of it is done without a word to another lane.  7373 x 128256 x 4096 bf16 5.7 to
// 5.9 ms (1310 to 1360 TFLOP/s); 6 rows 155 us, W read at 6.8 TB/s.
template <typename T>
struct Stats : Logits<T> {
    const int32_t* tokens;
    const int* live;  // or null: every row
    int v0;           // the product's first column in the vocabulary
    int rows;         // of `part`
    MaxSum* part;
    float* picked;
    template <class C>
    __device__ __attribute__((always_inline)) void finish(const Part& p, typename C::Acc (&acc)[C::FN][C::FM]) const {
        const int l = p.lane % C::kB;
        const bool first = p.lane < C::kB;  // of the lanes that share a row
        MaxSum* red = reinterpret_cast<MaxSum*>(p.lds);
        MaxSum all[C::FM];
        each(std::make_integer_sequence<int, C::FM>(), [&](auto j) __attribute__((always_inline)) {
            const int m = p.m0 + j * C::kB + l;
            float top = -INFINITY, sum = 0.f;
            values<C>(acc, j, [&](float z) __attribute__((always_inline)) { return top = fmaxf(top, z), z; });
            const float ref = top == -INFINITY ? 0.f : top;
            values<C>(acc, j, [&](float z) __attribute__((always_inline)) { return sum += exp_of(z - ref), z; });
            all[j] = {top, sum};
#pragma unroll
            for (int s = C::kB; s < 64; s *= 2) all[j] = joined(all[j], {__shfl_xor(all[j].top, s), __shfl_xor(all[j].sum, s)});
            const int x = m < p.M ? tokens[live ? live[m] : m] - v0 - p.n0 : -1;
            const bool here = x >= 0 && x < C::WN && p.n0 + x < p.N;
            if (__ballot(here) == 0) return;
            lay<C>(p, acc, std::integral_constant<int, j * C::kB / 32>());
            if (here && first) picked[m] = rows_of<C>(p)[(j * C::kB % 32 + l) * (C::WN + 4) + x];
            settle();
        });
        __syncthreads();
        if (first)
#pragma unroll
            for (int j = 0; j < C::FM; ++j) red[p.w % C::kWavesN * C::BM + p.w / C::kWavesN * C::WM + j * C::kB + l] = all[j];
        __syncthreads();
        const int t = threadIdx.x, m = p.tm * C::BM + t;
        if (t < C::BM && m < p.M) {
            MaxSum v = red[t];
#pragma unroll
            for (int i = 1; i < C::kWavesN; ++i) v = joined(v, red[i * C::BM + t]);
            part[(int64_t)p.tn * rows + m] = v;
        }
    }
};

// The outputs of row r from its maximum, sum and token's logit.  stats: the
// maximum and 1 / S, both 0 for a row of -inf alone.
__device__ inline void finish_row(const Outputs& o, int64_t r, int x, int V, MaxSum v, float picked) {
    if (!in_use(o, r, x, V)) return;
    const bool some = v.top != -INFINITY || v.sum != v.sum;
    const float ls = logf(v.sum);
    o.loss[r] = some ? ls - (picked - v.top) : INFINITY;
    o.lse[r] = some ? v.top + ls : -INFINITY;
    if (o.stats) {
        o.stats[2 * r] = some ? v.top : 0.f;
        o.stats[2 * r + 1] = some ? 1.f / v.sum : 0.f;
    }
}

// Folds the tiles' parts of each row in use and writes the outputs of its row:
// `across` rows a workgroup, the parts of each over the other threads.
struct Fold {
    const MaxSum* part;
    const float* picked;
    const int32_t* tokens;
    const int *live, *count;  // or null: every row
    int M, V, parts, across;
    Outputs out;
};
__global__ __launch_bounds__(kLiveThreads) void k_fold(Fold a) {
    __shared__ MaxSum red[kLiveThreads];
    const int t = threadIdx.x, c = t % a.across, g = t / a.across, groups = kLiveThreads / a.across;
    const int rows = a.live ? *a.count : a.M, m = blockIdx.x * a.across + c;
    if ((int)blockIdx.x * a.across >= rows) return;
    MaxSum v = {-INFINITY, 0.f};
    if (m < rows)
        for (int i = g; i < a.parts; i += groups) v = joined(v, a.part[(int64_t)i * a.M + m]);
    red[t] = v;
    __syncthreads();
    for (int s = groups / 2; s > 0; s /= 2) {
        if (g < s) red[t] = joined(red[t], red[t + s * a.across]);
        __syncthreads();
    }
    if (g != 0 || m >= rows) return;
    const int64_t r = a.live ? a.live[m] : m;
    finish_row(a.out, r, a.tokens[r], a.V, red[t], a.picked[m]);
}

// Where the product's sum over k is split, because its tiles are few, the splits'
// sums of the logits are in memory, part [split][M][V] (a few million in all).
struct Small {
    const float* part;
    int splits, M, V;
    const void* bias;
    const int32_t* tokens;
    const int *live, *count;  // or null: every row
};
template <typename T>
__device__ inline float logit(const Small& a, int m, int v) {
    float z = a.bias ? to_f(static_cast<const T*>(a.bias)[v]) : 0.f;
    for (int s = 0; s < a.splits; ++s) z += a.part[((int64_t)s * a.M + m) * a.V + v];
    return z;
}
template <typename T>
__global__ __launch_bounds__(kThreads) void k_small_stats(Small a, Outputs out) {
    __shared__ MaxSum red[kThreads];
    __shared__ float picked;
    const int m = blockIdx.x, t = threadIdx.x;
    if (a.live && m >= *a.count) return;
    const int64_t r = a.live ? a.live[m] : m;
    const int x = a.tokens[r];
    MaxSum all = {-INFINITY, 0.f};
    for (int v = t; v < a.V; v += kThreads) {
        const float z = logit<T>(a, m, v);
        all = joined(all, {z, z == -INFINITY ? 0.f : z == z ? 1.f : z});
        if (v == x) picked = z;
    }
    red[t] = all;
    __syncthreads();
    for (int s = kThreads / 2; s > 0; s /= 2) {
        if (t < s) red[t] = joined(red[t], red[t + s]);
        __syncthreads();
    }
    if (t == 0) finish_row(out, r, x, a.V, red[0], picked);
}

// ------------------------------------------------------------------ backward
// What dz of a row needs: dz = both p - one [token].
struct Weights {
    const float *stats, *g_loss, *g_lse;  // a gradient may be null
};
struct RowWeights {
    float top, inv, one, both;
    __device__ float of(float z) const {
        // p from the difference itself; 0 whatever the weight where p = 0
        const float q = exp_of(z - top) * inv;
        return q == 0.f ? 0.f : both * q;
    }
};
__device__ inline RowWeights weights_of(const Weights& a, int64_t r) {
    RowWeights w{a.stats[2 * r], a.stats[2 * r + 1], 0.f, 0.f};
    w.one = a.g_loss && w.inv != 0.f ? a.g_loss[r] : 0.f;
    w.both = w.one + (a.g_lse ? a.g_lse[r] : 0.f);
    return w;
}

// From the logits in memory; dz unrounded takes the first split's place.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_small_slope(Small a, Weights weights, T* dz, int64_t ld) {
    const int m = blockIdx.x;
    if (m >= *a.count) return;
    const int64_t r = a.live[m];
    const int x = a.tokens[r];
    const RowWeights w = weights_of(weights, r);
    float* first = const_cast<float*>(a.part) + (int64_t)m * a.V;
    for (int v = threadIdx.x; v < a.V; v += kThreads) {
        float d = w.of(logit<T>(a, m, v));
        if (v == x) d -= w.one;
        first[v] = d;
        put(dz + m * ld + v, d);
    }
}

// A product's tiles, and the waves that share a tile's rows out.
struct Tiling {
    int bm, bn, waves_m;
};
// The waves' shares of `rows` rows: of whole tiles, since a wave of a tile
// writes its sums whether or not it has a row.
__host__ __device__ inline int wave_rows(int rows, const Tiling& t) { return (rows + t.bm - 1) / t.bm * t.waves_m; }

// Turns a piece's logits, columns v0 on, into dz, rounded, dz [rows][ld]; and
// its columns' sums over each wave's rows, unrounded, part [wave_rows][V].
template <typename T>
struct Slope : Logits<T> {  // the bias: of the piece
    const int32_t* tokens;
    const int* live;
    Weights weights;
    int v0, V;
    T* dz;
    int64_t ld;
    float* part;  // or null
    template <class C>
    __device__ __attribute__((always_inline)) void finish(const Part& p, typename C::Acc (&acc)[C::FN][C::FM]) const {
        const int l = p.lane % C::kB;
        const bool first = p.lane < C::kB;  // of the lanes that share a row
        constexpr int kLanes = C::WN / 4, kAtOnce = 64 / kLanes, kPitch = C::WN + 4;
        const int c = p.lane % kLanes * 4, n = p.n0 + c;
        float sum[4] = {};
        each(std::make_integer_sequence<int, C::WM / 32>(), [&](auto j) __attribute__((always_inline)) {
            constexpr int kBlocks = 32 / C::kB;
            int at[kBlocks];
            float minus[kBlocks];
            each(std::make_integer_sequence<int, kBlocks>(), [&](auto k) __attribute__((always_inline)) {
                const int m = p.m0 + j * 32 + k * C::kB + l;
                RowWeights row{0.f, 0.f, 0.f, 0.f};
                at[k] = -1;
                if (m < p.M) {
                    const int r = live[m];
                    row = weights_of(weights, r);
                    at[k] = tokens[r] - v0 - p.n0;
                }
                minus[k] = row.one;
                values<C>(acc, std::integral_constant<int, j * kBlocks + k>(), [&](float z) __attribute__((always_inline)) { return row.of(z); });
            });
            lay<C>(p, acc, j);
            float* rows = rows_of<C>(p);
#pragma unroll
            for (int k = 0; k < kBlocks; ++k)
                if (first && at[k] >= 0 && at[k] < C::WN) rows[(k * C::kB + l) * kPitch + at[k]] -= minus[k];
            settle();
            if (n < p.N)
#pragma unroll 4
                for (int r = p.lane / kLanes; r < 32; r += kAtOnce) {
                    const int row = p.m0 + j * 32 + r;
                    if (row >= p.M) break;
                    const f32x4 q = *reinterpret_cast<const f32x4*>(rows + r * kPitch + c);
                    put4(dz + row * ld + n, {q[0], q[1], q[2], q[3]});  // ld has whole fours
                    if (part)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[i] += q[i];
                }
            settle();
        });
        if (!part) return;
#pragma unroll
        for (int s = kLanes; s < 64; s *= 2)
#pragma unroll
            for (int i = 0; i < 4; ++i) sum[i] += __shfl_xor(sum[i], s);
        if (p.lane < kLanes)
            for (int i = 0; i < 4 && n + i < p.N; ++i)
                part[(int64_t)(p.tm * C::kWavesM + p.w / C::kWavesN) * V + v0 + n + i] = sum[i];
    }
};

// dbias[v] = the sum of the parts, in a fixed order: 64 columns a workgroup,
// every sixteenth part to a wave.
template <typename T>
__global__ __launch_bounds__(kLiveThreads) void k_bias_fold(const float* part, const int* count, Tiling tiles, int V, T* out) {
    __shared__ float sums[kLiveThreads / 64][64];
    const int c = threadIdx.x & 63, w = threadIdx.x >> 6, n = blockIdx.x * 64 + c;
    const int parts = wave_rows(*count, tiles);
    float s = 0.f;
    if (n < V)
        for (int i = w; i < parts; i += kLiveThreads / 64) s += part[(int64_t)i * V + n];
    sums[w][c] = s;
    __syncthreads();
    if (w == 0 && n < V) {
        for (int i = 1; i < kLiveThreads / 64; ++i) s += sums[i][c];
        put(out + n, s);
    }
}

// ---------------------------------------------------------------- host side
inline bool entropy_ok(const spec_dtype& d, long long M, long long V, long long K) {
    const int t = value_of(d);
    return (t == SPEC_BF16 || t == SPEC_F32) && M >= 1 && V >= 1 && K >= 1 && M <= SPEC_MAX_LINEAR && V <= SPEC_MAX_LINEAR &&
           K <= SPEC_MAX_LINEAR && M * K < (1ll << 33) && V * K < (1ll << 33);
}

// The product that gives logits.  Up to 64 rows take tiles of all of them by
// 128 of W, which read W once and past the caches.
enum Shape { kRows32, kRows64, kRows192, kLogits256, kLogits128, kLogits64 };
inline Shape shape_of(spec_dtype d, long long M, long long V, long long K) {
    if (M <= 32) return kRows32;
    if (M <= 64) return kRows64;
    const Size s = plan_of(d, M, V, K, 1, kNoSums, true).size;
    return s == kTile192 ? kRows192 : s == kTile256 ? kLogits256 : s == kTile128 ? kLogits128 : kLogits64;
}
// Where W's rows are no whole chunks, they are copied to padded ones first if
// more than 64 rows use them.
inline bool packs_weight(spec_dtype d, long long M, long long K) { return padded(d, K) != K && M > 64; }
inline Tiling tiling(Shape s, bool direct) {
    if (!direct || s == kLogits64) return {64, 64, 2};
    return s == kRows32 ? Tiling{32, 128, 1} : s == kRows64 ? Tiling{64, 128, 1} : s == kRows192 ? Tiling{192, 128, 2} : s == kLogits256 ? Tiling{256, 256, 2} : Tiling{128, 128, 2};
}
// The columns that one launch of such tiles takes: all, or whole tiles of them,
// so that its threads are counted in 32 bits (64 x 64: M V up to some 2^36).
inline int launch_columns(int M, int V, const Tiling& t) {
    const long long most = ((1ll << 32) / kThreads - 1) / ((M + t.bm - 1) / t.bm) * t.bn;
    return V < most ? V : (int)most;
}
template <typename T, class E>
void launch_logits(const Product& g, const E& e, Shape s, hipStream_t st) {
    if (!aligned(g, sizeof(T)))
        launch_tile<Tile<T, 64, 64, 32, 32, 2, false, false, false, false>>(g, e, st);
    else if (s == kRows32)
        launch_tile<Tile<T, 32, 128, 32, 32, 4, false, false, false, true, true>>(g, e, st);
    else if (s == kRows64)
        launch_tile<Tile<T, 64, 128, 64, 32, 3, false, false, false, true, true>>(g, e, st);
    else if (s == kRows192)
        launch_tile<Tile<T, 192, 128, 96, 64, 3, false, false, false, true>>(g, e, st);
    else
        launch_product<T, false, false>(g, e, s == kLogits256 ? kTile256 : s == kLogits128 ? kTile128 : kTile64, st);
}

template <typename T>
void pack(const void* x, const int* live, const int* count, long long rows, int K, int64_t ld, void* to, hipStream_t st) {
    const int64_t n = rows * (ld / (16 / (int64_t)sizeof(T)));
    k_pack<T><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(static_cast<const T*>(x), live, count, rows, K, ld, static_cast<T*>(to));
}
inline size_t matrix_bytes(spec_dtype d, long long rows, long long ld) { return align_up((size_t)(rows * ld) * elem(d), 256); }

// Few tiles of a long sum: it is split, as far as the logits of all splits stay
// within kSumsBytes.  By time alone they would take 8.4 GB of 16384 x 32000 x 65536
// fp32 (four splits).  Half of it costs 36838 x 2615 x 52288 bf16 its two splits:
// 9.9 -> 11.4 ms.
constexpr long long kSumsBytes = 1ll << 30;
inline Plan small_plan(spec_dtype d, long long M, long long V, long long K) { return plan_of(d, M, V, K, 1, kSumsBytes, false); }
inline size_t small_bytes(const Plan& p, long long M, long long V) { return p.splits > 1 ? align_up((size_t)(p.splits * M * V) * 4, 256) : 0; }

struct ForwardLayout {
    Plan small;
    size_t live, place, count, x, w, part, picked, total;
    bool few, packs;
};
inline ForwardLayout forward_layout(spec_dtype d, long long M, long long V, long long K) {
    ForwardLayout l;
    l.few = M <= 64;
    l.packs = packs_weight(d, M, K);
    l.small = small_plan(d, M, V, K);
    l.live = 0;
    l.place = align_up(l.live + (l.few ? 0 : M * 4), 256);
    l.count = align_up(l.place + (l.few ? 0 : M * 4), 256);
    l.x = l.count + 256;
    l.w = l.x + (l.few ? 0 : matrix_bytes(d, M, padded(d, K)));
    l.part = l.w + (l.packs ? matrix_bytes(d, V, padded(d, K)) : 0);
    l.picked = align_up(l.part + (l.small.splits > 1 ? small_bytes(l.small, M, V) : (size_t)((V + 63) / 64 * M) * sizeof(MaxSum)), 256);
    l.total = align_up(l.picked + M * 4, 256);
    return l;
}

template <typename T>
void entropy_forward(const void* x, const void* weight, const void* bias, const int32_t* tokens, int M, int V, int K, float* loss,
                     float* lse, int32_t* status, float* stats, spec_dtype d, char* ws, hipStream_t st) {
    const ForwardLayout lay = forward_layout(d, M, V, K);
    int *live = reinterpret_cast<int*>(ws + lay.live), *count = reinterpret_cast<int*>(ws + lay.count);
    const int64_t ld = padded(d, K);
    MaxSum* part = reinterpret_cast<MaxSum*>(ws + lay.part);
    float* picked = reinterpret_cast<float*>(ws + lay.picked);
    Product g{{x, x}, {weight, weight}, K, K, M, V, K, 0, nullptr, nullptr, 1, 1, 0};
    const Outputs out{loss, lse, stats, status};
    if (lay.few) {
        live = count = nullptr;
    } else {
        k_live<<<1, kLiveThreads, 0, st>>>({tokens, M, V, live, reinterpret_cast<int*>(ws + lay.place), count, out});
        pack<T>(x, live, count, M, K, ld, ws + lay.x, st);
        g.x[0] = g.x[1] = ws + lay.x;
        g.ldx = ld;
        g.live_m = count;
        if (lay.packs) {
            pack<T>(weight, nullptr, nullptr, V, K, ld, ws + lay.w, st);
            g.w[0] = g.w[1] = ws + lay.w;
            g.ldw = ld;
            g.K = (int)ld;  // the padding is zero
        }
    }
    if (lay.small.splits > 1) {
        float* z = reinterpret_cast<float*>(ws + lay.part);
        g.splits = lay.small.splits;
        launch_product<T, false, false>(g, Store<float>{{}, {z, z}, V, (int64_t)M * V, false, fours(z, V, 4)}, lay.small.size, st);
        k_small_stats<T><<<M, kThreads, 0, st>>>({z, g.splits, M, V, bias, tokens, live, count}, out);
        return;
    }
    const Shape s = shape_of(d, M, V, K);
    const Tiling t = tiling(s, aligned(g, sizeof(T)));
    const int bn = t.bn, piece = launch_columns(M, V, t);
    const T *w = static_cast<const T*>(g.w[0]), *b = static_cast<const T*>(bias);
    for (int v0 = 0; v0 < V; v0 += piece) {
        g.N = V - v0 < piece ? V - v0 : piece;
        g.w[0] = g.w[1] = w + v0 * g.ldw;
        launch_logits<T>(g, Stats<T>{{b ? b + v0 : nullptr}, tokens, live, v0, M, part + (int64_t)(v0 / bn) * M, picked}, s, st);
    }
    int across = 1;
    while (across < M && across < 64) across *= 2;
    k_fold<<<(M + across - 1) / across, kLiveThreads, 0, st>>>({part, picked, tokens, live, count, M, V, (V + bn - 1) / bn, across, out});
}

// A piece of the vocabulary: what keeps its dz within kPieceBytes.
constexpr long long kPieceBytes = 512ll << 20;
inline int piece_of(spec_dtype d, long long M, long long V) {
    const long long fit = kPieceBytes / (M * (long long)elem(d)) / 1024 * 1024, n = fit < 1024 ? 1024 : fit;
    return (int)(n < V ? n : V);
}
struct BackwardLayout {
    size_t live, place, count, x, w, dz, dx, dw, part, total;
    int piece, more;  // more: splits of dx where few rows are in use
    Plan px, pw, small;
    bool packs;
};
inline BackwardLayout backward_layout(spec_dtype d, long long M, long long V, long long K) {
    BackwardLayout l;
    l.piece = piece_of(d, M, V);
    l.small = small_plan(d, M, V, K);
    if (l.small.splits > 1) l.piece = (int)V;
    l.packs = packs_weight(d, M, K);
    l.px = plan_of(d, M, K, l.piece, 1, kAnySums, false);
    l.pw = plan_of(d, l.piece, K, M, 1, kAnySums, false);
    // room for up to four times the compute units' tiles
    const long long b = 256 >> l.px.size, tiles = ((M + b - 1) / b) * ((K + b - 1) / b), most = 1024 / tiles;
    l.more = (int)(most > kMaxSplits ? kMaxSplits : most < l.px.splits ? l.px.splits : most);
    l.live = 0;
    l.place = align_up(l.live + M * 4, 256);
    l.count = align_up(l.place + M * 4, 256);
    l.x = l.count + 256;
    l.w = l.x + matrix_bytes(d, M, padded(d, K));
    l.dz = l.w + (l.packs ? matrix_bytes(d, V, padded(d, K)) : 0);
    l.dx = l.dz + matrix_bytes(d, M, padded(d, l.piece));
    l.dw = align_up(l.dx + (size_t)(l.more * M * K) * 4, 256);
    l.part = align_up(l.dw + (l.pw.splits > 1 ? (size_t)l.pw.splits * l.piece * K * 4 : 0), 256);
    // the tiles are those of aligned operands or not: what a call has is not known here
    const Shape s = shape_of(d, M, l.piece, K);
    const int a = wave_rows((int)M, tiling(s, true)), u = wave_rows((int)M, tiling(s, false));
    l.total = align_up(l.part + (l.small.splits > 1 ? small_bytes(l.small, M, V) : (size_t)((a > u ? a : u) * V) * 4), 256);
    return l;
}

template <typename T>
void entropy_backward(const void* x, const void* weight, const void* bias, const int32_t* tokens, const float* stats,
                      const float* g_loss, const float* g_lse, int M, int V, int K, void* gx, void* gw, void* gb, spec_dtype d,
                      char* ws, hipStream_t st) {
    const BackwardLayout lay = backward_layout(d, M, V, K);
    int *live = reinterpret_cast<int*>(ws + lay.live), *place = reinterpret_cast<int*>(ws + lay.place);
    int* count = reinterpret_cast<int*>(ws + lay.count);
    const int64_t ld = padded(d, K);
    const T *xp = reinterpret_cast<const T*>(ws + lay.x), *wp = static_cast<const T*>(weight);
    T* dz = reinterpret_cast<T*>(ws + lay.dz);
    float *dx = reinterpret_cast<float*>(ws + lay.dx), *dw = reinterpret_cast<float*>(ws + lay.dw);
    float* part = gb ? reinterpret_cast<float*>(ws + lay.part) : nullptr;
    int64_t ldw = K;
    int kz = K;
    k_live<<<1, kLiveThreads, 0, st>>>({tokens, M, V, live, place, count, {}});
    pack<T>(x, live, count, M, K, ld, ws + lay.x, st);
    if (lay.packs) {
        pack<T>(weight, nullptr, nullptr, V, K, ld, ws + lay.w, st);
        wp = reinterpret_cast<const T*>(ws + lay.w);
        ldw = ld;
        kz = (int)ld;
    }
    const Shape shape = shape_of(d, M, lay.piece, K);
    const int64_t ldz = padded(d, lay.piece);
    Tiling tiles{};
    int dx_tile = 64;
    for (int v0 = 0; v0 < V; v0 += lay.piece) {
        const int n = V - v0 < lay.piece ? V - v0 : lay.piece;
        const T* w = wp + v0 * ldw;
        const Product z{{xp, xp}, {w, w}, ld, ldw, M, n, kz, 0, count, nullptr, 1, 1, 0};
        if (lay.small.splits > 1) {
            float* logits = reinterpret_cast<float*>(ws + lay.part);
            Product split = z;
            split.splits = lay.small.splits;
            launch_product<T, false, false>(split, Store<float>{{}, {logits, logits}, V, (int64_t)M * V, false, fours(logits, V, 4)}, lay.small.size, st);
            k_small_slope<T><<<M, kThreads, 0, st>>>({logits, split.splits, M, V, bias, tokens, live, count}, {stats, g_loss, g_lse}, dz, ldz);
            tiles = {1, 1, 1};  // the bias gradient sums rows
        } else {
            tiles = tiling(shape, aligned(z, sizeof(T)));
            launch_logits<T>(z, Slope<T>{{bias ? static_cast<const T*>(bias) + v0 : nullptr}, tokens, live, {stats, g_loss, g_lse}, v0, V, dz, ldz, part}, shape, st);
        }
        if (gx) {
            const Product p{{dz, dz}, {w, w}, ldz, ldw, M, K, n, 0, count, nullptr, 1, lay.px.splits, lay.more};
            dx_tile = aligned(p, sizeof(T)) ? 256 >> lay.px.size : 64;
            launch_product<T, false, true>(p, Store<float>{{}, {dx, dx}, K, (int64_t)M * K, v0 > 0, fours(dx, K, 4)}, lay.px.size, st);
        }
        if (gw) {
            T* out = static_cast<T*>(gw) + (int64_t)v0 * K;
            const Product p{{dz, dz}, {xp, xp}, ldz, ld, n, K, M, 0, nullptr, count, 1, lay.pw.splits, 0};
            if (lay.pw.splits > 1) {
                launch_product<T, true, true>(p, Store<float>{{}, {dw, dw}, K, (int64_t)n * K, false, fours(dw, K, 4)}, lay.pw.size, st);
                join(dw, lay.pw.splits, nullptr, {}, n, K, out, st);
            } else {
                launch_product<T, true, true>(p, Store<T>{{}, {out, out}, K, 0, false, fours(out, K, sizeof(T))}, lay.pw.size, st);
            }
        }
    }
    if (gx) join(dx, lay.px.splits, place, {count, dx_tile, lay.more}, M, K, static_cast<T*>(gx), st);
    if (gb) k_bias_fold<T><<<(V + 63) / 64, kLiveThreads, 0, st>>>(part, count, tiles, V, static_cast<T*>(gb));
}

}  // namespace

extern "C" size_t spec_cross_entropy_workspace_bytes(spec_dtype dtype, int M, int V, int K) {
    return entropy_ok(dtype, M, V, K) ? forward_layout(dtype, M, V, K).total : 0;
}

extern "C" spec_status spec_cross_entropy(const void* x, const void* weight, const void* bias, spec_dtype dtype,
                                          const int32_t* tokens, int M, int V, int K, float* out_loss, float* out_lse,
                                          int32_t* out_status, float* out_stats, void* workspace, size_t workspace_bytes,
                                          void* stream) {
    if (!type_ok(dtype)) return SPEC_EDTYPE;
    if (!entropy_ok(dtype, M, V, K) || !x || !weight || !tokens || !out_loss || !out_lse || !out_status) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_cross_entropy_workspace_bytes(dtype, M, V, K))) return SPEC_EWORKSPACE;
    char* ws = static_cast<char*>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (value_of(dtype) == SPEC_BF16)
        entropy_forward<bf16>(x, weight, bias, tokens, M, V, K, out_loss, out_lse, out_status, out_stats, dtype, ws, st);
    else
        entropy_forward<float>(x, weight, bias, tokens, M, V, K, out_loss, out_lse, out_status, out_stats, dtype, ws, st);
    return launched();
}

extern "C" size_t spec_cross_entropy_grad_workspace_bytes(spec_dtype dtype, int M, int V, int K) {
    return entropy_ok(dtype, M, V, K) ? backward_layout(dtype, M, V, K).total : 0;
}

extern "C" spec_status spec_cross_entropy_grad(const void* x, const void* weight, const void* bias, spec_dtype dtype,
                                               const int32_t* tokens, const float* stats, const float* grad_loss,
                                               const float* grad_lse, int M, int V, int K, void* grad_x, void* grad_weight,
                                               void* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
    if (!type_ok(dtype)) return SPEC_EDTYPE;
    if (!entropy_ok(dtype, M, V, K) || !x || !weight || !tokens || !stats) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_cross_entropy_grad_workspace_bytes(dtype, M, V, K))) return SPEC_EWORKSPACE;
    char* ws = static_cast<char*>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (value_of(dtype) == SPEC_BF16)
        entropy_backward<bf16>(x, weight, bias, tokens, stats, grad_loss, grad_lse, M, V, K, grad_x, grad_weight, grad_bias, dtype, ws, st);
    else
        entropy_backward<float>(x, weight, bias, tokens, stats, grad_loss, grad_lse, M, V, K, grad_x, grad_weight, grad_bias, dtype, ws, st);
    return launched();
}

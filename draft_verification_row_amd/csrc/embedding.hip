// embedding.hip -- the rows of a table that given tokens pick, scaled, and the
// table's gradient, for gfx950 (MI355X).
//
//   y[i] = s W[t_i]                     W [V][H], y [n][H]
//   dW[v] = s sum over i with t_i = v of dy[i]
// Both are bound by memory.  The gradient is made row by row of the table, with
// the positions sorted by token, so that each of its bytes is written once, no
// two workgroups add to the same one, and the order of its sums is fixed (that of i,
// with each whole piece of a long run summed by itself).  Sums are fp32 and
// rounded once.
#include "tiles.h"

namespace {

// Sixteen bytes of a row, from element k on, as floats and back; at any
// alignment, `len` the row's length.
template <typename T>
struct Chunk {
    static constexpr int kElems = 16 / (int)sizeof(T);
    float v[kElems];
    __device__ void set(u32x4 q) {
#pragma unroll
        for (int j = 0; j < kElems; ++j)
            v[j] = __uint_as_float(sizeof(T) == 4 ? q[j % 4] : (j & 1) ? q[j >> 1] & 0xffff0000u : q[j >> 1] << 16);
    }
    __device__ void store(T* row, int k, int len, bool whole, float scale) const {
        struct Any {
            u32x4 v;
        } __attribute__((packed, aligned(sizeof(T))));
        if (k + kElems <= len) {
            float o[kElems];
#pragma unroll
            for (int j = 0; j < kElems; ++j) o[j] = v[j] * scale;
            u32x4 q;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if constexpr (sizeof(T) == 2)
                    q[j] = pack_bf16(o[2 * j], o[2 * j + 1]);
                else
                    q[j] = __float_as_uint(o[j]);
            if (whole)
                __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(row + k));
            else
                reinterpret_cast<Any*>(row + k)->v = q;
        } else {
            for (int j = 0; j < kElems && k + j < len; ++j) put(row + k + j, v[j] * scale);
        }
    }
};
template <typename T>
__device__ inline u32x4 raw_chunk(const T* row, int k, int len, bool whole) {
    return whole ? *reinterpret_cast<const u32x4*>(row + k) : chunk_of(row, k, len);
}

// How a row is shared out: `lanes` threads a row, a power of two.
inline int lanes_of(int across) {
    int lanes = 8;
    while (lanes < kThreads && lanes < across) lanes *= 2;
    return lanes;
}

struct Lookup {
    const void* weight;
    const int32_t* tokens;
    int n, V, H, lanes;
    float scale;
    void* out;
    bool whole;
};
// -1: zeros; other tokens outside the table: NaN.
template <typename T>
__global__ __launch_bounds__(kThreads) void k_lookup(Lookup a) {
    constexpr int kElems = Chunk<T>::kElems;
    const int r = blockIdx.x * (kThreads / a.lanes) + threadIdx.x / a.lanes;
    if (r >= a.n) return;
    const int x = a.tokens[r];
    const bool in = x >= 0 && x < a.V;
    const T* row = static_cast<const T*>(a.weight) + (int64_t)(in ? x : 0) * a.H;
    T* out = static_cast<T*>(a.out) + (int64_t)r * a.H;
#pragma unroll 2
    for (int k = threadIdx.x % a.lanes * kElems; k < a.H; k += a.lanes * kElems) {
        Chunk<T> c;
        if (in) {
            c.set(raw_chunk(row, k, a.H, a.whole));
        } else {
#pragma unroll
            for (int j = 0; j < kElems; ++j) c.v[j] = x == -1 ? 0.f : NAN;
        }
        c.store(out, k, a.H, a.whole, in ? a.scale : 1.f);
    }
}

// ------------------------------------------------------------------- sorting
// The place of each position among all, by token and then by position: the
// number of positions that come before it.  64 positions a workgroup, a lane
// each, whose waves count over a share of the tokens each, read as scalars:
// 28 us for 16384 positions, growing with their square.
// Tokens outside the table are not below V as unsigned numbers: they come last.
constexpr int kRankWaves = 16;
__global__ __launch_bounds__(64 * kRankWaves) void k_rank(const uint32_t* __restrict__ tokens, int n, uint32_t* sorted, int* position) {
    __shared__ int sums[kRankWaves][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int first = blockIdx.x * 64, i = first + lane;
    const uint32_t mine = tokens[min(i, n - 1)];
    const int per = ((n + kRankWaves - 1) / kRankWaves + 63) / 64 * 64, begin = min(w * per, n), end = min(begin + per, n);
    int before = 0;
    // the shares are whole 64s, as the workgroup's own positions are
    const int a = min(end, max(begin, first)), b = min(end, max(a, first + 64));
#pragma unroll 16
    for (int j = begin; j < a; ++j) before += tokens[j] <= mine;
    for (int j = a; j < b; ++j) before += tokens[j] < mine || (tokens[j] == mine && j < i);
#pragma unroll 16
    for (int j = b; j < end; ++j) before += tokens[j] < mine;
    sums[w][lane] = before;
    __syncthreads();
    if (w == 0 && i < n) {
        for (int s = 1; s < kRankWaves; ++s) before += sums[s][lane];
        sorted[before] = mine;
        position[before] = i;
    }
}

// ------------------------------------------------------------------ gradient
// Runs of one token longer than kRun are summed in parts: a sorted piece of kRun
// positions that is all one token has its sum in part [piece][H].
constexpr int kRun = 32;
struct TableGrad {
    const void* dy;
    const uint32_t* sorted;
    const int* position;
    const int* start;
    int n, V, H, lanes;  // lanes: threads a row
    float* part;
    float scale;
    void* out;
    bool whole_in, whole_out;
};
template <typename T>
__global__ __launch_bounds__(kThreads) void k_runs(TableGrad a) {
    const int first = blockIdx.x * kRun;
    const uint32_t x = a.sorted[first];
    if (first + kRun > a.n || x >= (uint32_t)a.V || a.sorted[first + kRun - 1] != x) return;
    for (int k = threadIdx.x * Chunk<T>::kElems; k < a.H; k += kThreads * Chunk<T>::kElems) {
        float sum[Chunk<T>::kElems] = {};
#pragma unroll 8
        for (int i = 0; i < kRun; ++i) {
            Chunk<T> c;
            c.set(raw_chunk(static_cast<const T*>(a.dy) + (int64_t)a.position[first + i] * a.H, k, a.H, a.whole_in));
#pragma unroll
            for (int j = 0; j < c.kElems; ++j) sum[j] += c.v[j];
        }
        float* to = a.part + (int64_t)blockIdx.x * a.H + k;
        for (int j = 0; j < Chunk<T>::kElems && k + j < a.H; ++j) to[j] = sum[j];
    }
}

// start[v], v in [0, V]: the first sorted position whose token is not below v.
__global__ __launch_bounds__(kThreads) void k_starts(const uint32_t* sorted, int n, int V, int* start) {
    const int v = blockIdx.x * kThreads + threadIdx.x;
    if (v > V) return;
    int lo = 0;
    for (int hi = n; lo < hi;) {
        const int at = (lo + hi) / 2;
        if (sorted[at] < (uint32_t)v)
            lo = at + 1;
        else
            hi = at;
    }
    start[v] = lo;
}

// A workgroup writes kRowsEach rows of the table's gradient after each other, or
// that many groups of narrower rows, `lanes` threads a row.  128256 x 4096 bf16,
// 16384 tokens: 270 us (4.4 TB/s written and read), 215 with no token (4.9 TB/s;
// 4 or 16 rows each are 4 to 8% slower, stores through the caches 5%).
constexpr int kRowsEach = 8;
template <typename T>
__global__ __launch_bounds__(kThreads) void k_table_grad(TableGrad a) {
    constexpr int kElems = Chunk<T>::kElems, kAhead = 8;
    const int groups = kThreads / a.lanes, group = threadIdx.x / a.lanes, lane = threadIdx.x % a.lanes;
    const int v0 = blockIdx.x * kRowsEach * groups + group;
    int from[kRowsEach], to[kRowsEach];
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        const int v = min(v0 + i * groups, a.V - 1);
        from[i] = a.start[v];
        to[i] = a.start[v + 1];
    }
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        const int v = v0 + i * groups;
        if (v >= a.V) break;
        // whole pieces of the run have their sums already
        const int first = (from[i] + kRun - 1) / kRun * kRun, last = to[i] / kRun * kRun;
        const int stop = last > first ? first : to[i], again = last > first ? last : to[i];
        for (int k = lane * kElems; k < a.H; k += a.lanes * kElems) {
            Chunk<T> sum;
#pragma unroll
            for (int j = 0; j < kElems; ++j) sum.v[j] = 0.f;
            auto add = [&](int q0, int q1) {
                for (int q = q0; q < q1; q += kAhead) {
                    u32x4 raw[kAhead];
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        raw[u] = raw_chunk(static_cast<const T*>(a.dy) + (int64_t)a.position[min(q + u, q1 - 1)] * a.H, k, a.H, a.whole_in);
#pragma unroll
                    for (int u = 0; u < kAhead; ++u) {
                        if (q + u >= q1) break;
                        Chunk<T> c;
                        c.set(raw[u]);
#pragma unroll
                        for (int j = 0; j < kElems; ++j) sum.v[j] += c.v[j];
                    }
                }
            };
            add(from[i], stop);
            for (int q = first; q < last; q += kRun * kAhead) {
                float part[kAhead][kElems];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const float* at = a.part + (int64_t)min(q / kRun + u, last / kRun - 1) * a.H + k;
#pragma unroll
                    for (int j = 0; j < kElems; ++j) part[u][j] = k + j < a.H ? at[j] : 0.f;
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (q + u * kRun < last)
#pragma unroll
                        for (int j = 0; j < kElems; ++j) sum.v[j] += part[u][j];
            }
            add(again, to[i]);
            sum.store(static_cast<T*>(a.out) + (int64_t)v * a.H, k, a.H, a.whole_out, a.scale);
        }
    }
}

// ---------------------------------------------------------------- host side
constexpr long long kMaxTable = 1ll << 34;  // elements: launches stay below 2^32 threads
inline bool embedding_ok(const spec_dtype& d, long long n, long long V, long long H) {
    const int t = value_of(d);
    return (t == SPEC_BF16 || t == SPEC_F32) && n >= 1 && V >= 1 && H >= 1 && n <= SPEC_MAX_LINEAR && V <= SPEC_MAX_LINEAR &&
           H <= SPEC_MAX_LINEAR && n * H < kMaxTable && V * H < kMaxTable;
}
struct EmbeddingLayout {
    size_t sorted, position, start, part, total;
};
inline EmbeddingLayout embedding_layout(long long n, long long V, long long H) {
    EmbeddingLayout l;
    l.sorted = 0;
    l.position = align_up(n * 4, 256);
    l.start = 2 * l.position;
    l.part = align_up(l.start + (V + 1) * 4, 256);
    l.total = align_up(l.part + (size_t)(n / kRun * H) * 4, 256);
    return l;
}

template <typename T>
void lookup(const void* weight, const int32_t* tokens, float scale, int n, int V, int H, void* out, hipStream_t st) {
    constexpr int kElems = Chunk<T>::kElems;
    const int across = (H + kElems - 1) / kElems;
    const bool whole = H % kElems == 0 && ((uintptr_t)weight | (uintptr_t)out) % 16 == 0;
    const int lanes = lanes_of(across), rows = kThreads / lanes;
    k_lookup<T><<<(n + rows - 1) / rows, kThreads, 0, st>>>({weight, tokens, n, V, H, lanes, scale, out, whole});
}

template <typename T>
void table_grad(const int32_t* tokens, const void* dy, float scale, int n, int V, int H, void* out, char* ws, hipStream_t st) {
    constexpr int kElems = Chunk<T>::kElems;
    const EmbeddingLayout lay = embedding_layout(n, V, H);
    uint32_t* sorted = reinterpret_cast<uint32_t*>(ws + lay.sorted);
    int* position = reinterpret_cast<int*>(ws + lay.position);
    const int lanes = lanes_of((H + kElems - 1) / kElems);
    const bool whole = H % kElems == 0;
    int* start = reinterpret_cast<int*>(ws + lay.start);
    const TableGrad g{dy, sorted, position, start, n, V, H, lanes, reinterpret_cast<float*>(ws + lay.part), scale, out,
                      whole && (uintptr_t)dy % 16 == 0, whole && (uintptr_t)out % 16 == 0};
    k_rank<<<(n + 63) / 64, 64 * kRankWaves, 0, st>>>(reinterpret_cast<const uint32_t*>(tokens), n, sorted, position);
    if (n >= kRun) k_runs<T><<<n / kRun, kThreads, 0, st>>>(g);
    k_starts<<<V / kThreads + 1, kThreads, 0, st>>>(sorted, n, V, start);
    const int rows = kRowsEach * (kThreads / lanes);
    k_table_grad<T><<<(V + rows - 1) / rows, kThreads, 0, st>>>(g);
}

}  // namespace

extern "C" spec_status spec_embedding(const void* weight, spec_dtype dtype, const int32_t* tokens, float scale, int n, int V, int H,
                                      void* out, void* stream) {
    if (!type_ok(dtype)) return SPEC_EDTYPE;
    if (!embedding_ok(dtype, n, V, H) || !isfinite(scale) || !weight || !tokens || !out) return SPEC_EINVAL;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (value_of(dtype) == SPEC_BF16)
        lookup<bf16>(weight, tokens, scale, n, V, H, out, st);
    else
        lookup<float>(weight, tokens, scale, n, V, H, out, st);
    return launched();
}

extern "C" size_t spec_embedding_grad_workspace_bytes(spec_dtype dtype, int n, int V, int H) {
    return embedding_ok(dtype, n, V, H) ? embedding_layout(n, V, H).total : 0;
}

extern "C" spec_status spec_embedding_grad(const int32_t* tokens, const void* grad_out, spec_dtype dtype, float scale, int n, int V,
                                           int H, void* grad_weight, void* workspace, size_t workspace_bytes, void* stream) {
    if (!type_ok(dtype)) return SPEC_EDTYPE;
    if (!embedding_ok(dtype, n, V, H) || !isfinite(scale) || !tokens || !grad_out || !grad_weight) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_embedding_grad_workspace_bytes(dtype, n, V, H))) return SPEC_EWORKSPACE;
    char* ws = static_cast<char*>(workspace);
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (value_of(dtype) == SPEC_BF16)
        table_grad<bf16>(tokens, grad_out, scale, n, V, H, grad_weight, ws, st);
    else
        table_grad<float>(tokens, grad_out, scale, n, V, H, grad_weight, ws, st);
    return launched();
}

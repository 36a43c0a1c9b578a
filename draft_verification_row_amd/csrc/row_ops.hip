// row_ops.hip -- operators on logit rows beside the verification rules, for
// gfx950 (MI355X): the log probabilities of given tokens with entropy and top
// alternatives, the divergence KL(p || q) of a draft from its target, and the
// gradients of both.
//
// With m the maximum of a row, d_j = l_j - m, S = sum e^d_j and
// A = sum e^d_j d_j:
//   log p_x = d_x - ln S            H = ln S - A / S
//   d log p_x / d l_j = [j = x] - p_j
//   dH / d l_j        = -p_j (ln p_j + H)
// and for a target row l and a draft row d with maxima m, n and sums S, R:
//   KL = U / S + ln(R / S),  U = sum e^(l_j - m) ((l_j - m) - (d_j - n))
//   dKL / d d_j = q_j - p_j.
// Differences are taken before they are scaled to base 2, so rows of the
// type's lowest value stay finite, and a row's constant offset cancels
// exactly in U.
#include <hip/hip_runtime.h>

#include <limits.h>
#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include "spec_verify.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnroll = 4;                       // 16-byte loads per thread and tile
constexpr int kTileVecs = kThreads * kUnroll;    // 16 KiB
constexpr int kMaxParts = 32;                     // workgroups per row, at most one a lane
constexpr float kLog2e = 1.44269504088896340736f;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
constexpr int kRsrcWord3 = 0x00020000;  // gfx9-family raw buffer, 32-bit data format

// --------------------------------------------------------------- row access
// A row is read in whole 16-byte blocks whatever its alignment: block i holds
// the elements i * kVec - shift + j.  The first and the last block may reach
// past the row, by less than 16 bytes and inside the same aligned block as
// bytes of the row, and those elements are set to -inf; blocks past the end
// are not accessed (the descriptor's size ends there).
__device__ inline float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ inline float widen(float v) { return v; }

template <typename T>
struct Row {
    static constexpr int kVec = 16 / (int)sizeof(T);
    __amdgpu_buffer_rsrc_t rsrc;
    int shift, nvec;  // blocks up to the row's end, or to `end`
    int stop;         // elements up to there
    __device__ Row(const T* row, int V, int end = INT_MAX) {
        const uintptr_t a = (uintptr_t)row, a0 = a & ~(uintptr_t)15;
        shift = (int)(a - a0) / (int)sizeof(T);
        nvec = min((shift + V + kVec - 1) / kVec, end);
        stop = min(V, nvec * kVec - shift);
        rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(a0), (short)0, nvec * 16, kRsrcWord3);
    }
    __device__ int first(int i) const { return i * kVec - shift; }  // element of block i's place 0
    // ONCE: a non-temporal load, for rows that the caches cannot keep
    template <bool ONCE>
    __device__ u32x4 raw(int i) const { return __builtin_amdgcn_raw_buffer_load_b128(rsrc, i * 16, 0, ONCE ? 2 : 0); }
    // the elements e .. e + kVec - 1, widened; -inf outside the row
    __device__ void unpack(u32x4 q, int e, float (&v)[kVec]) const {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(q[j] << 16);
                v[2 * j + 1] = __uint_as_float(q[j] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(q[j]);
        }
        if (e < 0 || e + kVec > stop) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (e + j < 0 || e + j >= stop) v[j] = -INFINITY;
        }
    }
};

// Blocks of one row cut where another row's blocks start: from(i) holds this
// row's elements that lie under the other row's block i.  Where the two rows
// are aligned alike that is one load, else two neighbouring ones (the second
// a cache hit) and a shift by the same count in every lane.
template <typename T>
struct Beside {
    static constexpr int kVec = Row<T>::kVec;
    Row<T> r;
    int block, dwords, bytes;  // block offset, then the shift
    __device__ Beside(const T* row, int V, const Row<T>& other) : r(row, V) {
        const int d = r.shift - other.shift;
        block = d < 0 ? -1 : 0;
        const int by = (d < 0 ? d + kVec : d) * (int)sizeof(T);
        dwords = by >> 2;
        bytes = by & 3;
    }
    __device__ bool aligned() const { return (dwords | bytes) == 0; }
    template <bool ONCE, bool ALIGNED>
    __device__ u32x4 from(int i) const {
        // block -1 lies past the descriptor's size like any other outside block
        const u32x4 a = r.template raw<ONCE && ALIGNED>(i + block);
        if constexpr (ALIGNED) return a;
        const u32x4 b = r.template raw<false>(i + block + 1);
        u32x4 q;
        uint32_t x[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) {
            uint32_t w = j < 4 ? a[j & 3] : b[0];
            if (dwords == 1) w = j + 1 < 4 ? a[(j + 1) & 3] : b[(j + 1) & 3];
            if (dwords == 2) w = j + 2 < 4 ? a[(j + 2) & 3] : b[(j + 2) & 3];
            if (dwords == 3) w = j + 3 < 4 ? a[(j + 3) & 3] : b[(j + 3) & 3];
            x[j] = w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __builtin_amdgcn_alignbyte(x[j + 1], x[j], bytes);
        return q;
    }
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ inline uint32_t pack_bf16(float lo, float hi) {  // round to nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}
__device__ inline float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }  // 0 below 2^-126

// A row's gradient, written block by block like Row reads: whole blocks at
// once where the output row is aligned like the input row; ONCE: past the
// caches too.
template <bool ONCE, typename T>
__device__ inline void store_block(T* row, const Row<T>& r, int i, bool whole, const float (&v)[Row<T>::kVec]) {
    constexpr int kVec = Row<T>::kVec;
    const int e = r.first(i);
    u32x4 q;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = __float_as_uint(v[j]);
    }
    if (whole && e >= 0 && e + kVec <= r.stop) {
        if constexpr (ONCE)
            __builtin_nontemporal_store(q, reinterpret_cast<u32x4*>(row + e));
        else
            *reinterpret_cast<u32x4*>(row + e) = q;
        return;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (e + j >= 0 && e + j < r.stop) {
            if constexpr (sizeof(T) == 2)
                row[e + j] = (uint16_t)(q[j >> 1] >> (16 * (j & 1)));
            else
                row[e + j] = v[j];
        }
}

// --------------------------------------------------------- running statistics
// The reference a row's differences are taken from: its maximum so far, or 0
// while nothing finite was seen (then every difference is -inf, every term 0).
__device__ inline float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

struct Soft {  // of a set of logits: max, sum e^(l-m), sum e^(l-m) (l-m)
    float m, s, a;
};

// x seen from the larger maximum m of a union (selects, no branches: these
// sit in the joins' dependent chains)
__device__ inline Soft rebase(const Soft& x, float m) {
    const float d = x.m - ref_of(m), f = exp2_(d * kLog2e);
    const float a = f * fmaf(x.s, d, x.a);
    return {m, x.s * f, f > 0.f ? a : 0.f};  // a NaN is in s too
}
__device__ inline Soft join(const Soft& x, const Soft& y) {
    const float m = fmaxf(x.m, y.m);
    const Soft p = rebase(x, m), q = rebase(y, m);
    return {m, p.s + q.s, p.a + q.a};
}

struct Pair {  // of two rows' logits: maxima, sums, U of the comment above, and
    float m, s, n, r, u, w;  // the largest target logit under a draft's -inf
};
__device__ inline Pair rebase(const Pair& x, float m, float n) {
    const float d = x.m - ref_of(m), f = exp2_(d * kLog2e);
    const float c = x.n - ref_of(n), g = exp2_(c * kLog2e);
    const float u = f * fmaf(x.s, d - c, x.u);
    return {m, x.s * f, n, x.r * g, f > 0.f && x.s != 0.f ? u : 0.f, x.w};
}
__device__ inline Pair join(const Pair& x, const Pair& y) {
    const float m = fmaxf(x.m, y.m), n = fmaxf(x.n, y.n);
    const Pair p = rebase(x, m, n), q = rebase(y, m, n);
    return {m, p.s + q.s, n, p.r + q.r, p.u + q.u, fmaxf(p.w, q.w)};
}

__device__ inline Soft shfl_xor(const Soft& x, int k) {
    return {__shfl_xor(x.m, k), __shfl_xor(x.s, k), __shfl_xor(x.a, k)};
}
__device__ inline Pair shfl_xor(const Pair& x, int k) {
    return {__shfl_xor(x.m, k), __shfl_xor(x.s, k), __shfl_xor(x.n, k), __shfl_xor(x.r, k), __shfl_xor(x.u, k),
            __shfl_xor(x.w, k)};
}
// Joined over the workgroup, in a fixed order; every thread gets the result.
template <typename S>
__device__ inline S join_group(S x) {
    __shared__ S part[kWaves];
#pragma unroll
    for (int k = 1; k < 64; k <<= 1) x = join(x, shfl_xor(x, k));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) x = join(x, part[w]);
    __syncthreads();
    return x;
}

// ------------------------------------------------------ token log probabilities
struct LpArgs {
    const void* logits;
    const int32_t* tokens;
    int rows, V, top_n;
    float *logprob, *entropy;
    int32_t* top_tokens;
    float* top_logprob;
    int32_t* status;
    float* stats;  // [rows][4]: max, ln of the sum, entropy, 1 / sum or 0 where the row does not count
    int parts, chunk;  // workgroups per row, and blocks each reads
    uint32_t* counters;
    uint64_t* records;
};

__device__ inline uint32_t ordered(float v) {  // whole numbers in the floats' order
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ inline float unordered(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
// Order of alternatives: by value, then by lowest index; -0 equals +0.
__device__ inline uint64_t key_of(float v, int e) { return ((uint64_t)ordered(v + 0.f) << 32) | (uint32_t)~e; }
constexpr uint64_t kKeyNone = 0x007fffffffffffffull;  // the largest key of a -inf
__device__ inline float key_value(uint64_t k) { return unordered((uint32_t)(k >> 32)); }
__device__ inline int key_index(uint64_t k) { return (int)~(uint32_t)k; }

constexpr uint32_t kOrderLowest = 0x00800000u;  // of the lowest finite float

// Two values, as their orders, that at least n and at least k (k <= n <= 64)
// of the wave's values reach: the n-th and the k-th largest cut to their
// upper 16 bits (exact for bf16), by bisection with one compare of all lanes
// a bit.  At least the lowest finite value.
struct Bounds {
    uint32_t nth, kth;
};
__device__ inline Bounds bounds_of_wave(float v, int n, int k) {
    const uint32_t o = ordered(v);
    uint32_t x = 0, y = 0;
#pragma unroll
    for (int bit = 31; bit >= 16; --bit) {
        const uint32_t c = x | (1u << bit), d = y | (1u << bit);
        x = __popcll(__ballot(o >= c)) >= n ? c : x;
        y = __popcll(__ballot(o >= d)) >= k ? d : y;
    }
    return {max(x, kOrderLowest), max(y, kOrderLowest)};
}

// Best tokens of what a workgroup has read: keys in key[0 .. count), in
// falling order.
constexpr int kCand = 1024, kFound = 256;
static_assert(kCand >= SPEC_MAX_TOP * SPEC_MAX_TOP, "the fold's candidates fit");
struct Best {
    uint64_t key[kCand];
    uint64_t sorted[SPEC_MAX_TOP];
    uint64_t found[kWaves][kFound];  // of one tile, by wave
    uint64_t red[kWaves];
    Bounds bound[kWaves];
    int count;
};

// Keeps the n best of the first c keys, sorted; returns their number.  Keys
// differ, so a key's place is the number of keys above it; four neighbouring
// threads count for one key.
__device__ inline int keep_best(Best& b, int c, int n) {
    const int t = threadIdx.x, sub = t & 3;
    for (int i0 = 0; i0 < c; i0 += kThreads / 4) {
        const int i = i0 + (t >> 2);
        const uint64_t k = i < c ? b.key[i] : ~0ull;
        int above = 0;
        for (int j = sub; j < c; j += 16) {
            uint64_t o[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) o[s] = b.key[min(j + 4 * s, c - 1)];
#pragma unroll
            for (int s = 0; s < 4; ++s) above += j + 4 * s < c && o[s] > k;
        }
        above += __builtin_amdgcn_mov_dpp(above, 0xB1, 0xf, 0xf, true);  // lane ^ 1
        above += __builtin_amdgcn_mov_dpp(above, 0x4E, 0xf, 0xf, true);  // lane ^ 2
        if (sub == 0 && i < c && above < n) b.sorted[above] = k;
    }
    __syncthreads();
    const int m = min(c, n);
    if (t < m) b.key[t] = b.sorted[t];
    __syncthreads();
    return m;
}

// The same by n rounds of a workgroup-wide maximum over the registers' keys
// and the first c of the list: for tiles of equal logits, which give more
// candidates than the list holds.
template <typename T, int U>
__device__ int keep_best_by_rounds(Best& b, int c, int n, const float (&v)[U][Row<T>::kVec], const int (&e)[U]) {
    const int t = threadIdx.x;
    const uint64_t mine = t < c ? b.key[t] : 0;
    uint64_t last = ~0ull;
    int got = 0;
    for (; got < n; ++got) {
        uint64_t k = mine < last ? mine : 0;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < Row<T>::kVec; ++j) {
                const uint64_t o = key_of(v[u][j], e[u] + j);
                if (o < last && o > k) k = o;
            }
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)k, s);
            k = o > k ? o : k;
        }
        if ((t & 63) == 0) b.red[t >> 6] = k;
        __syncthreads();
        k = b.red[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) k = b.red[w] > k ? b.red[w] : k;
        if (t == 0) b.sorted[got] = k;
        __syncthreads();
        if (k <= kKeyNone) break;
        last = k;
    }
    if (t < got) b.key[t] = b.sorted[t];
    __syncthreads();
    return got;
}

// Outputs of one row from its statistics and its sorted best keys.
template <typename T>
__device__ inline void lp_finish(const LpArgs& a, int r, int x, const T* row, const Soft& st, const uint64_t* best, int count) {
    const int t = threadIdx.x;
    const bool some = st.s != 0.f;  // false: a row of -inf alone
    const float ref = ref_of(st.m), ls = logf(st.s), H = some ? ls - st.a / st.s : 0.f;
    if (t == 0) {
        a.logprob[r] = some ? (widen(row[x]) - ref) - ls : -INFINITY;
        a.entropy[r] = H;
        a.status[r] = 0;
        if (a.stats) *reinterpret_cast<float4*>(a.stats + (size_t)r * 4) = make_float4(ref, ls, H, some ? 1.f / st.s : 0.f);
    }
    if (t < a.top_n) {
        const bool is = t < count && best[t] > kKeyNone;
        a.top_tokens[(size_t)r * a.top_n + t] = is ? key_index(best[t]) : -1;
        a.top_logprob[(size_t)r * a.top_n + t] = is ? (key_value(best[t]) - ref) - ls : -INFINITY;
    }
}

__device__ inline void publish(uint64_t* p, uint64_t v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint64_t published(const uint64_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint64_t two(float a, float b) { return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a); }
__device__ inline float low(uint64_t w) { return __uint_as_float((uint32_t)w); }
__device__ inline float high(uint64_t w) { return __uint_as_float((uint32_t)(w >> 32)); }

// Whether this workgroup is the last of the row's `parts` to come here: what
// the others published before is then visible, since published words are
// written and read with agent-scope atomics, past the XCDs' caches, and have
// arrived before the counter is raised (a release fence would write back and
// invalidate the whole XCD's cache: 47 us beside 27 for the divergence of 160
// rows of 128256, timed together).  The last one leaves the counter at zero.
__device__ inline bool last_to_come(uint32_t* counter, int parts) {
    __shared__ int last;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t n = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        last = n + 1 == (uint32_t)parts;
        if (last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    asm volatile("" ::: "memory");
    return last;
}

// A row is read by `parts` workgroups of `chunk` blocks each; the last of them
// to finish folds what all have published.  Each keeps running statistics per
// thread, joined at the end, and (TOP) its best tokens: a bound that at least
// top_n of a tile's elements reach, from the threads' maxima, leaves some tens
// of candidates, which are ranked by counting; later tiles only look for
// logits above the last one kept (their indices are higher, so a tie loses).
// U: blocks per thread and tile.  The next tile is loaded while one is worked
// on.
// Bound by reading where there are many rows: 2048 rows of 151936 bf16 take
// 111 us (median; 5.6 TB/s), and 183 us with 20 alternatives, whose scan for
// candidates costs about as many instructions as the statistics.  144 rows of
// 128256 take 15 us (2.5 TB/s), 25 us with 20; with 48 padded rows among them,
// which take their share of the split, 31 us; six rows 7.8 us, and 11.3 us
// with 5: there it is the launch, the join and the fold, one after the other.
template <typename T, bool TOP, int U, bool ONCE>
__global__ __launch_bounds__(kThreads) void k_logprobs(LpArgs a) {
    constexpr int kVec = Row<T>::kVec;
    const int r = blockIdx.x / a.parts, part = blockIdx.x % a.parts, t = threadIdx.x, w = t >> 6;
    const T* row = static_cast<const T*>(a.logits) + (size_t)r * a.V;
    const int x = a.tokens[r];
    if (x < 0 || x >= a.V) {  // padded, or not a token
        if (part != 0) return;
        for (int i = t; i < a.top_n; i += kThreads) {
            a.top_tokens[(size_t)r * a.top_n + i] = -1;
            a.top_logprob[(size_t)r * a.top_n + i] = 0.f;
        }
        if (t == 0) {
            a.logprob[r] = 0.f;
            a.entropy[r] = 0.f;
            a.status[r] = x != -1;
            if (a.stats) *reinterpret_cast<float4*>(a.stats + (size_t)r * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }
    __shared__ Best best;
    const int begin = part * a.chunk;
    const Row<T> R(row, a.V, begin + a.chunk);
    Soft st{-INFINITY, 0.f, 0.f};
    int count = 0;
    u32x4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) q[u] = R.template raw<ONCE>(begin + u * kThreads + t);
    for (int base = begin; base < R.nvec; base += U * kThreads) {
        float v[U][kVec], m = -INFINITY;
        int e[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            e[u] = R.first(base + u * kThreads + t);
            R.unpack(q[u], e[u], v[u]);
            q[u] = R.template raw<ONCE>(base + (U + u) * kThreads + t);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < kVec; ++j) m = fmaxf(m, v[u][j]);
        st = rebase(st, fmaxf(st.m, m));
        const float ref = ref_of(st.m);
        // a tile's own sums first: a row's sum is then no long chain of small
        // terms added to a large one
        float s = 0.f, sd = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float d = v[u][j] - ref, f = exp2_(d * kLog2e);
                s += f;
                sd = fmaf(f, fmaxf(d, -3.0e38f), sd);
            }
        st.s += s;
        st.a += sd;
        if constexpr (TOP) {
            uint32_t order;
            if (count < a.top_n) {
                // each wave has top_n values from its nth on, and the waves
                // together from the lowest of their kth on
                const Bounds o = bounds_of_wave(m, a.top_n, (a.top_n + kWaves - 1) / kWaves);
                if ((t & 63) == 0) best.bound[w] = o;
                if (t == 0) best.count = count;
                __syncthreads();
                uint32_t nth = 0, kth = ~0u;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) {
                    nth = max(nth, best.bound[i].nth);
                    kth = min(kth, best.bound[i].kth);
                }
                order = max(nth, kth);
            } else {
                order = ordered(key_value(best.key[a.top_n - 1])) + 1;
                if (t == 0) best.count = count;
                __syncthreads();
            }
            const float bound = unordered(order);
            if (__ballot(m >= bound)) {
                int n = 0;
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < kVec; ++j) {
                        const bool hit = v[u][j] >= bound;
                        const uint64_t hits = __ballot(hit);
                        if (hits) {
                            const int i = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(hits >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)hits, 0));
                            if (hit && i < kFound) best.found[w][i] = key_of(v[u][j], e[u] + j);
                            n += __popcll(hits);
                        }
                    }
                int at = 0;
                if ((t & 63) == 0) at = atomicAdd(&best.count, n <= kFound ? n : kCand + 1);
                at = __builtin_amdgcn_readfirstlane(at);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                for (int i = t & 63; i < n && n <= kFound && at + n <= kCand; i += 64) best.key[at + i] = best.found[w][i];
            }
            __syncthreads();
            const int c = best.count;
            if (c > kCand)
                count = keep_best_by_rounds<T, U>(best, count, a.top_n, v, e);
            else if (c > count)
                count = keep_best(best, c, a.top_n);
            else
                __syncthreads();  // best.count is read before it is set again
        }
    }
    st = join_group(st);
    if (a.parts > 1) {
        const int words = 2 + (TOP ? a.top_n : 0);
        uint64_t* rec = a.records + ((size_t)r * a.parts + part) * words;
        if (t == 0) {
            publish(rec, two(st.m, st.s));
            publish(rec + 1, two(st.a, 0.f));
        }
        if constexpr (TOP)
            if (t < a.top_n) publish(rec + 2 + t, t < count ? best.key[t] : 0);
        if (!last_to_come(a.counters + r, a.parts)) return;
        rec = a.records + (size_t)r * a.parts * words;
        st = {-INFINITY, 0.f, 0.f};
        if constexpr (TOP) {
            // Every part's list is sorted: the n-th largest of the parts' best
            // (or the largest of their n-th) bounds what can count, and leaves
            // at most n lists, or fewer parts than n.
            constexpr int kKeys = kMaxParts * SPEC_MAX_TOP / kThreads;
            const int n = a.top_n, total = a.parts * n;
            uint64_t k[kKeys], head = 0, tail = 0;
#pragma unroll
            for (int u = 0; u < kKeys; ++u) {
                const int i = u * kThreads + t;
                k[u] = i < total ? published(rec + (size_t)(i / n) * words + 2 + i % n) : 0;
            }
            if (t < a.parts) {
                const uint64_t w0 = published(rec + (size_t)t * words), w1 = published(rec + (size_t)t * words + 1);
                head = published(rec + (size_t)t * words + 2);
                tail = published(rec + (size_t)t * words + 1 + n);
                st = {low(w0), high(w0), low(w1)};
            }
            if (t < 64) {
                best.key[t] = head;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                int above = 0;
#pragma unroll 8
                for (int j = 0; j < kMaxParts; ++j) above += best.key[j] > head;
                uint64_t bound = above == n - 1 ? head : 0;
                bound = tail > bound ? tail : bound;
#pragma unroll
                for (int s = 1; s < 64; s <<= 1) {
                    const uint64_t o = __shfl_xor((unsigned long long)bound, s);
                    bound = o > bound ? o : bound;
                }
                if (t == 0) {
                    best.red[0] = bound;
                    best.count = 0;
                }
            }
            __syncthreads();
            const uint64_t bound = best.red[0];
#pragma unroll
            for (int u = 0; u < kKeys; ++u)
                if (k[u] != 0 && k[u] >= bound) best.key[atomicAdd(&best.count, 1)] = k[u];
            __syncthreads();
            count = keep_best(best, best.count, n);
        } else if (t < a.parts) {
            const uint64_t w0 = published(rec + (size_t)t * words), w1 = published(rec + (size_t)t * words + 1);
            st = {low(w0), high(w0), low(w1)};
        }
        st = join_group(st);
        for (int i = t; i < a.parts * words; i += kThreads) rec[i] = 0;
    }
    lp_finish(a, r, x, row, st, best.key, count);
}

struct LpGradArgs {
    const void* logits;
    const int32_t* tokens;
    const float *stats, *g_logprob, *g_entropy;
    int rows, V, tiles;
    void* grad;
};

// One workgroup per tile of a row: reads its logits and writes their gradient,
// bound by both.
template <typename T, bool ONCE>
__global__ __launch_bounds__(kThreads) void k_logprobs_grad(LpGradArgs a) {
    constexpr int kVec = Row<T>::kVec;
    const int r = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles, t = threadIdx.x;
    const size_t at = (size_t)r * a.V;
    const T* row = static_cast<const T*>(a.logits) + at;
    T* out = static_cast<T*>(a.grad) + at;
    const Row<T> R(row, a.V);
    const bool whole = (((uintptr_t)row ^ (uintptr_t)out) & 15) == 0;
    const int x = a.tokens[r];
    const float* s = a.stats + (size_t)r * 4;
    const bool live = x >= 0 && x < a.V && s[3] != 0.f;
    const float ref = s[0], ls = s[1], H = s[2], inv = s[3];
    const float gl = a.g_logprob ? a.g_logprob[r] : 0.f, ge = a.g_entropy ? a.g_entropy[r] : 0.f;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int i = tile * kTileVecs + u * kThreads + t;
        if (i >= R.nvec) break;
        float v[kVec];
        if (live) {
            R.unpack(R.template raw<ONCE>(i), R.first(i), v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                // p from the difference itself: ln S would bring its own
                // rounding and the difference's with it into the exponent
                const float d = v[j] - ref, p = exp2_(d * kLog2e) * inv;
                // p first: it bounds what ln p + H and any weight can grow to
                float g = p == 0.f ? 0.f : -fmaf(ge, p * ((d - ls) + H), gl * p);
                if (R.first(i) + j == x) g += gl;
                v[j] = g;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = 0.f;
        }
        store_block<ONCE>(out, R, i, whole, v);
    }
}

// ------------------------------------------------------------ draft divergence
struct KlArgs {
    const void *target, *draft;
    const uint8_t* mask;  // [B][K], or null: every row counts
    int K, Kt, V, tiles;  // target rows per request: Kt >= K
    float* kl;
    float* stats;  // [B*K][4]: max and 1 / sum or 0 for an empty row, target then draft
    const float* g_kl;
    void* grad;
    int parts, chunk;  // as in LpArgs
    uint32_t* counters;
    uint64_t* records;
};

// Split over workgroups like k_logprobs.  Blocks follow the target's row.
// Bound by reading both rows and, close behind, by two exponentials a token:
// 187 us for 2048 rows of 128255 bf16 (median; 5.6 TB/s), 216 us with a tenth
// of them masked in between; 19.5 us for 128 rows of 128256, 24 us with 32
// masked ones among them, which take their share of the split.
template <typename T, bool ONCE, bool ALIGNED>
__device__ inline void kl_sweep(const Row<T>& P, const Beside<T>& Q, int begin, Pair& st) {
    constexpr int kVec = Row<T>::kVec;
    constexpr int kSteps = kUnroll / 2;  // two rows: as many loads in flight
    u32x4 x[kSteps], y[kSteps];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
        x[u] = P.template raw<ONCE>(begin + u * kThreads + (int)threadIdx.x);
        y[u] = Q.template from<ONCE, ALIGNED>(begin + u * kThreads + (int)threadIdx.x);
    }
    for (int base = begin; base < P.nvec; base += kSteps * kThreads) {
        float p[kSteps][kVec], q[kSteps][kVec], m = -INFINITY, n = -INFINITY, least = INFINITY;
#pragma unroll
        for (int u = 0; u < kSteps; ++u) {
            const int i = base + u * kThreads + (int)threadIdx.x, e = P.first(i);
            P.unpack(x[u], e, p[u]);
            P.unpack(y[u], e, q[u]);
            x[u] = P.template raw<ONCE>(i + kSteps * kThreads);
            y[u] = Q.template from<ONCE, ALIGNED>(i + kSteps * kThreads);
        }
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                m = fmaxf(m, p[u][j]);
                n = fmaxf(n, q[u][j]);
                least = fminf(least, q[u][j]);
            }
        if (least == -INFINITY) {
#pragma unroll
            for (int u = 0; u < kSteps; ++u)
#pragma unroll
                for (int j = 0; j < kVec; ++j) st.w = fmaxf(st.w, q[u][j] == -INFINITY ? p[u][j] : -INFINITY);
        }
        st = rebase(st, fmaxf(st.m, m), fmaxf(st.n, n));
        const float mr = ref_of(st.m), nr = ref_of(st.n);
        float s = 0.f, r = 0.f, gap = 0.f;  // a tile's own sums first
#pragma unroll
        for (int u = 0; u < kSteps; ++u)
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float d = p[u][j] - mr, c = q[u][j] - nr;
                const float f = exp2_(d * kLog2e), g = exp2_(c * kLog2e);
                s += f;
                r += g;
                gap += f > 0.f ? f * (d - c) : 0.f;
            }
        st.s += s;
        st.r += r;
        st.u += gap;
    }
}

constexpr float kLeastLog = -745.f;  // e^-745 is the smallest positive double

template <typename T, bool ONCE>
__global__ __launch_bounds__(kThreads) void k_draft_kl(KlArgs a) {
    const int r = blockIdx.x / a.parts, part = blockIdx.x % a.parts, t = threadIdx.x;
    if (a.mask && !a.mask[r]) {
        if (t == 0 && part == 0) {
            a.kl[r] = 0.f;
            if (a.stats) *reinterpret_cast<float4*>(a.stats + (size_t)r * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }
    const int b = r / a.K, k = r % a.K, begin = part * a.chunk;
    const Row<T> P(static_cast<const T*>(a.target) + ((size_t)b * a.Kt + k) * a.V, a.V, begin + a.chunk);
    const Beside<T> Q(static_cast<const T*>(a.draft) + (size_t)r * a.V, a.V, P);
    Pair st{-INFINITY, 0.f, -INFINITY, 0.f, 0.f, -INFINITY};
    if (Q.aligned())
        kl_sweep<T, ONCE, true>(P, Q, begin, st);
    else
        kl_sweep<T, ONCE, false>(P, Q, begin, st);
    st = join_group(st);
    if (a.parts > 1) {
        uint64_t* rec = a.records + ((size_t)r * a.parts + part) * 3;
        if (t == 0) {
            publish(rec, two(st.m, st.s));
            publish(rec + 1, two(st.n, st.r));
            publish(rec + 2, two(st.u, st.w));
        }
        if (!last_to_come(a.counters + r, a.parts)) return;
        rec = a.records + (size_t)r * a.parts * 3;
        st = {-INFINITY, 0.f, -INFINITY, 0.f, 0.f, -INFINITY};
        if (t < a.parts) {
            const uint64_t w0 = published(rec + t * 3), w1 = published(rec + t * 3 + 1), w2 = published(rec + t * 3 + 2);
            st = {low(w0), high(w0), low(w1), high(w1), low(w2), high(w2)};
        }
        st = join_group(st);
        for (int i = t; i < a.parts * 3; i += kThreads) rec[i] = 0;
    }
    if (t == 0) {
        // one logarithm of the quotient: two would each bring their rounding
        const float ls = logf(st.s), gap = logf(st.r / st.s);
        // an empty target row says nothing; an empty draft row is infinitely
        // far, and so is a token that the draft excludes and the target does
        // not: p is positive as a double, also where e^(l - m) is 0 as a float
        const bool excluded = (st.w - st.m) - ls > kLeastLog;
        a.kl[r] = st.s == 0.f ? 0.f : st.r == 0.f || excluded ? INFINITY : st.u / st.s + gap;
        if (a.stats) *reinterpret_cast<float4*>(a.stats + (size_t)r * 4) = make_float4(ref_of(st.m), st.s == 0.f ? 0.f : 1.f / st.s,
                                                                                     ref_of(st.n), st.r == 0.f ? 0.f : 1.f / st.r);
    }
}

// One workgroup per tile of a draft row: reads both rows, writes the gradient,
// bound by that: 2048 rows of 128255 bf16 take 269 us (median) for 1.58 GB (5.9
// TB/s), 262 us with a tenth of them masked.
template <typename T, bool ONCE, bool ALIGNED>
__device__ inline void kl_grad_tile(const KlArgs& a, const Row<T>& D, const Beside<T>& P, T* out, bool whole, int tile, const float4& s, float g) {
    constexpr int kVec = Row<T>::kVec;
    u32x4 x[kUnroll], y[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int i = tile * kTileVecs + u * kThreads + (int)threadIdx.x;
        x[u] = D.template raw<ONCE>(i);
        y[u] = P.template from<ONCE, ALIGNED>(i);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int i = tile * kTileVecs + u * kThreads + (int)threadIdx.x;
        if (i >= D.nvec) break;
        float q[kVec], p[kVec];
        D.unpack(x[u], D.first(i), q);
        D.unpack(y[u], D.first(i), p);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            q[j] = g * (exp2_((q[j] - s.z) * kLog2e) * s.w - exp2_((p[j] - s.x) * kLog2e) * s.y);
        store_block<ONCE>(out, D, i, whole, q);
    }
}

template <typename T, bool ONCE>
__global__ __launch_bounds__(kThreads) void k_draft_kl_grad(KlArgs a) {
    constexpr int kVec = Row<T>::kVec;
    const int r = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles, t = threadIdx.x;
    const int b = r / a.K, k = r % a.K;
    const T* drow = static_cast<const T*>(a.draft) + (size_t)r * a.V;
    T* out = static_cast<T*>(a.grad) + (size_t)r * a.V;
    const Row<T> D(drow, a.V);
    const bool whole = (((uintptr_t)drow ^ (uintptr_t)out) & 15) == 0;
    const float4 s = *reinterpret_cast<const float4*>(a.stats + (size_t)r * 4);
    if ((a.mask && !a.mask[r]) || s.y == 0.f || s.w == 0.f) {  // nothing to learn from
        const float zero[kVec] = {};
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int i = tile * kTileVecs + u * kThreads + t;
            if (i < D.nvec) store_block<ONCE>(out, D, i, whole, zero);
        }
        return;
    }
    const Beside<T> P(static_cast<const T*>(a.target) + ((size_t)b * a.Kt + k) * a.V, a.V, D);
    const float g = a.g_kl[r];
    if (P.aligned())
        kl_grad_tile<T, ONCE, true>(a, D, P, out, whole, tile, s, g);
    else
        kl_grad_tile<T, ONCE, false>(a, D, P, out, whole, tile, s, g);
}

// ---------------------------------------------------------------- host side
// An enum's value from its bytes: a caller may have put any number there.
template <typename E>
inline int value_of(const E& e) {
    static_assert(sizeof(E) == sizeof(int), "enums of the ABI are ints");
    int v;
    memcpy(&v, &e, sizeof v);
    return v;
}
inline bool dtype_ok(const spec_dtype& d) { return value_of(d) == SPEC_F32 || value_of(d) == SPEC_BF16; }

// Tiles of a row at any alignment.
inline int tiles_of(spec_dtype d, int V) {
    const int vec = d == SPEC_BF16 ? 8 : 4;
    return ((V + vec - 1) / vec + 1 + kTileVecs - 1) / kTileVecs;
}
// One workgroup per tile, in a launch of fewer than 2^32 threads.
inline bool rows_ok(spec_dtype d, long long rows, int V) {
    return rows >= 1 && rows < (1ll << 24) && V >= 1 && V <= SPEC_MAX_V && rows * tiles_of(d, V) < (1ll << 24);
}
inline bool ws_ok(const void* p, size_t bytes, size_t need) {
    return p && (uintptr_t)p % 256 == 0 && bytes >= need;
}

// How a row is split: over as many workgroups as it takes to have kGroups in
// all, of whole 4 KiB steps, and at most kMaxParts.  Kernel us of log probs
// with kGroups 512 / 256 / 1024: 144 rows of 128256 with 20 alternatives
// 25.3 / 31.7 / 30.2, 512 rows without 28.6 / 26.7 / 32.1; six rows with 5
// alternatives in 63 / 43 / 22 parts 13.1 / 11.8 / 11.1, since the fold reads
// every part's records.
constexpr int kGroups = 512;
struct Split {
    int parts, chunk;
};
inline Split split_of(spec_dtype d, long long rows, int V) {
    const int vec = d == SPEC_BF16 ? 8 : 4;
    const int nvec = (V + 2 * vec - 2) / vec;  // at the worst alignment
    const int steps = (nvec + kThreads - 1) / kThreads;
    const long long want = (kGroups + rows - 1) / rows;
    int parts = (int)(want < steps ? want : steps);
    if (parts > kMaxParts) parts = kMaxParts;
    const int chunk = (steps + parts - 1) / parts * kThreads;
    return {(nvec + chunk - 1) / chunk, chunk};
}
// Logits beyond what the chip's caches hold are read past them, and their
// gradients written past them: nothing would be left there for the next reader
// (log probs with their gradient, 2048 rows of 151936 bf16: 349 us through the
// caches, 323 with the loads past them, 299 with the stores too; 160 rows of
// 128256 of KL are slower so, 48.5 and 46.3).
inline bool read_once(spec_dtype d, long long rows, int V) {
    return rows * V * (d == SPEC_BF16 ? 2 : 4) > (256ll << 20);
}

// A workgroup that reads one 4 KiB step takes one block a thread.  Rows that
// are read once are many, so none is split into single steps.
template <typename T, bool TOP>
void launch_logprobs(const LpArgs& a, bool once, unsigned grid, hipStream_t st) {
    if (once)
        k_logprobs<T, TOP, kUnroll, true><<<grid, kThreads, 0, st>>>(a);
    else if (a.chunk == kThreads)
        k_logprobs<T, TOP, 1, false><<<grid, kThreads, 0, st>>>(a);
    else
        k_logprobs<T, TOP, kUnroll, false><<<grid, kThreads, 0, st>>>(a);
}
template <typename T>
void launch_logprobs(const LpArgs& a, bool once, unsigned grid, hipStream_t st) {
    a.top_n ? launch_logprobs<T, true>(a, once, grid, st) : launch_logprobs<T, false>(a, once, grid, st);
}

// Counters of the rows, then `words` 8-byte words for each part of each row.
inline size_t counter_bytes(long long rows) { return ((size_t)rows * 4 + 255) / 256 * 256; }
inline size_t split_bytes(const Split& s, long long rows, int words) {
    return s.parts == 1 ? 256 : counter_bytes(rows) + ((size_t)rows * s.parts * words * 8 + 255) / 256 * 256;
}

}  // namespace

extern "C" size_t spec_logprobs_workspace_bytes(spec_dtype dtype, int rows, int V, int top_n) {
    if (!dtype_ok(dtype) || !rows_ok(dtype, rows, V) || top_n < 0 || top_n > SPEC_MAX_TOP) return 0;
    return split_bytes(split_of(dtype, rows, V), rows, 2 + top_n);
}

extern "C" spec_status spec_token_logprobs(const void* logits, spec_dtype dtype, const int32_t* tokens, int rows,
                                           int V, int top_n, float* out_logprob, float* out_entropy,
                                           int32_t* out_top_tokens, float* out_top_logprob, int32_t* out_status,
                                           float* out_stats, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype)) return SPEC_EDTYPE;
    if (!rows_ok(dtype, rows, V) || top_n < 0 || top_n > SPEC_MAX_TOP) return SPEC_EINVAL;
    if (!logits || !tokens || !out_logprob || !out_entropy || !out_status) return SPEC_EINVAL;
    if (top_n > 0 && (!out_top_tokens || !out_top_logprob)) return SPEC_EINVAL;
    if ((uintptr_t)out_stats % 16) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_logprobs_workspace_bytes(dtype, rows, V, top_n))) return SPEC_EWORKSPACE;
    const Split s = split_of(dtype, rows, V);
    char* ws = static_cast<char*>(workspace);
    const LpArgs a{logits, tokens, rows, V, top_n, out_logprob, out_entropy, out_top_tokens, out_top_logprob,
                   out_status, out_stats, s.parts, s.chunk, reinterpret_cast<uint32_t*>(ws),
                   reinterpret_cast<uint64_t*>(ws + counter_bytes(rows))};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const unsigned grid = (unsigned)rows * (unsigned)s.parts;
    if (dtype == SPEC_BF16)
        launch_logprobs<uint16_t>(a, read_once(dtype, rows, V), grid, st);
    else
        launch_logprobs<float>(a, read_once(dtype, rows, V), grid, st);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

extern "C" spec_status spec_token_logprobs_grad(const void* logits, spec_dtype dtype, const int32_t* tokens,
                                                const float* stats, const float* grad_logprob,
                                                const float* grad_entropy, int rows, int V, void* out_grad,
                                                void* stream) {
    if (!dtype_ok(dtype)) return SPEC_EDTYPE;
    if (!rows_ok(dtype, rows, V) || !logits || !tokens || !stats || !out_grad) return SPEC_EINVAL;
    if ((uintptr_t)stats % 16) return SPEC_EINVAL;
    const int tiles = tiles_of(dtype, V);
    const LpGradArgs a{logits, tokens, stats, grad_logprob, grad_entropy, rows, V, tiles, out_grad};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const unsigned grid = (unsigned)rows * (unsigned)tiles;
    const bool once = read_once(dtype, rows, V);
    if (dtype == SPEC_BF16)
        once ? k_logprobs_grad<uint16_t, true><<<grid, kThreads, 0, st>>>(a) : k_logprobs_grad<uint16_t, false><<<grid, kThreads, 0, st>>>(a);
    else
        once ? k_logprobs_grad<float, true><<<grid, kThreads, 0, st>>>(a) : k_logprobs_grad<float, false><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

namespace {
inline bool kl_ok(spec_dtype d, int B, int K, int Kt, int V) {
    return B >= 1 && K >= 1 && Kt >= K && rows_ok(d, (long long)B * K, V) && (long long)B * Kt < (1ll << 31);
}
}  // namespace

extern "C" size_t spec_draft_kl_workspace_bytes(spec_dtype dtype, int B, int K, int V) {
    return dtype_ok(dtype) && kl_ok(dtype, B, K, K, V) ? split_bytes(split_of(dtype, (long long)B * K, V), (long long)B * K, 3) : 0;
}

extern "C" spec_status spec_draft_kl(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                                     const uint8_t* mask, int B, int K, int target_rows, int V, float* out_kl,
                                     float* out_stats, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype)) return SPEC_EDTYPE;
    if (!kl_ok(dtype, B, K, target_rows, V) || !target_logits || !draft_logits || !out_kl) return SPEC_EINVAL;
    if ((uintptr_t)out_stats % 16) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_draft_kl_workspace_bytes(dtype, B, K, V))) return SPEC_EWORKSPACE;
    const Split s = split_of(dtype, (long long)B * K, V);
    char* ws = static_cast<char*>(workspace);
    const KlArgs a{target_logits, draft_logits, mask, K, target_rows, V, 0, out_kl, out_stats, nullptr, nullptr,
                   s.parts, s.chunk, reinterpret_cast<uint32_t*>(ws),
                   reinterpret_cast<uint64_t*>(ws + counter_bytes((long long)B * K))};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const unsigned grid = (unsigned)(B * K) * (unsigned)s.parts;
    const bool once = read_once(dtype, (long long)B * K, V);
    if (dtype == SPEC_BF16)
        once ? k_draft_kl<uint16_t, true><<<grid, kThreads, 0, st>>>(a) : k_draft_kl<uint16_t, false><<<grid, kThreads, 0, st>>>(a);
    else
        once ? k_draft_kl<float, true><<<grid, kThreads, 0, st>>>(a) : k_draft_kl<float, false><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

extern "C" spec_status spec_draft_kl_grad(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                                          const uint8_t* mask, const float* stats, const float* grad_kl, int B,
                                          int K, int target_rows, int V, void* out_grad, void* stream) {
    if (!dtype_ok(dtype)) return SPEC_EDTYPE;
    if (!kl_ok(dtype, B, K, target_rows, V) || !target_logits || !draft_logits || !stats || !grad_kl || !out_grad)
        return SPEC_EINVAL;
    if ((uintptr_t)stats % 16) return SPEC_EINVAL;
    const int tiles = tiles_of(dtype, V);
    const KlArgs a{target_logits, draft_logits, mask, K, target_rows, V, tiles, nullptr, const_cast<float*>(stats), grad_kl, out_grad, 1, 0, nullptr, nullptr};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const unsigned grid = (unsigned)(B * K) * (unsigned)tiles;
    const bool once = read_once(dtype, (long long)B * K, V);
    if (dtype == SPEC_BF16)
        once ? k_draft_kl_grad<uint16_t, true><<<grid, kThreads, 0, st>>>(a) : k_draft_kl_grad<uint16_t, false><<<grid, kThreads, 0, st>>>(a);
    else
        once ? k_draft_kl_grad<float, true><<<grid, kThreads, 0, st>>>(a) : k_draft_kl_grad<float, false><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

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
//   KL = U / S - ln S + ln R,  U = sum e^(l_j - m) ((l_j - m) - (d_j - n))
//   dKL / d d_j = q_j - p_j.
// Differences are taken before they are scaled to base 2, so rows of the
// type's lowest value stay finite, and a row's constant offset cancels
// exactly in U.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kUnroll = 4;                       // 16-byte loads per thread and tile
constexpr int kTileVecs = kThreads * kUnroll;    // 16 KiB
constexpr float kLog2e = 1.44269504088896340736f;

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
constexpr int kRsrcWord3 = 0x00020000;  // gfx9-family raw buffer, 32-bit data format

// --------------------------------------------------------------- row access
// A row is read in whole 16-byte blocks whatever its alignment: block i holds
// the elements i * kVec - shift + j.  The first and the last block may reach
// past the row, by less than 16 bytes and inside the same aligned block as
// bytes of the row, and those elements are set to -inf; blocks past the last
// are not accessed (the descriptor's size ends there).
template <typename T>
struct Row {
    static constexpr int kVec = 16 / (int)sizeof(T);
    __amdgpu_buffer_rsrc_t rsrc;
    int shift, nvec, V;
    __device__ Row(const T* row, int V_) : V(V_) {
        const uintptr_t a = (uintptr_t)row, a0 = a & ~(uintptr_t)15;
        shift = (int)(a - a0) / (int)sizeof(T);
        nvec = (shift + V + kVec - 1) / kVec;
        rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(a0), (short)0, nvec * 16, kRsrcWord3);
    }
    __device__ int first(int i) const { return i * kVec - shift; }  // element of block i's place 0
    __device__ u32x4 raw(int i) const { return __builtin_amdgcn_raw_buffer_load_b128(rsrc, i * 16, 0, 0); }
    __device__ void load(int i, float (&v)[kVec]) const {
        unpack(raw(i), i, v);
    }
    __device__ void unpack(u32x4 q, int i, float (&v)[kVec]) const {
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
        const int e = first(i);
        if (e < 0 || e + kVec > V) {
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                if (e + j < 0 || e + j >= V) v[j] = -INFINITY;
        }
    }
    __device__ static float at(const T* row, int e) {
        if constexpr (sizeof(T) == 2)
            return __uint_as_float((uint32_t)row[e] << 16);
        else
            return row[e];
    }
};

__device__ inline uint16_t to_bf16(float f) {  // round to nearest even
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40);
    return (uint16_t)((u + 0x7fffu + ((u >> 16) & 1)) >> 16);
}

// A row's gradient, written block by block like Row reads: whole blocks at
// once where the output row is aligned like the input row.
template <typename T>
__device__ inline void store_block(T* row, const Row<T>& r, int i, bool whole, const float (&v)[Row<T>::kVec]) {
    constexpr int kVec = Row<T>::kVec;
    const int e = r.first(i);
    if (whole && e >= 0 && e + kVec <= r.V) {
        u32x4 q;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                q[j] = (uint32_t)to_bf16(v[2 * j]) | ((uint32_t)to_bf16(v[2 * j + 1]) << 16);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) q[j] = __float_as_uint(v[j]);
        }
        *reinterpret_cast<u32x4*>(row + e) = q;
        return;
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j)
        if (e + j >= 0 && e + j < r.V) {
            if constexpr (sizeof(T) == 2)
                row[e + j] = to_bf16(v[j]);
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

// x seen from the larger maximum m of a union
__device__ inline Soft rebase(const Soft& x, float m) {
    const float d = x.m - ref_of(m), f = exp2f(d * kLog2e);
    return {m, x.s * f, f > 0.f ? f * fmaf(x.s, d, x.a) : (x.a != x.a ? x.a : 0.f)};
}
__device__ inline Soft join(const Soft& x, const Soft& y) {
    const float m = fmaxf(x.m, y.m);
    const Soft p = rebase(x, m), q = rebase(y, m);
    return {m, p.s + q.s, p.a + q.a};
}

struct Pair {  // of two rows' logits: maxima, sums, and U of the comment above
    float m, s, n, r, u;
};
__device__ inline Pair rebase(const Pair& x, float m, float n) {
    const float d = x.m - ref_of(m), f = exp2f(d * kLog2e);
    const float c = x.n - ref_of(n), g = exp2f(c * kLog2e);
    return {m, x.s * f, n, x.r * g, f > 0.f && x.s != 0.f ? f * fmaf(x.s, d - c, x.u) : 0.f};
}
__device__ inline Pair join(const Pair& x, const Pair& y) {
    const float m = fmaxf(x.m, y.m), n = fmaxf(x.n, y.n);
    const Pair p = rebase(x, m, n), q = rebase(y, m, n);
    return {m, p.s + q.s, n, p.r + q.r, p.u + q.u};
}

__device__ inline Soft shfl_xor(const Soft& x, int k) {
    return {__shfl_xor(x.m, k), __shfl_xor(x.s, k), __shfl_xor(x.a, k)};
}
__device__ inline Pair shfl_xor(const Pair& x, int k) {
    return {__shfl_xor(x.m, k), __shfl_xor(x.s, k), __shfl_xor(x.n, k), __shfl_xor(x.r, k), __shfl_xor(x.u, k)};
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
    float* stats;  // [rows][4]: max, ln of the sum, entropy, 1 where the row counts
};

// Order of alternatives: by value, then by lowest index; -0 equals +0.
__device__ inline uint64_t key_of(float v, int e) {
    const uint32_t u = __float_as_uint(v + 0.f);
    const uint32_t o = (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)~e;
}
constexpr uint64_t kKeyNone = 0x007fffffffffffffull;  // the largest key of a -inf
__device__ inline float key_value(uint64_t k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ inline int key_index(uint64_t k) { return (int)~(uint32_t)k; }

template <typename T>
__global__ __launch_bounds__(kThreads) void k_logprobs(LpArgs a) {
    constexpr int kVec = Row<T>::kVec;
    const int r = blockIdx.x, t = threadIdx.x;
    const T* row = static_cast<const T*>(a.logits) + (size_t)r * a.V;
    const int x = a.tokens[r];
    if (x < 0 || x >= a.V) {  // padded, or not a token
        for (int i = t; i < a.top_n; i += kThreads) {
            a.top_tokens[(size_t)r * a.top_n + i] = -1;
            a.top_logprob[(size_t)r * a.top_n + i] = 0.f;
        }
        if (t == 0) {
            a.logprob[r] = 0.f;
            a.entropy[r] = 0.f;
            a.status[r] = x != -1;
            if (a.stats) {
                float* s = a.stats + (size_t)r * 4;
                s[0] = s[1] = s[2] = s[3] = 0.f;
            }
        }
        return;
    }
    const Row<T> R(row, a.V);
    Soft st{-INFINITY, 0.f, 0.f};
    for (int i = t; i < R.nvec; i += kThreads) {
        float v[kVec];
        R.load(i, v);
        float m = v[0];
#pragma unroll
        for (int j = 1; j < kVec; ++j) m = fmaxf(m, v[j]);
        st = rebase(st, fmaxf(st.m, m));
        const float ref = ref_of(st.m);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const float d = v[j] - ref, e = exp2f(d * kLog2e);
            st.s += e;
            st.a = fmaf(e, fmaxf(d, -3.0e38f), st.a);
        }
    }
    st = join_group(st);
    const bool some = st.s != 0.f;  // false: a row of -inf alone
    const float ref = ref_of(st.m), ls = logf(st.s), H = some ? ls - st.a / st.s : 0.f;
    if (t == 0) {
        a.logprob[r] = some ? (Row<T>::at(row, x) - ref) - ls : -INFINITY;
        a.entropy[r] = H;
        a.status[r] = 0;
        if (a.stats) {
            float* s = a.stats + (size_t)r * 4;
            s[0] = ref;
            s[1] = ls;
            s[2] = H;
            s[3] = some ? 1.f : 0.f;
        }
    }
    __shared__ uint64_t best[kWaves];
    uint64_t last = ~0ull;
    for (int n = 0; n < a.top_n; ++n) {  // the best key below the last one
        uint64_t k = 0;
        for (int i = t; i < R.nvec; i += kThreads) {
            float v[kVec];
            R.load(i, v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const uint64_t c = key_of(v[j], R.first(i) + j);
                if (c < last && c > k) k = c;
            }
        }
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)k, s);
            k = o > k ? o : k;
        }
        if ((t & 63) == 0) best[t >> 6] = k;
        __syncthreads();
        k = best[0];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) k = best[w] > k ? best[w] : k;
        __syncthreads();
        if (t == 0) {
            const bool is = k > kKeyNone;
            a.top_tokens[(size_t)r * a.top_n + n] = is ? key_index(k) : -1;
            a.top_logprob[(size_t)r * a.top_n + n] = is ? (key_value(k) - ref) - ls : -INFINITY;
        }
        last = k;
    }
}

struct LpGradArgs {
    const void* logits;
    const int32_t* tokens;
    const float *stats, *g_logprob, *g_entropy;
    int rows, V, tiles;
    void* grad;
};

// One workgroup per tile of a row: reads its logits and writes their gradient.
template <typename T>
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
    const float ref = s[0], ls = s[1], H = s[2];
    const float gl = a.g_logprob ? a.g_logprob[r] : 0.f, ge = a.g_entropy ? a.g_entropy[r] : 0.f;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int i = tile * kTileVecs + u * kThreads + t;
        if (i >= R.nvec) break;
        float v[kVec];
        if (live) {
            R.load(i, v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float lp = (v[j] - ref) - ls, p = exp2f(lp * kLog2e);
                float g = -p * fmaf(ge, fmaxf(lp, -3.0e38f) + H, gl);
                if (R.first(i) + j == x) g += gl;
                v[j] = g;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = 0.f;
        }
        store_block(out, R, i, whole, v);
    }
}

// ------------------------------------------------------------ draft divergence
struct KlArgs {
    const void *target, *draft;
    const uint8_t* mask;  // [B][K], or null: every row counts
    int K, Kt, V, tiles;  // target rows per request: Kt >= K
    float* kl;
    float* stats;  // [B*K][4]: max and ln of the sum, target then draft
    const float* g_kl;
    void* grad;
};

template <typename T>
__global__ __launch_bounds__(kThreads) void k_draft_kl(KlArgs a) {
    constexpr int kVec = Row<T>::kVec;
    const int r = blockIdx.x, t = threadIdx.x;
    if (a.mask && !a.mask[r]) {
        if (t == 0) {
            a.kl[r] = 0.f;
            if (a.stats) {
                float* s = a.stats + (size_t)r * 4;
                s[0] = s[1] = s[2] = s[3] = 0.f;
            }
        }
        return;
    }
    const int b = r / a.K, k = r % a.K;
    const Row<T> P(static_cast<const T*>(a.target) + ((size_t)b * a.Kt + k) * a.V, a.V);
    const T* drow = static_cast<const T*>(a.draft) + (size_t)r * a.V;
    Pair st{-INFINITY, 0.f, -INFINITY, 0.f, 0.f};
    // the two rows may be aligned differently: blocks follow the target's, the
    // draft's elements are read one by one
    for (int i = t; i < P.nvec; i += kThreads) {
        float p[kVec], q[kVec];
        P.load(i, p);
        const int e = P.first(i);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            q[j] = e + j >= 0 && e + j < a.V ? Row<T>::at(drow, e + j) : -INFINITY;
        float m = p[0], n = q[0];
#pragma unroll
        for (int j = 1; j < kVec; ++j) {
            m = fmaxf(m, p[j]);
            n = fmaxf(n, q[j]);
        }
        st = rebase(st, fmaxf(st.m, m), fmaxf(st.n, n));
        const float mr = ref_of(st.m), nr = ref_of(st.n);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            const float d = p[j] - mr, c = q[j] - nr;
            const float f = exp2f(d * kLog2e), g = exp2f(c * kLog2e);
            st.s += f;
            st.r += g;
            st.u += f > 0.f ? f * (d - c) : 0.f;
        }
    }
    st = join_group(st);
    if (t == 0) {
        const float ls = logf(st.s), lr = logf(st.r);
        // an empty target row says nothing; an empty draft row is infinitely far
        a.kl[r] = st.s == 0.f ? 0.f : st.r == 0.f ? INFINITY : st.u / st.s - ls + lr;
        if (a.stats) {
            float* s = a.stats + (size_t)r * 4;
            s[0] = ref_of(st.m);
            s[1] = ls;
            s[2] = ref_of(st.n);
            s[3] = lr;
        }
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_draft_kl_grad(KlArgs a) {
    constexpr int kVec = Row<T>::kVec;
    const int r = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles, t = threadIdx.x;
    const int b = r / a.K, k = r % a.K;
    const T* prow = static_cast<const T*>(a.target) + ((size_t)b * a.Kt + k) * a.V;
    const T* drow = static_cast<const T*>(a.draft) + (size_t)r * a.V;
    T* out = static_cast<T*>(a.grad) + (size_t)r * a.V;
    const Row<T> D(drow, a.V);
    const bool whole = (((uintptr_t)drow ^ (uintptr_t)out) & 15) == 0;
    const float* s = a.stats + (size_t)r * 4;
    const float m = s[0], ls = s[1], n = s[2], lr = s[3];
    const bool live = (!a.mask || a.mask[r]) && ls != -INFINITY && lr != -INFINITY;
    const float g = a.g_kl[r];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int i = tile * kTileVecs + u * kThreads + t;
        if (i >= D.nvec) break;
        float v[kVec];
        if (live) {
            D.load(i, v);
            const int e = D.first(i);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const float pl = e + j >= 0 && e + j < a.V ? Row<T>::at(prow, e + j) : -INFINITY;
                const float q = exp2f(((v[j] - n) - lr) * kLog2e), p = exp2f(((pl - m) - ls) * kLog2e);
                v[j] = g * (q - p);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kVec; ++j) v[j] = 0.f;
        }
        store_block(out, D, i, whole, v);
    }
}

// ---------------------------------------------------------------- host side
inline bool dtype_ok(spec_dtype d) { return d == SPEC_F32 || d == SPEC_BF16; }

// Tiles of a row at any alignment.
inline int tiles_of(spec_dtype d, int V) {
    const int vec = d == SPEC_BF16 ? 8 : 4;
    return ((V + vec - 1) / vec + 1 + kTileVecs - 1) / kTileVecs;
}
// One workgroup per tile, in a launch of fewer than 2^32 threads.
inline bool rows_ok(spec_dtype d, long long rows, int V) {
    return rows >= 1 && V >= 1 && V <= SPEC_MAX_V && rows * tiles_of(d, V) < (1ll << 24);
}
inline bool ws_ok(const void* p, size_t bytes, size_t need) {
    return need == 0 || (p && (uintptr_t)p % 256 == 0 && bytes >= need);
}

}  // namespace

extern "C" size_t spec_logprobs_workspace_bytes(spec_dtype dtype, int rows, int V, int top_n) {
    if (!dtype_ok(dtype) || !rows_ok(dtype, rows, V) || top_n < 0 || top_n > SPEC_MAX_TOP) return 0;
    return 256;
}

extern "C" spec_status spec_token_logprobs(const void* logits, spec_dtype dtype, const int32_t* tokens, int rows,
                                           int V, int top_n, float* out_logprob, float* out_entropy,
                                           int32_t* out_top_tokens, float* out_top_logprob, int32_t* out_status,
                                           float* out_stats, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype)) return SPEC_EDTYPE;
    if (!rows_ok(dtype, rows, V) || top_n < 0 || top_n > SPEC_MAX_TOP) return SPEC_EINVAL;
    if (!logits || !tokens || !out_logprob || !out_entropy || !out_status) return SPEC_EINVAL;
    if (top_n > 0 && (!out_top_tokens || !out_top_logprob)) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_logprobs_workspace_bytes(dtype, rows, V, top_n))) return SPEC_EWORKSPACE;
    const LpArgs a{logits, tokens, rows, V, top_n, out_logprob, out_entropy, out_top_tokens, out_top_logprob, out_status, out_stats};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == SPEC_BF16)
        k_logprobs<uint16_t><<<rows, kThreads, 0, st>>>(a);
    else
        k_logprobs<float><<<rows, kThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

extern "C" spec_status spec_token_logprobs_grad(const void* logits, spec_dtype dtype, const int32_t* tokens,
                                                const float* stats, const float* grad_logprob,
                                                const float* grad_entropy, int rows, int V, void* out_grad,
                                                void* stream) {
    if (!dtype_ok(dtype)) return SPEC_EDTYPE;
    if (!rows_ok(dtype, rows, V) || !logits || !tokens || !stats || !out_grad) return SPEC_EINVAL;
    const int tiles = tiles_of(dtype, V);
    const LpGradArgs a{logits, tokens, stats, grad_logprob, grad_entropy, rows, V, tiles, out_grad};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const unsigned grid = (unsigned)rows * (unsigned)tiles;
    if (dtype == SPEC_BF16)
        k_logprobs_grad<uint16_t><<<grid, kThreads, 0, st>>>(a);
    else
        k_logprobs_grad<float><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

namespace {
inline bool kl_ok(spec_dtype d, int B, int K, int Kt, int V) {
    return B >= 1 && K >= 1 && Kt >= K && rows_ok(d, (long long)B * K, V) && (long long)B * Kt < (1ll << 31);
}
}  // namespace

extern "C" size_t spec_draft_kl_workspace_bytes(spec_dtype dtype, int B, int K, int V) {
    return dtype_ok(dtype) && kl_ok(dtype, B, K, K, V) ? 256 : 0;
}

extern "C" spec_status spec_draft_kl(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                                     const uint8_t* mask, int B, int K, int target_rows, int V, float* out_kl,
                                     float* out_stats, void* workspace, size_t workspace_bytes, void* stream) {
    if (!dtype_ok(dtype)) return SPEC_EDTYPE;
    if (!kl_ok(dtype, B, K, target_rows, V) || !target_logits || !draft_logits || !out_kl) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_draft_kl_workspace_bytes(dtype, B, K, V))) return SPEC_EWORKSPACE;
    const KlArgs a{target_logits, draft_logits, mask, K, target_rows, V, 0, out_kl, out_stats, nullptr, nullptr};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    if (dtype == SPEC_BF16)
        k_draft_kl<uint16_t><<<B * K, kThreads, 0, st>>>(a);
    else
        k_draft_kl<float><<<B * K, kThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

extern "C" spec_status spec_draft_kl_grad(const void* target_logits, const void* draft_logits, spec_dtype dtype,
                                          const uint8_t* mask, const float* stats, const float* grad_kl, int B,
                                          int K, int target_rows, int V, void* out_grad, void* stream) {
    if (!dtype_ok(dtype)) return SPEC_EDTYPE;
    if (!kl_ok(dtype, B, K, target_rows, V) || !target_logits || !draft_logits || !stats || !grad_kl || !out_grad)
        return SPEC_EINVAL;
    const int tiles = tiles_of(dtype, V);
    const KlArgs a{target_logits, draft_logits, mask, K, target_rows, V, tiles, nullptr, const_cast<float*>(stats), grad_kl, out_grad};
    const hipStream_t st = static_cast<hipStream_t>(stream);
    const unsigned grid = (unsigned)(B * K) * (unsigned)tiles;
    if (dtype == SPEC_BF16)
        k_draft_kl_grad<uint16_t><<<grid, kThreads, 0, st>>>(a);
    else
        k_draft_kl_grad<float><<<grid, kThreads, 0, st>>>(a);
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP;
}

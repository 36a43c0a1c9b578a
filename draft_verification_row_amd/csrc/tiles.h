// tiles.h -- what the matrix products share: types and conversions, activations,
// matrix instructions on 16-byte chunks, the order of tiles, loads straight to
// LDS, and the checks of arguments.
#ifndef SPEC_TILES_H
#define SPEC_TILES_H

#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>
#include <utility>

#include "spec_verify.h"

namespace {

constexpr int kThreads = 256;

__host__ __device__ inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

typedef uint16_t bf16;  // bit patterns

__device__ inline float to_f(bf16 v) { return __uint_as_float((uint32_t)v << 16); }
__device__ inline float to_f(float v) { return v; }
__device__ inline void put(float* p, float v) { *p = v; }
__device__ inline void put(bf16* p, float f) {  // round to nearest even
    const uint32_t u = __float_as_uint(f);
    *p = (u & 0x7fffffffu) > 0x7f800000u ? (bf16)((u >> 16) | 0x40)
                                         : (bf16)((u + 0x7fffu + ((u >> 16) & 1)) >> 16);
}

// ---------------------------------------------------------------- activation
// 1 / (1 + e^-z) by the hardware's base-2 exponential and reciprocal, each good
// to a unit in the last place: an epilogue of one wave a SIMD is bound by its
// instructions (8192 x 4096 x 4096 with silu and residual: 350 us with expf
// and a division).
__device__ inline float sigmoid_of(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504088896340736f));
}
__device__ inline float act_of(float z, int act) {
    switch (act) {
        case SPEC_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
        case SPEC_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
        case SPEC_ACT_SILU: return z * sigmoid_of(z);
        default: return z;
    }
}
__device__ inline float act_slope(float z, int act) {
    switch (act) {
        case SPEC_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case SPEC_ACT_GELU:
            return 0.5f * (1.f + erff(z * 0.70710678118654752f)) +
                   z * __builtin_amdgcn_exp2f(-0.72134752044448170368f * z * z) * 0.39894228040143268f;
        case SPEC_ACT_SILU: {
            const float s = sigmoid_of(z);
            return s * fmaf(z, 1.f - s, 1.f);
        }
        default: return 1.f;
    }
}

// ------------------------------------------------------------ matrix product
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Both types are staged by 16-byte chunks (8 bf16 or 4 fp32 of one row), and
// a lane's operand of a matrix instruction is one chunk: 32x32x16 takes two
// chunks of 32 rows at once, lane l holding row l % 32 and chunk l / 32.  In
// fp32 the same two chunks are four 32x32x2 products, the i-th of the chunks'
// i-th elements; the order of the sum over k is the same for both operands.
__device__ inline f32x16 mfma32(bf16, u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ inline f32x16 mfma32(float, u32x4 a, u32x4 b, f32x16 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[i], y[i], c, 0, 0, 0);
    return c;
}

// One chunk of a row from element k on: zero past K, which need not be a whole
// number of chunks, and at any alignment of the row.
template <typename T>
__device__ inline u32x4 chunk_of(const T* row, int k, int K) {
    constexpr int kElems = 16 / (int)sizeof(T);
    struct Any {
        u32x4 v;
    } __attribute__((packed, aligned(sizeof(T))));
    if (k + kElems <= K) return reinterpret_cast<const Any*>(row + k)->v;
    u32x4 q = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < kElems; ++j)
        if (k + j < K) {
            if constexpr (sizeof(T) == 2)
                q[j >> 1] |= (uint32_t)row[k + j] << (16 * (j & 1));
            else
                q[j] = __float_as_uint(row[k + j]);
        }
    return q;
}

// ---------------------------------------------------------------- elements
__device__ inline uint32_t pack_bf16(float lo, float hi) {  // round to nearest even
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2){lo, hi}, bf16x2));
}
__device__ inline void put4(float* p, const float (&v)[4]) { *reinterpret_cast<f32x4*>(p) = (f32x4){v[0], v[1], v[2], v[3]}; }
__device__ inline void put4(bf16* p, const float (&v)[4]) {
    *reinterpret_cast<u32x2*>(p) = (u32x2){pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}
__device__ inline void get4(const float* p, float (&v)[4]) {
    const f32x4 q = *reinterpret_cast<const f32x4*>(p);
    for (int i = 0; i < 4; ++i) v[i] = q[i];
}
__device__ inline void get4(const bf16* p, float (&v)[4]) {
    const u32x2 q = *reinterpret_cast<const u32x2*>(p);
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float((i & 1) ? q[i >> 1] & 0xffff0000u : q[i >> 1] << 16);
}

// Four values as they lie in memory, so that a load ahead of its use stays one.
template <typename O>
using Raw4 = std::conditional_t<sizeof(O) == 2, u32x2, f32x4>;
__device__ inline float raw4_at(u32x2 q, int i) { return __uint_as_float((i & 1) ? q[i >> 1] & 0xffff0000u : q[i >> 1] << 16); }
__device__ inline float raw4_at(f32x4 q, int i) { return q[i]; }

// ------------------------------------------------------------ order and loads
// Consecutive workgroups go to different XCDs (blockIdx % 8); each XCD takes a
// run of neighbouring tiles instead, in columns of kGroupM tiles along m, so
// that its L2 holds what its tiles share.
constexpr int kXcds = 8, kGroupM = 8;
__device__ inline void tile_of(int id, int count, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int per = count / kXcds, rest = count % kXcds, x = id % kXcds, i = id / kXcds;
    const int at = x * per + min(x, rest) + i;
    const int group = kGroupM * tiles_n, first = at / group * kGroupM;
    const int high = min(kGroupM, tiles_m - first), in = at % group;
    tm = first + in % high;
    tn = in / high;
}

// 16 bytes a lane from the buffer straight to LDS at base + AT + lane * 16.
// NT: read once, not to be kept in the caches.  m0 cannot be listed as
// clobbered (the compiler reserves it); it is free, since nothing else in these
// kernels uses it.
template <int AT, bool NT>
__device__ inline void to_lds(__amdgpu_buffer_rsrc_t rsrc, uint32_t base, uint32_t voffset, uint32_t soffset) {
    if constexpr (NT)
        asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds"
                     :: "s"(base), "v"(voffset), "s"(rsrc), "s"(soffset), "n"(AT) : "memory", "scc");
    else
        asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :: "s"(base), "v"(voffset), "s"(rsrc), "s"(soffset), "n"(AT) : "memory", "scc");
}
template <int... I, typename F>
__device__ __attribute__((always_inline)) inline void each(std::integer_sequence<int, I...>, F f) {
    (f(std::integral_constant<int, I>()), ...);
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
inline bool types_ok(const spec_dtype& dtype, const spec_dtype& out_dtype) {
    const int d = value_of(dtype), o = value_of(out_dtype);
    return d == SPEC_BF16 ? (o == SPEC_BF16 || o == SPEC_F32) : d == SPEC_F32 && o == SPEC_F32;
}
inline bool act_ok(const spec_activation& a) { return value_of(a) >= SPEC_ACT_NONE && value_of(a) <= SPEC_ACT_SILU; }
inline bool type_ok(const spec_dtype& d) { return value_of(d) == SPEC_BF16 || value_of(d) == SPEC_F32; }
inline size_t elem(spec_dtype d) { return d == SPEC_BF16 ? 2 : 4; }
inline bool ws_ok(const void* p, size_t bytes, size_t need) {
    return p && (uintptr_t)p % 256 == 0 && bytes >= need;
}
inline spec_status launched() { return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP; }
inline long long padded(spec_dtype d, long long n) {
    const long long c = 16 / (long long)elem(d);
    return (n + c - 1) / c * c;
}

}  // namespace

#endif  // SPEC_TILES_H

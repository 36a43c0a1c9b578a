// linear.hip -- the matrix product that a draft head is made of, for gfx950
// (MI355X): y = residual + act(x W^T + bias) and its gradients.
//
//   z = x W^T + bias        x [M][K], W [N][K], bias [N]
//   y = residual + act(z)   residual, y, z [M][N]
//   dz = dy act'(z)         dx = dz W, dW = dz^T x, dbias = sum over rows of dz
// Products are summed in fp32; bias, activation and residual are applied to
// the fp32 sum and the result is rounded once.
#include <hip/hip_runtime.h>

#include <math.h>
#include <stddef.h>
#include <stdint.h>

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
__device__ inline float act_of(float z, int act) {
    switch (act) {
        case SPEC_ACT_RELU: return z > 0.f ? z : (z != z ? z : 0.f);
        case SPEC_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
        case SPEC_ACT_SILU: return z / (1.f + expf(-z));
        default: return z;
    }
}
__device__ inline float act_slope(float z, int act) {
    switch (act) {
        case SPEC_ACT_RELU: return z > 0.f ? 1.f : 0.f;
        case SPEC_ACT_GELU:
            return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
        case SPEC_ACT_SILU: {
            const float s = 1.f / (1.f + expf(-z));
            return s * fmaf(z, 1.f - s, 1.f);
        }
        default: return 1.f;
    }
}

// ------------------------------------------------------------ matrix product
// C[m][n] = sum_k A[m sam + k sak] B[n sbn + k sbk]
struct Gemm {
    const void *A, *B;
    int64_t sam, sak, sbn, sbk;
    int M, N, K;
    const void *bias, *residual;
    int act;
    void *out, *preact;
};

constexpr int kTile = 64, kStep = 16;

// 64 x 64 outputs per workgroup, 4 x 4 per thread, fp32 multiply-adds from LDS.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void k_gemm(Gemm g) {
    __shared__ float As[kStep][kTile + 4], Bs[kStep][kTile + 4];
    const T* A = static_cast<const T*>(g.A);
    const T* B = static_cast<const T*>(g.B);
    const int tn = (g.N + kTile - 1) / kTile;
    const int m0 = (blockIdx.x / tn) * kTile, n0 = (blockIdx.x % tn) * kTile;
    const int t = threadIdx.x, tx = t % 16, ty = t / 16;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < g.K; k0 += kStep) {
        for (int i = t; i < kTile * kStep; i += kThreads) {
            const int k = i % kStep, r = i / kStep;
            const bool in = k0 + k < g.K;
            As[k][r] = in && m0 + r < g.M ? to_f(A[(m0 + r) * g.sam + (k0 + k) * g.sak]) : 0.f;
            Bs[k][r] = in && n0 + r < g.N ? to_f(B[(n0 + r) * g.sbn + (k0 + k) * g.sbk]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(As[k][ty * 4 + i], Bs[k][tx * 4 + j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (m >= g.M || n >= g.N) continue;
            const size_t at = (size_t)m * g.N + n;
            float z = acc[i][j];
            if (g.bias) z += to_f(static_cast<const T*>(g.bias)[n]);
            if (g.preact) put(static_cast<T*>(g.preact) + at, z);
            float y = act_of(z, g.act);
            if (g.residual) y += to_f(static_cast<const O*>(g.residual)[at]);
            put(static_cast<O*>(g.out) + at, y);
        }
}

// dz = dy act'(z), rounded to the operands' type
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void k_slope(const O* dy, const T* preact, int act, size_t n, T* dz) {
    for (size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kThreads)
        put(dz + i, to_f(dy[i]) * (preact ? act_slope(to_f(preact[i]), act) : 1.f));
}

// dbias[n] = sum over m of dz[m][n]: one wave per 64 columns
template <typename T>
__global__ __launch_bounds__(64) void k_colsum(const T* dz, int M, int N, T* out) {
    const int n = blockIdx.x * 64 + threadIdx.x;
    if (n >= N) return;
    float s = 0.f;
    for (int m = 0; m < M; ++m) s += to_f(dz[(size_t)m * N + n]);
    put(out + n, s);
}

// ---------------------------------------------------------------- host side
inline bool types_ok(spec_dtype d, spec_dtype o) {
    return d == SPEC_BF16 ? (o == SPEC_BF16 || o == SPEC_F32) : d == SPEC_F32 && o == SPEC_F32;
}
constexpr long long kMaxElems = 1ll << 35;
inline bool sizes_ok(long long M, long long N, long long K) {
    return M >= 1 && N >= 1 && K >= 1 && M <= SPEC_MAX_LINEAR && N <= SPEC_MAX_LINEAR && K <= SPEC_MAX_LINEAR &&
           M * N < kMaxElems && M * K < kMaxElems && N * K < kMaxElems;
}
inline bool act_ok(int a) { return a >= SPEC_ACT_NONE && a <= SPEC_ACT_SILU; }
inline size_t elem(spec_dtype d) { return d == SPEC_BF16 ? 2 : 4; }
inline bool ws_ok(const void* p, size_t bytes, size_t need) {
    return p && (uintptr_t)p % 256 == 0 && bytes >= need;
}
inline spec_status launched() { return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_EHIP; }

void launch_gemm(const Gemm& g, spec_dtype d, spec_dtype o, hipStream_t st) {
    const unsigned grid = (unsigned)((g.M + kTile - 1) / kTile) * (unsigned)((g.N + kTile - 1) / kTile);
    if (d == SPEC_F32)
        k_gemm<float, float><<<grid, kThreads, 0, st>>>(g);
    else if (o == SPEC_F32)
        k_gemm<bf16, float><<<grid, kThreads, 0, st>>>(g);
    else
        k_gemm<bf16, bf16><<<grid, kThreads, 0, st>>>(g);
}

}  // namespace

extern "C" size_t spec_linear_workspace_bytes(spec_dtype dtype, int M, int N, int K) {
    if (!types_ok(dtype, SPEC_F32) || !sizes_ok(M, N, K)) return 0;
    return 256;
}

extern "C" spec_status spec_linear(const void* x, const void* weight, const void* bias, const void* residual,
                                   spec_dtype dtype, spec_dtype out_dtype, spec_activation activation, int M, int N,
                                   int K, void* out, void* out_preact, void* workspace, size_t workspace_bytes,
                                   void* stream) {
    if (!types_ok(dtype, out_dtype)) return SPEC_EDTYPE;
    if (!sizes_ok(M, N, K) || !act_ok(activation) || !x || !weight || !out) return SPEC_EINVAL;
    if (!ws_ok(workspace, workspace_bytes, spec_linear_workspace_bytes(dtype, M, N, K))) return SPEC_EWORKSPACE;
    const Gemm g{x, weight, K, 1, K, 1, M, N, K, bias, residual, activation, out, out_preact};
    launch_gemm(g, dtype, out_dtype, static_cast<hipStream_t>(stream));
    return launched();
}

extern "C" size_t spec_linear_grad_workspace_bytes(spec_dtype dtype, int M, int N, int K) {
    if (!types_ok(dtype, SPEC_F32) || !sizes_ok(M, N, K)) return 0;
    return align_up((size_t)M * N * elem(dtype), 256);
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
    const size_t n = (size_t)M * N;
    const unsigned grid = (unsigned)((n + kThreads - 1) / kThreads < 65536 ? (n + kThreads - 1) / kThreads : 65536);
    const void* z = activation == SPEC_ACT_NONE ? nullptr : preact;
    if (dtype == SPEC_F32)
        k_slope<float, float><<<grid, kThreads, 0, st>>>((const float*)grad_out, (const float*)z, activation, n, (float*)workspace);
    else if (out_dtype == SPEC_F32)
        k_slope<bf16, float><<<grid, kThreads, 0, st>>>((const float*)grad_out, (const bf16*)z, activation, n, (bf16*)workspace);
    else
        k_slope<bf16, bf16><<<grid, kThreads, 0, st>>>((const bf16*)grad_out, (const bf16*)z, activation, n, (bf16*)workspace);
    if (grad_bias) {
        if (dtype == SPEC_F32)
            k_colsum<float><<<(N + 63) / 64, 64, 0, st>>>((const float*)workspace, M, N, (float*)grad_bias);
        else
            k_colsum<bf16><<<(N + 63) / 64, 64, 0, st>>>((const bf16*)workspace, M, N, (bf16*)grad_bias);
    }
    if (grad_x)
        launch_gemm({workspace, weight, N, 1, 1, K, M, K, N, nullptr, nullptr, 0, grad_x, nullptr}, dtype, dtype, st);
    if (grad_weight)
        launch_gemm({workspace, x, 1, N, 1, K, N, K, M, nullptr, nullptr, 0, grad_weight, nullptr}, dtype, dtype, st);
    return launched();
}

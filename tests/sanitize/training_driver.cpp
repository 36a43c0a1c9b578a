// Host-side driver of the training operators' C ABI under AddressSanitizer and
// UndefinedBehaviorSanitizer: every size query over the range of its arguments,
// and every entry point with arguments it must reject.  No kernel is launched.
#include <stdint.h>
#include <stdio.h>

#include "spec_verify.h"

static int failures = 0;
#define CHECK(c) do { if (!(c)) { ++failures; fprintf(stderr, "%s:%d: %s\n", __FILE__, __LINE__, #c); } } while (0)

int main() {
    const int sizes[] = {INT32_MIN, -1, 0, 1, 7, 64, 65, 700, 8192, 128256, 1 << 20, (1 << 20) + 1, INT32_MAX};
    const spec_dtype types[] = {SPEC_F32, SPEC_BF16};
    for (spec_dtype dt : types)
        for (int m : sizes)
            for (int n : sizes)
                for (int k : sizes) {
                    const bool ok = m > 0 && n > 0 && k > 0 && m <= 1 << 20 && n <= 1 << 20 && k <= 1 << 20;
                    const size_t q[] = {spec_embedding_grad_workspace_bytes(dt, m, n, k), spec_gated_linear_workspace_bytes(dt, m, n, k),
                                        spec_gated_linear_grad_workspace_bytes(dt, m, n, k), spec_cross_entropy_workspace_bytes(dt, m, n, k),
                                        spec_cross_entropy_grad_workspace_bytes(dt, m, n, k)};
                    for (size_t b : q) CHECK(ok || b == 0);
                }
    void* p = (void*)4096;
    int32_t* t = (int32_t*)4096;
    float* f = (float*)4096;
    const spec_dtype bf = SPEC_BF16;
    const spec_activation silu = SPEC_ACT_SILU;
    const size_t big = (size_t)1 << 40;
    CHECK(spec_embedding(nullptr, bf, t, 1.f, 4, 8, 16, p, nullptr) == SPEC_EINVAL);
    CHECK(spec_embedding(p, bf, t, 1.f, 0, 8, 16, p, nullptr) == SPEC_EINVAL);
    CHECK(spec_embedding_grad(t, nullptr, bf, 1.f, 4, 8, 16, p, p, big, nullptr) == SPEC_EINVAL);
    CHECK(spec_embedding_grad(t, p, bf, 1.f, 4, 8, 16, p, p, 0, nullptr) == SPEC_EWORKSPACE);
    CHECK(spec_gated_linear(p, p, p, bf, silu, 4, 8, 16, p, f, nullptr, p, big, nullptr) == SPEC_EINVAL);
    CHECK(spec_gated_linear(p, p, p, bf, silu, 4, 8, 16, p, f, f, p, 0, nullptr) == SPEC_EWORKSPACE);
    CHECK(spec_gated_linear_grad(p, nullptr, p, f, f, p, bf, silu, 4, 8, 16, p, p, p, p, big, nullptr) == SPEC_EINVAL);
    CHECK(spec_gated_linear_grad(p, p, p, f, f, p, bf, silu, 4, 8, 16, p, p, p, (void*)4097, big, nullptr) == SPEC_EWORKSPACE);
    CHECK(spec_cross_entropy(p, p, nullptr, bf, nullptr, 4, 8, 16, f, f, t, f, p, big, nullptr) == SPEC_EINVAL);
    CHECK(spec_cross_entropy(p, p, nullptr, bf, t, 4, 8, 16, f, f, t, f, p, 1, nullptr) == SPEC_EWORKSPACE);
    CHECK(spec_cross_entropy_grad(p, p, nullptr, bf, t, nullptr, f, f, 4, 8, 16, p, p, p, p, big, nullptr) == SPEC_EINVAL);
    CHECK(spec_cross_entropy_grad(p, p, nullptr, bf, t, f, f, f, 4, 8, 16, p, p, p, nullptr, big, nullptr) == SPEC_EWORKSPACE);
    printf("%d failures\n", failures);
    return failures != 0;
}

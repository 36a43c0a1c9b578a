// Sanitizer driver for the host side of the head operators' C entry points
// (test infrastructure): the size queries over the whole range of their
// arguments, and every entry point with arguments that it must reject before
// anything is enqueued, under an AddressSanitizer / UndefinedBehaviorSanitizer
// build of the library's host code.  No kernel is launched and no device is
// needed.  Exit status 0 when every call returned the expected status.
#include <climits>
#include <cstdint>
#include <cstdio>

#include "spec_verify.h"

static int failures = 0;

static void expect(const char* what, int got, int want) {
    if (got != want) {
        std::printf("FAIL %s: status %d, want %d\n", what, got, want);
        ++failures;
    }
}

int main() {
    void* P = reinterpret_cast<void*>(uintptr_t(4096));
    void* odd = reinterpret_cast<void*>(uintptr_t(4100));
    void* W = reinterpret_cast<void*>(uintptr_t(1) << 20);
    auto* I = static_cast<int32_t*>(P);
    auto* F = static_cast<float*>(P);
    auto* G = static_cast<float*>(odd);
    const size_t all = ~size_t(0);

    // size queries: no overflow anywhere, 0 exactly where the call refuses
    const int n[] = {INT_MIN, -1, 0, 1, 2, 63, 64, 65, 4095, 32000, 65536, 262144, 262145, 1 << 20, (1 << 20) + 1, 1 << 24, INT_MAX};
    const spec_dtype types[] = {SPEC_F32, SPEC_BF16};
    long asked = 0;
    for (spec_dtype d : types)
        for (int a : n)
            for (int b : n)
                for (int c : n) {
                    const size_t lp = spec_logprobs_workspace_bytes(d, a, b, c);
                    if (lp == 0) expect("logprobs refused", spec_token_logprobs(P, d, I, a, b, c, F, F, I, F, I, nullptr, W, all, nullptr), SPEC_EINVAL);
                    const size_t kl = spec_draft_kl_workspace_bytes(d, a, b, c);
                    if (kl == 0) expect("kl refused", spec_draft_kl(P, P, d, nullptr, a, b, b, c, F, nullptr, W, all, nullptr), SPEC_EINVAL);
                    const size_t l = spec_linear_workspace_bytes(d, a, b, c), g = spec_linear_grad_workspace_bytes(d, a, b, c);
                    if (l == 0) expect("linear refused", spec_linear(P, P, nullptr, nullptr, d, d, SPEC_ACT_NONE, a, b, c, P, nullptr, W, all, nullptr), SPEC_EINVAL);
                    if (g == 0) expect("linear grad refused", spec_linear_grad(P, P, nullptr, P, d, d, SPEC_ACT_NONE, a, b, c, P, P, P, W, all, nullptr), SPEC_EINVAL);
                    expect("linear queries agree", (l == 0) == (g == 0), 1);
                    // one byte short, and a workspace off its alignment
                    if (lp) expect("logprobs short", spec_token_logprobs(P, d, I, a, b, c, F, F, I, F, I, nullptr, W, lp - 1, nullptr), SPEC_EWORKSPACE);
                    if (kl) expect("kl short", spec_draft_kl(P, P, d, nullptr, a, b, b, c, F, nullptr, W, kl - 1, nullptr), SPEC_EWORKSPACE);
                    if (l) expect("linear short", spec_linear(P, P, nullptr, nullptr, d, d, SPEC_ACT_NONE, a, b, c, P, nullptr, W, l - 1, nullptr), SPEC_EWORKSPACE);
                    if (g) expect("linear grad short", spec_linear_grad(P, P, nullptr, P, d, d, SPEC_ACT_NONE, a, b, c, P, P, P, W, g - 1, nullptr), SPEC_EWORKSPACE);
                    if (l) expect("linear misaligned", spec_linear(P, P, nullptr, nullptr, d, d, SPEC_ACT_NONE, a, b, c, P, nullptr, odd, all, nullptr), SPEC_EWORKSPACE);
                    ++asked;
                }

    // log probabilities
    expect("lp null", spec_token_logprobs(nullptr, SPEC_BF16, I, 4, 100, 0, F, F, nullptr, nullptr, I, nullptr, W, all, nullptr), SPEC_EINVAL);
    expect("lp top null", spec_token_logprobs(P, SPEC_BF16, I, 4, 100, 3, F, F, nullptr, F, I, nullptr, W, all, nullptr), SPEC_EINVAL);
    expect("lp stats", spec_token_logprobs(P, SPEC_BF16, I, 4, 100, 0, F, F, nullptr, nullptr, I, G, W, all, nullptr), SPEC_EINVAL);
    expect("lp dtype", spec_token_logprobs(P, (spec_dtype)2, I, 4, 100, 0, F, F, nullptr, nullptr, I, nullptr, W, all, nullptr), SPEC_EDTYPE);
    expect("lp grad dtype", spec_token_logprobs_grad(P, (spec_dtype)7, I, F, F, F, 4, 100, P, nullptr), SPEC_EDTYPE);
    expect("lp grad stats", spec_token_logprobs_grad(P, SPEC_F32, I, G, F, F, 4, 100, P, nullptr), SPEC_EINVAL);
    expect("lp grad rows", spec_token_logprobs_grad(P, SPEC_F32, I, F, F, F, INT_MAX, 262144, P, nullptr), SPEC_EINVAL);
    expect("lp grad out", spec_token_logprobs_grad(P, SPEC_F32, I, F, F, F, 4, 100, nullptr, nullptr), SPEC_EINVAL);
    // divergence
    expect("kl rows", spec_draft_kl(P, P, SPEC_BF16, nullptr, 2, 3, 2, 100, F, nullptr, W, all, nullptr), SPEC_EINVAL);
    expect("kl target rows", spec_draft_kl(P, P, SPEC_BF16, nullptr, 65536, 1, INT_MAX, 100, F, nullptr, W, all, nullptr), SPEC_EINVAL);
    expect("kl dtype", spec_draft_kl(P, P, (spec_dtype)3, nullptr, 2, 3, 3, 100, F, nullptr, W, all, nullptr), SPEC_EDTYPE);
    expect("kl grad null", spec_draft_kl_grad(P, P, SPEC_BF16, nullptr, F, nullptr, 2, 3, 3, 100, P, nullptr), SPEC_EINVAL);
    expect("kl grad stats", spec_draft_kl_grad(P, P, SPEC_BF16, nullptr, G, F, 2, 3, 3, 100, P, nullptr), SPEC_EINVAL);
    // product
    expect("linear types", spec_linear(P, P, nullptr, nullptr, SPEC_F32, SPEC_BF16, SPEC_ACT_NONE, 4, 8, 16, P, nullptr, W, all, nullptr), SPEC_EDTYPE);
    expect("linear act", spec_linear(P, P, nullptr, nullptr, SPEC_F32, SPEC_F32, (spec_activation)4, 4, 8, 16, P, nullptr, W, all, nullptr), SPEC_EINVAL);
    expect("linear grad preact", spec_linear_grad(P, P, nullptr, P, SPEC_F32, SPEC_F32, SPEC_ACT_SILU, 4, 8, 16, P, P, P, W, all, nullptr), SPEC_EINVAL);
    expect("linear grad x", spec_linear_grad(nullptr, P, P, P, SPEC_F32, SPEC_F32, SPEC_ACT_SILU, 4, 8, 16, P, P, P, W, all, nullptr), SPEC_EINVAL);

    std::printf("heads sanitizer driver: %ld sizes, %d failures\n", asked, failures);
    return failures ? 1 : 0;
}

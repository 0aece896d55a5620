// layers_check.cpp - drives the host side of the decoding layers' entry points for a
// build whose host code runs under AddressSanitizer and UndefinedBehaviorSanitizer.
// Test infrastructure: built and run by tests/test_layers_host.py, on a machine with
// or without a GPU.
//
// Every call made here fails validation, so it returns before any HIP call and its
// pointers are never dereferenced.  Each size in turn takes values that break naive
// size arithmetic; sizes that are good give the workspaces' sizes alone.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "../../include/fp4.h"

namespace {

int failures = 0;
long calls = 0;

uint8_t *const A16 = reinterpret_cast<uint8_t *>(uintptr_t{0x10000});
const int32_t *const I = reinterpret_cast<const int32_t *>(uintptr_t{0x10000});
float *const F = reinterpret_cast<float *>(uintptr_t{0x10000});
constexpr int64_t LMIN = std::numeric_limits<int64_t>::min(), LMAX = std::numeric_limits<int64_t>::max();
constexpr int32_t MIN = std::numeric_limits<int32_t>::min(), MAX = std::numeric_limits<int32_t>::max();

void refused(int got, int line) {
    ++calls;
    if (got == FP4_OK || got == FP4_E_HIP) {
        std::fprintf(stderr, "line %d: returned %d, expected an argument error\n", line, got);
        ++failures;
    }
}

void expect(bool holds, int line) {
    ++calls;
    if (!holds) {
        std::fprintf(stderr, "line %d: does not hold\n", line);
        ++failures;
    }
}

void linear(int64_t m, int64_t n, int64_t k, int line) {
    for (fp4_format fmt : {FP4_MXFP4, FP4_NVFP4}) {
        refused(fp4_linear_w4(fmt, A16, FP4_BF16, m, k, A16, A16, F, n, A16, FP4_BF16, nullptr), line);
        refused(fp4_linear_w4_packed(fmt, A16, FP4_F32, m, k, A16, F, n, A16, FP4_F32, nullptr), line);
    }
}

void route(int64_t tokens, int64_t hidden, int32_t experts, int32_t top_k, int line) {
    refused(fp4_moe_route(A16, FP4_BF16, tokens, hidden, A16, FP4_BF16, experts, top_k, 1,
                          reinterpret_cast<int32_t *>(A16), F, A16, SIZE_MAX, nullptr), line);
}

void experts(const fp4_moe_weights &w, int64_t tokens, int32_t top_k, int line) {
    for (fp4_format fmt : {FP4_MXFP4, FP4_NVFP4}) {
        refused(fp4_moe_experts(fmt, &w, A16, FP4_BF16, tokens, I, F, top_k, A16, FP4_BF16, A16,
                                SIZE_MAX, nullptr, nullptr), line);
        expect(fp4_moe_experts_workspace_bytes(&w, fmt, tokens, top_k, FP4_F32) == 0, line);
    }
}

void rotate(const fp4_head_rows &q, const fp4_head_rows &k, int32_t dim, int32_t rotary, int32_t seqs,
            int64_t tokens, int line) {
    refused(fp4_norm_rotate(&q, &k, FP4_BF16, FP4_F32, dim, 1e-6f, I, I, seqs, tokens,
                            reinterpret_cast<const double *>(A16), rotary, 0, nullptr, nullptr), line);
}

}  // namespace

int main() {
    for (int64_t v : {LMIN, LMIN + 1, (int64_t)-512, (int64_t)-1, (int64_t)0, (int64_t)1 << 27,
                      (int64_t)1 << 31, (int64_t)1 << 40, (int64_t)1 << 62, LMAX - 511, LMAX}) {
        linear(v, 64, 512, __LINE__);
        linear(4, v, 512, __LINE__);
        linear(4, 64, v, __LINE__);
        linear(v, v, v, __LINE__);
        route(v, 64, 16, 2, __LINE__);
        if (v <= 0 || v > MAX) route(4, v, 16, 2, __LINE__);
        const fp4_moe_weights good = {A16, A16, A16, A16, F, F, 64, 96, 8, 0};
        experts(good, v, 2, __LINE__);
        fp4_moe_weights w = good;
        w.hidden = v;
        experts(w, 4, 2, __LINE__);
        w = good;
        w.inner = v;
        experts(w, 4, 2, __LINE__);
        w.hidden = v;
        experts(w, 4, 2, __LINE__);
    }
    linear((1 << 19) + 1, 64, 512, __LINE__);
    linear(4, (1 << 26) + 1, 512, __LINE__);
    linear(4, 64, (1 << 20) + 512, __LINE__);
    route((1 << 19) + 1, 64, 16, 2, __LINE__);
    for (int32_t v : {MIN, -1, 0, 1025, MAX}) {
        route(4, 64, v, 2, __LINE__);
        route(4, 64, 16, v, __LINE__);
        fp4_moe_weights w = {A16, A16, A16, A16, F, F, 64, 96, v, 0};
        experts(w, 4, 2, __LINE__);
        w.experts = 8;
        experts(w, 4, v, __LINE__);
        expect(fp4_moe_route_workspace_bytes(4, 64, v) == 0, __LINE__);
    }
    // the largest sizes that fit: their workspaces in size_t
    const fp4_moe_weights most = {A16, A16, A16, A16, F, F, 1 << 14, 1 << 16, 1024, 0};
    expect(fp4_moe_experts_workspace_bytes(&most, FP4_MXFP4, 1 << 19, 32, FP4_F32) ==
               ((size_t)1 << 19) * 32 * 3 * (1 << 16) * 2, __LINE__);
    expect(fp4_moe_route_workspace_bytes(1 << 19, 64, 1024) == ((size_t)1 << 19) * 1024 * 8, __LINE__);

    const fp4_head_rows good = {A16, A16, 512, 128, 512, 128, A16, 4};
    for (int32_t v : {MIN, -128, -1, 0, 1, 32, 80, 300, MAX}) {
        rotate(good, good, v, 64, 2, 4, __LINE__);
        if (v != 32 && v != 80) rotate(good, good, 128, v, 2, 4, __LINE__);
        fp4_head_rows bad = good;
        if (v <= 0 || v == MAX) {
            bad.heads = v;
            rotate(bad, good, 128, 128, 2, 4, __LINE__);
            rotate(good, bad, 128, 128, 2, 4, __LINE__);
            rotate(good, good, 128, 128, v, 4, __LINE__);
        }
    }
    for (int64_t v : {LMIN, (int64_t)-1, (int64_t)1, (int64_t)1 << 61, LMAX}) {
        fp4_head_rows bad = good;
        bad.x_token_stride = v;
        rotate(bad, good, 128, 128, 2, 4, __LINE__);
        rotate(good, bad, 128, 128, 2, 4, __LINE__);
        bad = good;
        bad.y_head_stride = v;
        rotate(bad, good, 128, 128, 2, 4, __LINE__);
        if (v != 1) rotate(good, good, 128, 128, 2, v, __LINE__);
    }
    std::printf("%ld calls, %d failures\n", calls, failures);
    return failures != 0;
}

// kv_check.cpp - drives the host side of the cache entry points for a build
// whose host code runs under AddressSanitizer and UndefinedBehaviorSanitizer.
// Test infrastructure: built and run by tests/test_kv_host.py, on a machine with
// or without a GPU.
//
// Every call made here fails validation, or has no rows, so it returns before any
// HIP call and its pointers are never dereferenced.  Each size in turn takes
// values that break naive size arithmetic.
#include <cstdint>
#include <cstdio>
#include <limits>

#include "../../include/fp4.h"

namespace {

int failures = 0;
long calls = 0;

uint8_t *const A16 = reinterpret_cast<uint8_t *>(uintptr_t{0x10000});

void refused(int got, int line) {
    ++calls;
    if (got == FP4_OK || got == FP4_E_HIP) {
        std::fprintf(stderr, "line %d: returned %d, expected an argument error\n", line, got);
        ++failures;
    }
}

void refuse_all(const fp4_kv_cache &c, const fp4_kv_batch &b, int line) {
    refused(fp4_kv_cache_write(&c, &b, A16, 256, 64, A16, 256, 64, FP4_BF16, nullptr, nullptr), line);
    refused(fp4_kv_cache_read(&c, &b, A16, A16, FP4_F32, nullptr, nullptr), line);
    refused(fp4_kv_attention(&c, &b, A16, 256, 64, FP4_BF16, 4, 0.1f, 1, 0, A16, nullptr, nullptr, 0,
                             nullptr, nullptr), line);
    ++calls;
    if (fp4_kv_attention_workspace_bytes(&c, &b, 4, 0, FP4_BF16) != 0) ++failures;
}

}  // namespace

int main() {
    const int32_t *I = reinterpret_cast<const int32_t *>(A16);
    const fp4_kv_cache good_cache = {A16, A16, A16, A16, 64, 2, 64, 128};
    const fp4_kv_batch good_batch = {I, I, I, 8, 16, 4, 16};
    constexpr int32_t MIN = std::numeric_limits<int32_t>::min(), MAX = std::numeric_limits<int32_t>::max();
    constexpr int64_t LMIN = std::numeric_limits<int64_t>::min(), LMAX = std::numeric_limits<int64_t>::max();
    for (int64_t v : {LMIN, (int64_t)-1, (int64_t)0, (int64_t)MAX + 1, LMAX}) {
        fp4_kv_cache c = good_cache;
        c.pages = v;
        refuse_all(c, good_batch, __LINE__);
    }
    for (int32_t v : {MIN, -64, -1, 0, 1, 15, 24, 100, 257, MAX}) {
        fp4_kv_cache c = good_cache;
        c.block = v;
        refuse_all(c, good_batch, __LINE__);
        c = good_cache;
        c.head_dim = v;
        refuse_all(c, good_batch, __LINE__);
    }
    for (int32_t v : {MIN, -1, 0, 65536, MAX}) {
        fp4_kv_cache c = good_cache;
        c.kv_heads = v;
        refuse_all(c, good_batch, __LINE__);
    }
    for (int32_t v : {MIN, -1, 0, MAX}) {
        fp4_kv_batch b = good_batch;
        b.seqs = v;
        refuse_all(good_cache, b, __LINE__);
        b = good_batch;
        b.table_width = v;
        b.table_stride = LMAX;
        refuse_all(good_cache, b, __LINE__);
    }
    for (int64_t v : {LMIN, (int64_t)-1, (int64_t)(1 << 23) + 1, LMAX}) {
        fp4_kv_batch b = good_batch;
        b.tokens = v;
        refuse_all(good_cache, b, __LINE__);
    }
    for (int64_t v : {LMIN, (int64_t)-1, (int64_t)15}) {
        fp4_kv_batch b = good_batch;
        b.table_stride = v;
        refuse_all(good_cache, b, __LINE__);
    }
    for (int64_t v : {LMIN, (int64_t)-64, (int64_t)3, LMAX, LMAX - 7}) {
        refused(fp4_kv_cache_write(&good_cache, &good_batch, A16, v, 128, A16, 256, 128, FP4_BF16,
                                   nullptr, nullptr), __LINE__);
        refused(fp4_kv_cache_write(&good_cache, &good_batch, A16, 256, 128, A16, 256, v, FP4_F32,
                                   nullptr, nullptr), __LINE__);
        refused(fp4_kv_attention(&good_cache, &good_batch, A16, v, 128, FP4_BF16, 4, 0.1f, 1, 0, A16,
                                 nullptr, nullptr, 0, nullptr, nullptr), __LINE__);
    }
    for (int32_t v : {MIN, -4, 0, 1, 3, 65536, MAX})
        refused(fp4_kv_attention(&good_cache, &good_batch, A16, 512, 128, FP4_F32, v, 0.1f, 1, 0, A16,
                                 nullptr, nullptr, 0, nullptr, nullptr), __LINE__);
    // every shape that has a plan has a workspace size that is 0 or holds its parts
    for (int32_t width : {1, 7, 64, 4096, 1 << 19})
        for (int64_t tokens : {1, 5, 4096, 1 << 23})
            for (int32_t seqs : {1, 64, 1 << 20})
                for (int32_t heads : {1, 8, 65535})
                    for (int32_t window : {0, 1, 1000, MAX}) {
                        const fp4_kv_cache c = {A16, A16, A16, A16, MAX, 1, 256, 256};
                        const fp4_kv_batch b = {I, I, I, tokens, width, seqs, width};
                        for (fp4_dtype t : {FP4_F32, FP4_BF16}) {
                            const size_t n = fp4_kv_attention_workspace_bytes(&c, &b, heads, window, t);
                            ++calls;
                            if (n != 0 && n < 2 * (size_t)tokens * heads * 258 * 4) {
                                std::fprintf(stderr, "workspace %zu for %d %lld %d %d %d\n", n, width,
                                             (long long)tokens, seqs, heads, window);
                                ++failures;
                            }
                        }
                    }
    std::printf("%ld calls, %d failures\n", calls, failures);
    return failures != 0;
}

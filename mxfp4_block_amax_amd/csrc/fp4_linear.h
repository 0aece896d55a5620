// fp4_linear.h - which kernel takes a four-bit weight's linear layer of 17 tokens and
// more: host code alone.  Internal to libfp4.so.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace fp4dev {

constexpr int LINEAR_ROWS = 32;  // weight rows of a workgroup, up to 16 tokens
constexpr int WIDE_PARTS = 4;    // 16s of weight rows of a wave, more tokens

// The kernel for 17 tokens and more: the wide one with `tiles` of 16 tokens and 64
// row_waves rows, or (0) the 16-token one.  A kernel's time is its rounds of a workgroup a
// CU; `cost` is a round's.  (Packed MXFP4, K = 8192, the 16-token kernel, then 64 rows x 16
// and 32 tokens, then 128 x 16, 32 and 64: 64 x 2048 9.8, 13.7, 17.8, 20, 24, 38 us; 32 x
// 8192 21, 16, 20, 22, 26, 37; 64 x 8192 39, 30, 20, 22, 25, 39; 32 x 28672 65, 65, 43, 53,
// 33, 43; 64 x 28672 126, 112, 80, 103, 62, 47; 128 x 8192 74, 56, 39, 41, 27, 39.)  NVFP4
// and row-major weights take 5 to 25 % longer, every tile about alike: with K = 8192 the
// tile chosen is within 3 % of their best at all of these.  With K = 2048, where starting a
// workgroup and joining its sums weigh more, it is so at four of the six; 32 x 8192 takes
// 9.5 us where the 16-token kernel takes 7.3, 64 x 8192 12.7 where 128 rows x 16 take 9.5.
struct Wide {
    int tiles, row_waves, cost;
};
inline Wide wide_tile(int64_t M, int64_t N) {
    const int64_t tokens = (M + 15) / 16;
    const auto rounds = [](int64_t workgroups) { return (workgroups + 255) / 256; };
    Wide best = {0, 0, 8};
    int64_t least = best.cost * rounds((N + LINEAR_ROWS - 1) / LINEAR_ROWS * tokens);
    for (const Wide w : {Wide{1, 1, 12}, {2, 1, 15}, {1, 2, 17}, {2, 2, 20}, {4, 2, 30}}) {
        const int rows = 16 * WIDE_PARTS * w.row_waves;
        const int64_t time = w.cost * rounds((N + rows - 1) / rows * ((tokens + w.tiles - 1) / w.tiles));
        if (time < least) least = time, best = w;
    }
    return best;
}

}  // namespace fp4dev

// fp4_rotate.h - the norm and rotation of queries and keys: kernel arguments.
// Internal to libfp4.so.
#pragma once

#include <stdint.h>

namespace fp4dev {

// Rows [tokens, heads, head_dim] in and out (strides in elements), and the norm's
// weight [head_dim] or null.
struct HeadRows {
    const void *x;
    void *y;
    int64_t x_token, x_head, y_token, y_head;
    const void *weight;
    int32_t heads;
};

struct RotateArgs {
    HeadRows q, k;
    const double *frequencies;
    float eps;
    int32_t rotary;
    bool weight_f32;
};

}  // namespace fp4dev

// fp4_moe.h - a mixture of experts: limits and kernel arguments.  Internal to
// libfp4.so.
#pragma once

#include <stdint.h>

namespace fp4dev {

constexpr uint32_t FLAG_EXPERT_INDEX = 16;
constexpr int MOE_EXPERTS = 1024;  // experts of a layer, at most
constexpr int MOE_TOP_K = 32;      // experts of a token, at most

struct MoeWeights {
    const uint8_t *up_codes, *up_scales, *down_codes, *down_scales;
    const float *up_global, *down_global;
    int64_t hidden, inner;
    int32_t experts, global_stride;
};

}  // namespace fp4dev

// fp4_linear.hip - linear layers of few tokens with an FP4 weight and
// activations that keep their precision:
//
//   c_mn = s_g sum_b s_nb sum_{k in b} E2M1(code_nk) x_mk,
//
// s_g = 1 for MXFP4.  What it cannot do without is reading the weight once: a
// token's 2 N K operations are far below the MFMA's rate up to some 64 tokens.
#include "fp4_kernels.h"
#include "fp4_w4.h"

namespace fp4dev {
namespace {

struct LinearArgs {
    const void *x;
    const uint8_t *codes, *scales;  // packed: of the row tiles
    const float *s_g;
    void *c;
    int64_t M, N, K;
    int32_t row_tiles;
    bool out_bf16;
};

constexpr int LINEAR_ROWS = 32;  // weight rows of a workgroup

// A workgroup has 32 weight rows and up to 16 CT tokens; its waves take units of
// 256 K in turn, and add their sums in LDS in the order of the waves.
template <int FMT, bool X_F32, bool PACKED, int CT>
__global__ __launch_bounds__(1024) void linear_w4_kernel(LinearArgs A) {
    using XT = std::conditional_t<X_F32, float, uint16_t>;
    constexpr int NT = X_F32 ? 3 : 1;
    extern __shared__ f32x4_t sums[];  // [waves][2][CT][64]
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int waves = blockDim.x / WAVE;
    const int r = lane & 15, g = lane >> 4;
    const int tile = blockIdx.x % A.row_tiles;
    const int64_t m0 = (int64_t)(blockIdx.x / A.row_tiles) * (16 * CT);
    const int64_t n0 = (int64_t)tile * LINEAR_ROWS;

    W4Row<FMT> rows[2];
    const uint8_t *packed_codes = nullptr, *packed_scales = nullptr;
    if constexpr (PACKED) {
        packed_codes = A.codes + n0 * (A.K / 2);
        packed_scales = A.scales + n0 * (A.K / (FMT == 0 ? 32 : 16));
    } else {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            // rows past the last one read the last one's, for sums that are not stored
            const int64_t n = min(n0 + 16 * p + r, A.N - 1);
            rows[p] = {A.codes + n * (A.K / 2), A.scales + n * (A.K / (FMT == 0 ? 32 : 16))};
        }
    }
    const int stretch = PACKED ? packed_stretch(g) : g;
    const XT *x[CT];
    bool real[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
        real[t] = m0 + 16 * t + r < A.M;
        x[t] = (const XT *)A.x + (m0 + 16 * t + r) * A.K + 32 * stretch;
    }

    f32x4_t acc[2][CT] = {};
    uint32_t top[2] = {0, 0};
    const int64_t units = (A.K + W4_UNIT - 1) / W4_UNIT, full = A.K / W4_UNIT;
    for (int64_t u = wave; u < units; u += waves) {
        W4Unit<FMT> w[2];
        if constexpr (PACKED) {
            w4_load_packed<FMT>(packed_codes, packed_scales, u, lane, w);
        } else if (u < full) {
#pragma unroll
            for (int p = 0; p < 2; ++p) w[p] = w4_load<FMT>(rows[p], u, g);
        } else {
#pragma unroll
            for (int p = 0; p < 2; ++p) w[p] = w4_load_tail<FMT>(rows[p], u, g, A.K);
        }
w4_multiply<FMT>(
            w,
            [&](int t, int k) {
                Terms<NT> b = {};
                if (real[t] && (PACKED || u * W4_UNIT + k + 32 * stretch < A.K))
                    b = load_terms(x[t] + u * W4_UNIT + k);
                return b;
            },
            acc, top);
    }
    if constexpr (FMT == 0) w4_nan_rows(top, acc);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int t = 0; t < CT; ++t) sums[((wave * 2 + p) * CT + t) * WAVE + lane] = acc[p][t];
    __syncthreads();
    const float s_g = FMT == 0 ? 1.0f : *A.s_g;
    for (int i = threadIdx.x; i < 2 * CT * WAVE; i += blockDim.x) {
        f32x4_t s = sums[i];
        for (int w = 1; w < waves; ++w) s += sums[w * 2 * CT * WAVE + i];
        const int p = i / (CT * WAVE), t = i / WAVE % CT, l = i % WAVE;
        const int64_t m = m0 + 16 * t + (l & 15), n = n0 + 16 * p + 4 * (l >> 4);
        if (m >= A.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (n + j >= A.N) break;
            const float y = FMT == 0 ? s[j] : s[j] * s_g;
            if (A.out_bf16) ((__bf16 *)A.c)[m * A.N + n + j] = (__bf16)y;
            else ((float *)A.c)[m * A.N + n + j] = y;
        }
    }
}

template <int FMT, bool X_F32, bool PACKED>
hipError_t launch_tokens(const LinearArgs &A, hipStream_t s) {
    const int ct = A.M <= 16 ? 1 : A.M <= 32 ? 2 : 4;
    const int64_t token_tiles = (A.M + 16 * ct - 1) / (16 * ct);
    const int waves = ct == 4 ? 8 : 16;
    const dim3 grid((uint32_t)(A.row_tiles * token_tiles)), block(waves * WAVE);
    const size_t lds = (size_t)waves * 2 * ct * WAVE * sizeof(f32x4_t);
    if (ct == 1) linear_w4_kernel<FMT, X_F32, PACKED, 1><<<grid, block, lds, s>>>(A);
    else if (ct == 2) linear_w4_kernel<FMT, X_F32, PACKED, 2><<<grid, block, lds, s>>>(A);
    else linear_w4_kernel<FMT, X_F32, PACKED, 4><<<grid, block, lds, s>>>(A);
    return hipGetLastError();
}

template <int FMT, bool PACKED>
hipError_t launch_types(const LinearArgs &A, bool x_bf16, hipStream_t s) {
    return x_bf16 ? launch_tokens<FMT, false, PACKED>(A, s) : launch_tokens<FMT, true, PACKED>(A, s);
}

}  // namespace

bool linear_w4_fits(int64_t M, int64_t N) {
    const int64_t rows = (N + LINEAR_ROWS - 1) / LINEAR_ROWS, tokens = (M + 15) / 16;
    return rows <= INT32_MAX / tokens;
}

hipError_t launch_linear_w4(int fmt, const void *x, bool x_bf16, int64_t M, int64_t K,
                            const uint8_t *codes, const uint8_t *scales, const float *s_g,
                            bool packed, int64_t N, void *c, bool out_bf16, hipStream_t s) {
    const int32_t row_tiles = (int32_t)((N + LINEAR_ROWS - 1) / LINEAR_ROWS);
    const LinearArgs A = {x, codes, scales, s_g, c, M, N, K, row_tiles, out_bf16};
    if (fmt == 0)
        return packed ? launch_types<0, true>(A, x_bf16, s)
                      : launch_types<0, false>(A, x_bf16, s);
    return packed ? launch_types<1, true>(A, x_bf16, s)
                  : launch_types<1, false>(A, x_bf16, s);
}

}  // namespace fp4dev

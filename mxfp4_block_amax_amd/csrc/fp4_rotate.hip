// fp4_rotate.hip - what lies between the projection of queries and keys and the
// cache: each head's norm, and the rotation by position.
//
//   z = x / sqrt(mean x^2 + eps) * w            (without w: z = x)
//   (y_a, y_b) = (z_a c - z_b s, z_a s + z_b c),  c, s = cos, sin (position f_i)
//
// for the pairs i of the first `rotary` values of a head: (i, i + rotary / 2), or
// (2 i, 2 i + 1) interleaved; the others are y = z.  Sums and rotations are fp32,
// rounded once; a head's squares may be past fp32's range.  Angles are 64-bit: at
// position 10^6 an angle of 32 bits is off by some 0.06.  Bound by memory on prompts, by
// a launch on single tokens.
#include <type_traits>

#include "fp4_kernels.h"
#include "fp4_kv.h"
#include "fp4_rotate.h"

namespace fp4dev {
namespace {

constexpr int ROTATE_WAVES = 4;

// cos and sin of pos f, f in radians: whole turns are taken off exactly enough
// that what is left is good to 2^-50 turns.
__device__ __forceinline__ float2 cos_sin(int64_t pos, double f) {
    constexpr double kTurn = 0x1.45f306dc9c883p-3;     // 1 / (2 pi)
    constexpr double kTurnLow = -0x1.6b01ec5417056p-57;  // and the rest of it
    const double p = (double)pos * f, p_low = __builtin_fma((double)pos, f, -p);
    const double t = p * kTurn;
    const double t_low = __builtin_fma(p, kTurn, -t) + (p * kTurnLow + p_low * kTurn);
    double s, c;
    sincospi(2.0 * ((t - __builtin_rint(t)) + t_low), &s, &c);
    return make_float2((float)c, (float)s);
}

struct Eight {
    float v[8];
};

template <bool F32>
__device__ __forceinline__ Eight load_eight(const void *p, int64_t at) {
    Eight r;
    if constexpr (F32) {
        const uint4 *q = (const uint4 *)((const float *)p + at);
        widen_f32x8(q[0], q[1], r.v);
    } else {
        widen_bf16x8(*(const uint4 *)((const uint16_t *)p + at), r.v);
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ void store_eight(void *p, int64_t at, const Eight &x) {
    if constexpr (F32) {
        uint4 *q = (uint4 *)((float *)p + at);
        q[0] = make_uint4(f2u(x.v[0]), f2u(x.v[1]), f2u(x.v[2]), f2u(x.v[3]));
        q[1] = make_uint4(f2u(x.v[4]), f2u(x.v[5]), f2u(x.v[6]), f2u(x.v[7]));
    } else {
        __bf16 b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = (__bf16)x.v[i];
        uint4 w;
        __builtin_memcpy(&w, b, sizeof(w));
        *(uint4 *)((uint16_t *)p + at) = w;
    }
}

// A head's sum over its D / 16 lanes, the same in each.
template <int LANES>
__device__ __forceinline__ float head_sum(float s, int base) {
    s += dppf<QP_XOR1>(s);
    s += dppf<QP_XOR2>(s);
    if constexpr (LANES == 12) {
        const float a = __shfl(s, base, WAVE), b = __shfl(s, base + 4, WAVE);
        return a + b + __shfl(s, base + 8, WAVE);
    }
    if constexpr (LANES >= 8) s += __shfl_xor(s, 4, WAVE);
    if constexpr (LANES >= 16) s += __shfl_xor(s, 8, WAVE);
    return s;
}

// And the largest of non-negative floats, by their bits.
template <int LANES>
__device__ __forceinline__ uint32_t head_max(uint32_t m, int base) {
    m = max(m, dpp<QP_XOR1>(m));
    m = max(m, dpp<QP_XOR2>(m));
    if constexpr (LANES == 12) {
        const uint32_t a = __shfl(m, base, WAVE), b = __shfl(m, base + 4, WAVE);
        return max(max(a, b), (uint32_t)__shfl(m, base + 8, WAVE));
    }
    if constexpr (LANES >= 8) m = max(m, (uint32_t)__shfl_xor(m, 4, WAVE));
    if constexpr (LANES >= 16) m = max(m, (uint32_t)__shfl_xor(m, 8, WAVE));
    return m;
}

__device__ __forceinline__ float sum_of_squares(const Eight &a, const Eight &b) {
    float s = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        s = __builtin_fmaf(a.v[i], a.v[i], __builtin_fmaf(b.v[i], b.v[i], s));
    return s;
}

// A head whose squares fp32 does not hold, their mean below 2^-100 or infinite: scaled by
// the power of two that makes the largest of its values and sqrt(eps) 0.5 to 1, and eps by
// its square, so that values over the mean's root are what they were.  Returns 1 / root.
// Zeros and what is not finite stay as they are.
template <int D>
__device__ __forceinline__ float far_norm(Eight &a, Eight &b, float mean, float eps, int base) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        top = max(top, max(f2u(a.v[i]) & 0x7FFFFFFFu, f2u(b.v[i]) & 0x7FFFFFFFu));
    top = max(head_max<D / 16>(top, base), f2u(__builtin_sqrtf(eps)));
    if (top == 0 || top >= 0x7F800000u) return 1.0f / __builtin_sqrtf(mean);
    int e;
    (void)__builtin_frexpf(u2f(top), &e);
#pragma unroll
    for (int i = 0; i < 8; ++i) a.v[i] = ldexpf(a.v[i], -e), b.v[i] = ldexpf(b.v[i], -e);
    const float s = head_sum<D / 16>(sum_of_squares(a, b), base);
    return 1.0f / __builtin_sqrtf(s * (1.0f / D) + ldexpf(eps, -2 * e));
}

// A workgroup has a token and some of its heads, a wave 64 / (D / 16) heads at a
// time.  A lane has 16 values of a head, eight pairs: both halves of them, so that
// nothing is exchanged between lanes but a head's sum, and the pair's angles are
// eight in a row.  The workgroup computes the token's angles once, in LDS.  4 x 2048
// tokens of 32 + 8 heads of 128 take 36 us, 4.8 TB/s read and written; one token 3.4.
template <int D, bool F32, bool INTERLEAVED>
__global__ __launch_bounds__(ROTATE_WAVES *WAVE) void norm_rotate_kernel(RotateArgs A, KvBatch B,
                                                                        int32_t *status) {
    constexpr int LANES = D / 16, HEADS = WAVE / LANES;
    __shared__ float turn[D / 2][2];
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int64_t token = blockIdx.x;
    const int heads = A.q.heads + A.k.heads, groups = (heads + HEADS - 1) / HEADS;
    const int step = ROTATE_WAVES * gridDim.y;
    const int j = lane % LANES;
    const bool turned = 16 * j < A.rotary;
    // where the lane's two eights start
    const int at0 = !INTERLEAVED && turned ? 8 * j : 16 * j;
    const int at1 = !INTERLEAVED && turned ? A.rotary / 2 + 8 * j : 16 * j + 8;

    const Item it = find_item(B, (int)token, B.tokens, 1, 0, blockIdx.y == 0, status);
    const int64_t pos = (int64_t)it.length - it.count + it.piece;
    const bool none = it.seq >= B.seqs || it.count <= 0 || it.piece >= it.count || pos < 0;
    if (none && it.seq < B.seqs && threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
    for (int i = threadIdx.x; i < A.rotary / 2; i += ROTATE_WAVES * WAVE) {
        const float2 cs = cos_sin(none ? 0 : pos, A.frequencies[i]);
        turn[i][0] = cs.x;
        turn[i][1] = cs.y;
    }
    __syncthreads();
    for (int group = blockIdx.y * ROTATE_WAVES + wave; group < groups; group += step) {
        const int h = group * HEADS + lane / LANES;
        const bool real = lane < HEADS * LANES && h < heads;
        const bool is_q = h < A.q.heads;
        const int64_t head = is_q ? h : h - A.q.heads;
        const void *weight = is_q ? A.q.weight : A.k.weight;
        Eight a = {}, b = {};
        if (real && !none) {
            const void *x = is_q ? A.q.x : A.k.x;
            const int64_t at = token * (is_q ? A.q.x_token : A.k.x_token) +
                               head * (is_q ? A.q.x_head : A.k.x_head);
            a = load_eight<F32>(x, at + at0);
            b = load_eight<F32>(x, at + at1);
        }
        const int base = lane / LANES * LANES;
        const float s = head_sum<LANES>(sum_of_squares(a, b), base);
        if (real && weight != nullptr) {
            const float mean = s * (1.0f / D) + A.eps;
            // (all of a head's lanes go the same way)
            const float inv = __builtin_expect(mean >= 0x1p-100f && mean < __builtin_inff(), 1)
                                  ? 1.0f / __builtin_sqrtf(mean)
                                  : far_norm<D>(a, b, mean, A.eps, base);
            const Eight wa = A.weight_f32 ? load_eight<true>(weight, at0)
                                          : load_eight<false>(weight, at0);
            const Eight wb = A.weight_f32 ? load_eight<true>(weight, at1)
                                          : load_eight<false>(weight, at1);
#pragma unroll
            for (int i = 0; i < 8; ++i) a.v[i] = a.v[i] * inv * wa.v[i], b.v[i] = b.v[i] * inv * wb.v[i];
        }
        if (turned) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float c = turn[8 * j + i][0], n = turn[8 * j + i][1];
                float &u = !INTERLEAVED ? a.v[i] : i < 4 ? a.v[2 * i] : b.v[2 * i - 8];
                float &v = !INTERLEAVED ? b.v[i] : i < 4 ? a.v[2 * i + 1] : b.v[2 * i - 7];
                const float x = u, y = v;
                u = __builtin_fmaf(x, c, -(y * n));
                v = __builtin_fmaf(x, n, y * c);
            }
        }
        if (real) {
            void *y = is_q ? A.q.y : A.k.y;
            const int64_t at = token * (is_q ? A.q.y_token : A.k.y_token) +
                               head * (is_q ? A.q.y_head : A.k.y_head);
            if (none) a = {}, b = {};
            store_eight<F32>(y, at + at0, a);
            store_eight<F32>(y, at + at1, b);
        }
    }
}

template <int D, bool F32>
hipError_t launch_dim(const RotateArgs &A, const KvBatch &B, bool interleaved, int32_t *status,
                      hipStream_t s) {
    constexpr int HEADS = WAVE / (D / 16);
    const int groups = (A.q.heads + A.k.heads + HEADS - 1) / HEADS;
    const int all = (groups + ROTATE_WAVES - 1) / ROTATE_WAVES;
    // few tokens: a wave has one group of heads; many: it has several, with the
    // same angles
    const int64_t want = (1024 + B.tokens - 1) / B.tokens;
    const dim3 grid((uint32_t)B.tokens, (uint32_t)(want < all ? want : all));
    if (interleaved) norm_rotate_kernel<D, F32, true><<<grid, ROTATE_WAVES * WAVE, 0, s>>>(A, B, status);
    else norm_rotate_kernel<D, F32, false><<<grid, ROTATE_WAVES * WAVE, 0, s>>>(A, B, status);
    return hipGetLastError();
}

template <bool F32>
hipError_t launch_type(const RotateArgs &A, const KvBatch &B, int dim, bool interleaved,
                       int32_t *status, hipStream_t s) {
    switch (dim) {
        case 64: return launch_dim<64, F32>(A, B, interleaved, status, s);
        case 128: return launch_dim<128, F32>(A, B, interleaved, status, s);
        case 192: return launch_dim<192, F32>(A, B, interleaved, status, s);
        default: return launch_dim<256, F32>(A, B, interleaved, status, s);
    }
}

}  // namespace

hipError_t launch_norm_rotate(const RotateArgs &A, const int32_t *cu, const int32_t *lengths,
                              int32_t seqs, int32_t tokens, int dim, bool bf16, bool interleaved,
                              int32_t *status, hipStream_t s) {
    const KvBatch B = {cu, lengths, nullptr, 0, seqs, 0, tokens};
    return bf16 ? launch_type<false>(A, B, dim, interleaved, status, s)
                : launch_type<true>(A, B, dim, interleaved, status, s);
}

}  // namespace fp4dev

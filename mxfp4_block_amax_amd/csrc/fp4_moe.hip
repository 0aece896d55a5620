// fp4_moe.hip - a mixture of experts for few tokens: the router, and the gated
// products of the experts that it chooses, with FP4 weights.
//
// Router: l_te = sum_h x_th r_eh, the top_k largest of a token (the lower id of
// equal ones), weights exp(l) over the sum of exp(l) of the chosen or of all.
// Experts: out_t = sum_j w_tj Down_e (silu(Gate_e x_t) * (Up_e x_t)), e = e_tj.
//
// What the experts cannot do without is reading the weights of those that some
// token goes to; that bounds them up to some 64 tokens.
#include "fp4_kernels.h"
#include "fp4_moe.h"
#include "fp4_w4.h"

namespace fp4dev {
namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void flag(int32_t *status, uint32_t bits) {
    if (status != nullptr) atomicOr(status, (int32_t)bits);
}

// ---- router -----------------------------------------------------------------
// Sums are 64-bit, so that which experts a token gets does not hang on their
// order: two logits of a token are seldom nearer than 2^-40 of their size.
struct Wide8 {
    float v[8];
};
__device__ __forceinline__ Wide8 load8(const uint16_t *p) {
    Wide8 r;
    widen_bf16x8(*(const uint4 *)p, r.v);
    return r;
}
__device__ __forceinline__ Wide8 load8(const float *p) {
    Wide8 r;
    widen_f32x8(((const uint4 *)p)[0], ((const uint4 *)p)[1], r.v);
    return r;
}

constexpr int ROUTE_WAVES = 4;

// A workgroup has 16 tokens, 16 experts and one of `splits` ranges of K, its
// waves 32 values of K at a time in turn; v_mfma_f64_16x16x4_f64 eight times on
// the eight values that a lane loads of its token and of its expert.
template <typename XT, typename RT>
__global__ __launch_bounds__(ROUTE_WAVES *WAVE) void route_logits_kernel(
    const XT *x, const RT *router, double *logits, int64_t tokens, int64_t hidden, int experts,
    int expert_tiles, int splits) {
    __shared__ f64x4_t sums[ROUTE_WAVES][WAVE];
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int r = lane & 15, g = lane >> 4;
    const int tile = blockIdx.x % expert_tiles, split = blockIdx.x / expert_tiles % splits;
    const int64_t t0 = (int64_t)(blockIdx.x / (expert_tiles * splits)) * 16;
    const int e0 = tile * 16;
    const XT *xr = x + min(t0 + r, tokens - 1) * hidden;
    const RT *rr = router + (int64_t)min(e0 + r, experts - 1) * hidden;
    f64x4_t acc = {0, 0, 0, 0};
    for (int64_t k = 32 * (split * ROUTE_WAVES + wave); k < hidden; k += 32 * ROUTE_WAVES * splits) {
        Wide8 a = {}, b = {};
        if (k + 8 * g < hidden) {
            a = load8(xr + k + 8 * g);
            b = load8(rr + k + 8 * g);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)a.v[i], (double)b.v[i], acc, 0, 0, 0);
    }
    sums[wave][lane] = acc;
    __syncthreads();
    // a lane's sums: expert r, tokens g + 4 i
    for (int i = threadIdx.x; i < 256; i += ROUTE_WAVES * WAVE) {
        const int l = i & (WAVE - 1), j = i / WAVE;
        double s = sums[0][l][j];
#pragma unroll
        for (int w = 1; w < ROUTE_WAVES; ++w) s += sums[w][l][j];
        const int64_t t = t0 + (l >> 4) + 4 * j;
        const int e = e0 + (l & 15);
        if (t < tokens && e < experts) logits[(split * tokens + t) * experts + e] = s;
    }
}

// A wave has a token, a lane the experts lane + 64 i.
template <int PER_LANE>
__global__ __launch_bounds__(WAVE) void route_choose_kernel(const double *logits, int64_t tokens,
                                                            int experts, int splits, int top_k,
                                                            bool renormalize, int32_t *chosen,
                                                            float *weights) {
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    double v[PER_LANE];
    bool left[PER_LANE];
#pragma unroll
    for (int i = 0; i < PER_LANE; ++i) {
        const int e = lane + WAVE * i;
        left[i] = e < experts;
        v[i] = 0;
        if (!left[i]) continue;
        for (int s = 0; s < splits; ++s) v[i] += logits[(s * tokens + t) * experts + e];
    }
    double mine = 0, first = 0;  // slot `lane`'s logit, the largest
    int mine_e = 0;
    for (int j = 0; j < top_k; ++j) {
        // a lane's best; a NaN is below all others, and no expert (none left) below that
        double best = 0;
        int best_e = -1;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            if (!left[i]) continue;
            if (best_e < 0 || v[i] > best || (best != best && v[i] == v[i])) {
                best = v[i];
                best_e = lane + WAVE * i;
            }
        }
        for (int off = 1; off < WAVE; off <<= 1) {
            const double other = __shfl_xor(best, off, WAVE);
            const int other_e = __shfl_xor(best_e, off, WAVE);
            if (other_e < 0) continue;
            const bool on = other == other, bn = best == best;
            const bool better = best_e < 0 || (on && !bn) || other > best ||
                                ((other == best || (!on && !bn)) && other_e < best_e);
            if (better) best = other, best_e = other_e;
        }
        if (j == 0) first = best;
        if (lane == j) mine = best, mine_e = best_e;
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i)
            if (best_e == lane + WAVE * i) left[i] = false;
    }
    const double p = lane < top_k ? exp(mine - first) : 0.0;
    double sum = 0;
    if (renormalize) {
        sum = p;
    } else {
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i)
            if (lane + WAVE * i < experts) sum += exp(v[i] - first);
    }
    for (int off = 1; off < WAVE; off <<= 1) sum += __shfl_xor(sum, off, WAVE);
    if (lane < top_k) {
        chosen[t * top_k + lane] = mine_e;
        weights[t * top_k + lane] = (float)(p / sum);
    }
}

// ---- experts ----------------------------------------------------------------
constexpr int MOE_BLOCK = 64;  // tokens that share a reading of the weights

struct MoeArgs {
    const void *x;
    const int32_t *ids;
    const float *weights;
    MoeWeights W;
    uint16_t *act;  // [tokens, top_k][terms][inner] bf16
    void *out;
    int64_t tokens;
    int32_t top_k, slots;
    bool out_bf16;
};

// The slots of expert e among a block's tokens, tokens ascending; a token that
// names it twice has it once, in its first slot.  Called by one wave.
__device__ __forceinline__ int expert_pairs(const int32_t *ids, int pairs, int top_k, int e,
                                            uint16_t *list) {
    const int lane = threadIdx.x & (WAVE - 1);
    int n = 0;
    for (int base = 0; base < pairs; base += WAVE) {
        const int p = base + lane;
        bool has = p < pairs && ids[p] == e;
        if (has)
            for (int q = p / top_k * top_k; q < p; ++q) has = has && ids[q] != e;
        const uint64_t b = __ballot(has);
        if (has) list[n + __builtin_popcountll(b & ((1ull << lane) - 1))] = (uint16_t)p;
        n += __builtin_popcountll(b);
    }
    return n;
}

// A value as N bf16 terms: each the nearest to what the ones before left.
template <int N>
__device__ __forceinline__ void store_terms(uint16_t *p, int64_t stride, float v) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const __bf16 b = (__bf16)v;
        p[k * stride] = __builtin_bit_cast(uint16_t, b);
        const float rest = v - (float)b;
        v = __builtin_fabsf((float)b) < __builtin_inff() ? rest : 0.0f;
    }
}

constexpr int UP_WAVES = 8;

// Gate and up: a workgroup has 16 rows of each of one expert and the tokens of a
// block that go there, 16 CT of them at a time; its waves share K = hidden.
template <int FMT, bool X_F32, int CT>
__global__ __launch_bounds__(UP_WAVES *WAVE) void moe_up_kernel(MoeArgs A, int32_t *status) {
    using XT = std::conditional_t<X_F32, float, uint16_t>;
    constexpr int NT = X_F32 ? 3 : 1, NA = X_F32 ? 3 : 2;
    constexpr int BLK = FMT == 0 ? 32 : 16;
    __shared__ f32x4_t sums[UP_WAVES][2][CT][WAVE];
    __shared__ uint16_t list[MOE_BLOCK];
    __shared__ int count;
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int r = lane & 15, g = lane >> 4;
    const int64_t token0 = (int64_t)blockIdx.z * MOE_BLOCK;
    const int block = (int)min((int64_t)MOE_BLOCK, A.tokens - token0);
    const int pairs = block * A.top_k;
    const int32_t *ids = A.ids + token0 * A.top_k;
    // the workgroup's expert: one each, or one for every slot (its first of an expert)
    int e = blockIdx.y;
    if (A.slots) {
        if (e >= pairs) return;
        const int slot = e;
        e = ids[slot];
        if (e < 0 || e >= A.W.experts) {
            if (e != -1 && threadIdx.x == 0) flag(status, FLAG_EXPERT_INDEX);
            return;
        }
        bool earlier = false;
        for (int p = threadIdx.x; p < slot; p += UP_WAVES * WAVE) earlier = earlier || ids[p] == e;
        if (__syncthreads_or(earlier)) return;
    } else if (blockIdx.x == 0 && e == 0) {
        for (int p = threadIdx.x; p < pairs; p += UP_WAVES * WAVE)
            if (ids[p] < -1 || ids[p] >= A.W.experts) flag(status, FLAG_EXPERT_INDEX);
    }
    if (wave == 0) {
        const int n = expert_pairs(ids, pairs, A.top_k, e, list);
        if (lane == 0) count = n;
    }
    __syncthreads();
    const int n = count;
    if (n == 0) return;

    const int64_t K = A.W.hidden, inner = A.W.inner;
    const int64_t row0 = (int64_t)blockIdx.x * 16;
    W4Row<FMT> rows[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
        const int64_t row = ((int64_t)e * 2 + p) * inner + row0 + r;
        rows[p] = {A.W.up_codes + row * (K / 2), A.W.up_scales + row * (K / BLK)};
    }
    const float s_g = FMT == 0 ? 1.0f : A.W.up_global[(int64_t)e * A.W.global_stride];
    const int64_t units = (K + W4_UNIT - 1) / W4_UNIT, full = K / W4_UNIT;
    for (int c0 = 0; c0 < n; c0 += 16 * CT) {
        const XT *x[CT];
        bool real[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            real[t] = c0 + 16 * t + r < n;
            const int64_t token = token0 + (real[t] ? list[c0 + 16 * t + r] / A.top_k : 0);
            x[t] = (const XT *)A.x + token * K + 32 * g;
        }
        f32x4_t acc[2][CT] = {};
        uint32_t top[2] = {0, 0};
        for (int64_t u = wave; u < units; u += UP_WAVES) {
            W4Unit<FMT> w[2];
#pragma unroll
            for (int p = 0; p < 2; ++p)
                w[p] = u < full ? w4_load<FMT>(rows[p], u, g) : w4_load_tail<FMT>(rows[p], u, g, K);
            w4_multiply<FMT>(
                w,
                [&](int t, int k) {
                    Terms<NT> b = {};
                    if (real[t] && u * W4_UNIT + k + 32 * g < K) b = load_terms(x[t] + u * W4_UNIT + k);
                    return b;
                },
                acc, top);
        }
        if constexpr (FMT == 0) w4_nan_rows(top, acc);
        if (c0 > 0) __syncthreads();
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int t = 0; t < CT; ++t) sums[wave][p][t][lane] = acc[p][t];
        __syncthreads();
        for (int i = threadIdx.x; i < CT * WAVE; i += UP_WAVES * WAVE) {
            const int t = i / WAVE, l = i & (WAVE - 1);
            if (c0 + 16 * t + (l & 15) >= n) continue;
            f32x4_t gate = sums[0][0][t][l], up = sums[0][1][t][l];
#pragma unroll
            for (int w = 1; w < UP_WAVES; ++w) gate += sums[w][0][t][l], up += sums[w][1][t][l];
            const int64_t pair = token0 * A.top_k + list[c0 + 16 * t + (l & 15)];
            uint16_t *a = A.act + pair * NA * inner + row0 + 4 * (l >> 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float gj = gate[j] * s_g, uj = up[j] * s_g;
                store_terms<NA>(a + j, inner, gj / (1.0f + expf(-gj)) * uj);
            }
        }
    }
}

constexpr int DOWN_WAVES = 16;
constexpr int MOE_IDS = MOE_BLOCK * MOE_TOP_K;

// Down and the weighted sum: a workgroup has 16 rows of every expert that a
// block's tokens go to; its waves share the experts' K = inner, one after the
// other, and keep the tokens' sums over the experts.  A token that an expert does
// not have takes nothing of it, not a zero times its values.
template <int FMT, bool X_F32, int CT>
__global__ __launch_bounds__(DOWN_WAVES *WAVE) void moe_down_kernel(MoeArgs A) {
    constexpr int NA = X_F32 ? 3 : 2;
    constexpr int BLK = FMT == 0 ? 32 : 16;
    __shared__ union {
        struct {
            int32_t ids[MOE_IDS];
            uint32_t seen[MOE_EXPERTS / 32];
            uint16_t active[MOE_EXPERTS];
        } plan;
        f32x4_t sums[DOWN_WAVES][CT][WAVE];
    } sh;
    __shared__ int count;
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int r = lane & 15, g = lane >> 4;
    const int64_t token0 = (int64_t)blockIdx.y * (16 * CT);
    const int block = (int)min((int64_t)(16 * CT), A.tokens - token0);
    const int pairs = block * A.top_k;
    const int64_t K = A.W.inner, hidden = A.W.hidden;
    const int64_t row0 = (int64_t)blockIdx.x * 16;

    for (int i = threadIdx.x; i < MOE_EXPERTS / 32; i += DOWN_WAVES * WAVE) sh.plan.seen[i] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += DOWN_WAVES * WAVE) {
        const int e = A.ids[token0 * A.top_k + p];
        sh.plan.ids[p] = e;
        if (e >= 0 && e < A.W.experts) atomicOr(&sh.plan.seen[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (wave == 0) {
        // experts ascending: a lane has 32 of them, one word
        static_assert(MOE_EXPERTS / 32 <= WAVE, "a word a lane");
        uint32_t word = lane < MOE_EXPERTS / 32 ? sh.plan.seen[lane] : 0;
        int before = __builtin_popcount(word), all = before;
        for (int off = 1; off < WAVE; off <<= 1) {
            const int below = __shfl_up(all, off, WAVE);
            if (lane >= off) all += below;
        }
        before = all - before;
        for (; word; word &= word - 1) sh.plan.active[before++] = 32 * lane + __builtin_ctz(word);
        if (lane == WAVE - 1) count = all;
    }
    __syncthreads();

    const int per = (int)((K + W4_UNIT - 1) / W4_UNIT), full = (int)(K / W4_UNIT);
    const int64_t units = (int64_t)count * per;
    int64_t u = units * wave / DOWN_WAVES;
    const int64_t end = units * (wave + 1) / DOWN_WAVES;
    f32x4_t out[CT] = {};
    while (u < end) {
        const int at = (int)(u / per);
        const int e = __builtin_amdgcn_readfirstlane(sh.plan.active[at]);
        int v = (int)(u - (int64_t)at * per);
        const int v_end = (int)min((int64_t)per, v + end - u);
        u += v_end - v;
        // the lane's tokens' slots of this expert and their weight
        const uint16_t *a[CT];
        float share[CT];
        bool real[CT];
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            real[t] = false;
            share[t] = 0;
            a[t] = A.act;
            const int token = 16 * t + r;
            if (token >= block) continue;
            for (int j = A.top_k - 1; j >= 0; --j) {
                if (sh.plan.ids[token * A.top_k + j] != e) continue;
                const int64_t pair = (token0 + token) * A.top_k + j;
                real[t] = true;
                share[t] += A.weights[pair];
                a[t] = A.act + pair * NA * K + 32 * g;
            }
        }
        const int64_t row = (int64_t)e * hidden + row0 + r;
        const W4Row<FMT> rows = {A.W.down_codes + row * (K / 2), A.W.down_scales + row * (K / BLK)};
        f32x4_t acc[1][CT] = {};
        uint32_t top[1] = {0};
        for (; v < v_end; ++v) {
            W4Unit<FMT> w[1];
            w[0] = v < full ? w4_load<FMT>(rows, v, g) : w4_load_tail<FMT>(rows, v, g, K);
            w4_multiply<FMT>(
                w,
                [&](int t, int k) {
                    Terms<NA> b = {};
                    if (real[t] && v * W4_UNIT + k + 32 * g < K) {
#pragma unroll
                        for (int m = 0; m < NA; ++m)
                            b.p[m] = load_terms(a[t] + m * K + v * W4_UNIT + k).p[0];
                    }
                    return b;
                },
                acc, top);
        }
        if constexpr (FMT == 0) w4_nan_rows(top, acc);
        const float s_g = FMT == 0 ? 1.0f : A.W.down_global[(int64_t)e * A.W.global_stride];
#pragma unroll
        for (int t = 0; t < CT; ++t)
            if (real[t]) out[t] += acc[0][t] * (share[t] * s_g);
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < CT; ++t) sh.sums[wave][t][lane] = out[t];
    __syncthreads();
    for (int i = threadIdx.x; i < CT * WAVE; i += DOWN_WAVES * WAVE) {
        const int t = i / WAVE, l = i & (WAVE - 1), token = 16 * t + (l & 15);
        if (token >= block) continue;
        f32x4_t s = sh.sums[0][t][l];
#pragma unroll
        for (int w = 1; w < DOWN_WAVES; ++w) s += sh.sums[w][t][l];
        const int64_t at = (token0 + token) * hidden + row0 + 4 * (l >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (A.out_bf16) ((__bf16 *)A.out)[at + j] = (__bf16)s[j];
            else ((float *)A.out)[at + j] = s[j];
        }
    }
}

template <int FMT, bool X_F32>
hipError_t launch_experts(MoeArgs A, int32_t *status, hipStream_t s) {
    const int block = (int)(A.tokens < MOE_BLOCK ? A.tokens : MOE_BLOCK);
    A.slots = (int64_t)block * A.top_k < A.W.experts;
    const dim3 up((uint32_t)(A.W.inner / 16), (uint32_t)(A.slots ? block * A.top_k : A.W.experts),
                  (uint32_t)((A.tokens + MOE_BLOCK - 1) / MOE_BLOCK));
    if (block <= 16) moe_up_kernel<FMT, X_F32, 1><<<up, UP_WAVES * WAVE, 0, s>>>(A, status);
    else moe_up_kernel<FMT, X_F32, 4><<<up, UP_WAVES * WAVE, 0, s>>>(A, status);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int ct = block <= 16 ? 1 : 4;
    const dim3 down((uint32_t)(A.W.hidden / 16), (uint32_t)((A.tokens + 16 * ct - 1) / (16 * ct)));
    if (ct == 1) moe_down_kernel<FMT, X_F32, 1><<<down, DOWN_WAVES * WAVE, 0, s>>>(A);
    else moe_down_kernel<FMT, X_F32, 4><<<down, DOWN_WAVES * WAVE, 0, s>>>(A);
    return hipGetLastError();
}

int route_splits(int64_t tokens, int64_t hidden, int experts) {
    const int64_t tiles = (tokens + 15) / 16 * ((experts + 15) / 16);
    const int64_t most = (hidden + 32 * ROUTE_WAVES - 1) / (32 * ROUTE_WAVES);
    int64_t splits = (256 + tiles - 1) / tiles;
    if (splits > 16) splits = 16;
    return (int)(splits < most ? splits : most);
}

template <typename XT, typename RT>
hipError_t launch_logits(const void *x, const void *router, double *logits, int64_t tokens,
                         int64_t hidden, int experts, int splits, hipStream_t s) {
    const int expert_tiles = (experts + 15) / 16;
    const int64_t groups = (tokens + 15) / 16 * expert_tiles * splits;
    route_logits_kernel<XT, RT><<<(uint32_t)groups, ROUTE_WAVES * WAVE, 0, s>>>(
        (const XT *)x, (const RT *)router, logits, tokens, hidden, experts, expert_tiles, splits);
    return hipGetLastError();
}

}  // namespace

size_t route_workspace_bytes(int64_t tokens, int64_t hidden, int experts) {
    return (size_t)route_splits(tokens, hidden, experts) * tokens * experts * sizeof(double);
}

hipError_t launch_route(const void *x, bool x_bf16, int64_t tokens, int64_t hidden,
                        const void *router, bool router_bf16, int experts, int top_k,
                        bool renormalize, int32_t *chosen, float *weights, void *workspace,
                        hipStream_t s) {
    double *logits = (double *)workspace;
    const int splits = route_splits(tokens, hidden, experts);
    hipError_t e;
    if (x_bf16)
        e = router_bf16 ? launch_logits<uint16_t, uint16_t>(x, router, logits, tokens, hidden,
                                                            experts, splits, s)
                        : launch_logits<uint16_t, float>(x, router, logits, tokens, hidden, experts,
                                                         splits, s);
    else
        e = router_bf16 ? launch_logits<float, uint16_t>(x, router, logits, tokens, hidden, experts,
                                                         splits, s)
                        : launch_logits<float, float>(x, router, logits, tokens, hidden, experts,
                                                      splits, s);
    if (e != hipSuccess) return e;
    const dim3 grid((uint32_t)tokens);
    if (experts <= WAVE)
        route_choose_kernel<1><<<grid, WAVE, 0, s>>>(logits, tokens, experts, splits, top_k,
                                                     renormalize, chosen, weights);
    else if (experts <= 4 * WAVE)
        route_choose_kernel<4><<<grid, WAVE, 0, s>>>(logits, tokens, experts, splits, top_k,
                                                     renormalize, chosen, weights);
    else
        route_choose_kernel<16><<<grid, WAVE, 0, s>>>(logits, tokens, experts, splits, top_k,
                                                      renormalize, chosen, weights);
    return hipGetLastError();
}

size_t experts_workspace_bytes(int64_t tokens, int top_k, int64_t inner, bool x_bf16) {
    return (size_t)tokens * top_k * (x_bf16 ? 2 : 3) * inner * sizeof(uint16_t);
}

hipError_t launch_experts(int fmt, const MoeWeights &W, const void *x, bool x_bf16, int64_t tokens,
                          const int32_t *ids, const float *weights, int top_k, void *out,
                          bool out_bf16, void *workspace, int32_t *status, hipStream_t s) {
    const MoeArgs A = {x, ids, weights, W, (uint16_t *)workspace, out, tokens, top_k, 0, out_bf16};
    if (fmt == 0)
        return x_bf16 ? launch_experts<0, false>(A, status, s) : launch_experts<0, true>(A, status, s);
    return x_bf16 ? launch_experts<1, false>(A, status, s) : launch_experts<1, true>(A, status, s);
}

}  // namespace fp4dev

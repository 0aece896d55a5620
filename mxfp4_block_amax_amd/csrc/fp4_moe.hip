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

// A workgroup has 16 tokens, 16 experts and one of `splits` shares of K, its
// waves 32 values of K at a time in turn; v_mfma_f64_16x16x4_f64 eight times on
// the eight values that a lane loads of its token and of its expert.
template <typename XT, typename RT, int WAVES>
__global__ __launch_bounds__(WAVES *WAVE) void route_logits_kernel(
    const XT *x, const RT *router, double *logits, int64_t tokens, int64_t hidden, int experts,
    int expert_tiles, int splits) {
    __shared__ f64x4_t sums[WAVES][WAVE];
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int r = lane & 15, g = lane >> 4;
    const int tile = blockIdx.x % expert_tiles, split = blockIdx.x / expert_tiles % splits;
    const int64_t t0 = (int64_t)(blockIdx.x / (expert_tiles * splits)) * 16;
    const int e0 = tile * 16;
    const XT *xr = x + min(t0 + r, tokens - 1) * hidden;
    const RT *rr = router + (int64_t)min(e0 + r, experts - 1) * hidden;
    f64x4_t acc = {0, 0, 0, 0};
    const int h = (int)hidden, step = 32 * WAVES * splits;
    const auto load = [&](int k, Wide8 &a, Wide8 &b) {
        a = {}, b = {};
        if (k < h) {
            a = load8(xr + k);
            b = load8(rr + k);
        }
    };
    Wide8 a, b;
    int k = 32 * (split * WAVES + wave) + 8 * g;
    load(k, a, b);
    for (; k - 8 * g < h; k += step) {
        Wide8 a2, b2;
        load(k + step, a2, b2);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc = __builtin_amdgcn_mfma_f64_16x16x4f64((double)a.v[i], (double)b.v[i], acc, 0, 0, 0);
        a = a2, b = b2;
    }
    sums[wave][lane] = acc;
    __syncthreads();
    // a lane's sums: expert r, tokens g + 4 i
    for (int i = threadIdx.x; i < 256; i += WAVES * WAVE) {
        const int l = i & (WAVE - 1), j = i / WAVE;
        double s = sums[0][l][j];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) s += sums[w][l][j];
        const int64_t t = t0 + (l >> 4) + 4 * j;
        const int e = e0 + (l & 15);
        if (t < tokens && e < experts) logits[(split * tokens + t) * experts + e] = s;
    }
}

// A workgroup has a token, a thread an expert: its place is the number of experts
// before it, which a thread counts by itself, so that the time does not grow with top_k
// (a maximum over the wave for every place took 7 us for 4 of 64, 14 for 8 of 256).
__global__ __launch_bounds__(MOE_EXPERTS) void route_choose_kernel(const double *logits,
                                                                  int64_t tokens, int experts,
                                                                  int splits, int top_k,
                                                                  bool renormalize, int32_t *chosen,
                                                                  float *weights) {
    // keys that order as logits do, a NaN below all others; those of no expert below that
    __shared__ alignas(16) uint64_t keys[MOE_EXPERTS];
    __shared__ double places[MOE_TOP_K], sums[MOE_EXPERTS / WAVE];
    const int64_t t = blockIdx.x;
    const int e = threadIdx.x, lane = e & (WAVE - 1);
    double v = 0;
    if (e < experts) {
        const double *p = logits + t * experts + e;
        for (int s = 0; s < splits; s += 4) {
            double part[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) part[i] = s + i < splits ? p[(s + i) * tokens * experts] : 0.0;
#pragma unroll
            for (int i = 0; i < 4; ++i) v += part[i];
        }
    }
    const uint64_t bits = (uint64_t)__double_as_longlong(v == 0 ? 0.0 : v);  // -0 equals 0
    uint64_t key = bits >> 63 ? ~bits : bits | 1ull << 63;
    if (v != v) key = 1;
    if (e >= experts) key = 0;
    keys[e] = key;
    __syncthreads();
    // before e: greater keys, and equal ones of lower ids: all equal ones of the waves
    // before its own, none of those after
    int place = 0;
    const int own = __builtin_amdgcn_readfirstlane(e & ~(WAVE - 1));
#pragma unroll 16
    for (int j = 0; j < own; ++j) place += keys[j] >= key ? 1 : 0;
#pragma unroll 16
    for (int j = 0; j < WAVE; ++j) {
        const uint64_t other = keys[own + j];
        place += (j < lane ? other >= key : other > key) ? 1 : 0;
    }
#pragma unroll 16
    for (int j = own + WAVE; j < (int)blockDim.x; ++j) place += keys[j] > key ? 1 : 0;
    const bool mine = e < experts && place < top_k;
    if (mine) places[place] = v;
    __syncthreads();
    const double first = places[0];
    double p = 0;
    if (mine || (!renormalize && e < experts)) p = exp(v - first);
    // the sum in a fixed order: of the places, or over lanes and then waves
    double sum = 0;
    if (renormalize) {
        __syncthreads();
        if (mine) places[place] = p;
        __syncthreads();
        if (mine)
            for (int j = 0; j < top_k; ++j) sum += places[j];
    } else {
        double part = p;
        for (int off = 1; off < WAVE; off <<= 1) part += __shfl_xor(part, off, WAVE);
        if (lane == 0) sums[e / WAVE] = part;
        __syncthreads();
        if (mine)
            for (int w = 0; w < (int)blockDim.x / WAVE; ++w) sum += sums[w];
    }
    if (mine) {
        chosen[t * top_k + place] = e;
        weights[t * top_k + place] = (float)(p / sum);
    }
}

// ---- experts ----------------------------------------------------------------
constexpr int MOE_BLOCK = 64;  // tokens that share a reading of the weights
constexpr size_t LDS_BYTES = 160 * 1024 - 256;  // of a workgroup, but for small fixed arrays

struct MoeArgs {
    const void *x;
    const int32_t *ids;
    const float *weights;
    MoeWeights W;
    void *act;       // the gated values, [tokens, top_k][Gated::PLANES][inner] Gated::Value
    float *partial;  // [splits][tokens][hidden], of a down product in splits
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

// The slots of slot p's token, of up to 64.
__device__ __forceinline__ uint64_t own_slots(int p, int top_k) {
    return ((1ull << top_k) - 1) << (p / top_k * top_k);
}

// The gated values between the products, all 24 bits of them: of bf16 activations in
// fp32, which the second product splits into three bf16 terms, of fp32 ones in these terms
// already (4 and 6 bytes a value).  (Two terms, 17 bits, showed: outputs in bf16 were 1.4e-4
// away from those of a product in 32 bits, now 5e-6, and outputs in fp32 had their error.)
// The terms are columns of the second product, so the third one costs no matrix
// instruction.  Next to two terms side by side: 16 tokens of 128 experts, 4096 x 1536, 172
// us and 170; 64 of 128, 2048 x 768, 150 and 140; 32 of 64, 1408 in NVFP4, 119 and 121; 64
// of 8, 2816, 88 and 83: the splitting, by every workgroup.
template <bool X_F32, int TOKENS>
struct Gated {
    using X = std::conditional_t<X_F32, XPart<false, TOKENS, 3, true>, XPart<true, TOKENS, 1, true>>;
    using Value = std::conditional_t<X_F32, uint16_t, float>;
    static constexpr int PLANES = X_F32 ? 3 : 1;
};

__device__ __forceinline__ void store_gated(float *p, int64_t, const float (&v)[4]) {
    *(f32x4_t *)p = {v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store_gated(uint16_t *p, int64_t plane, const float (&v)[4]) {
    u32x2_t t[3];
    split_f32x4(v, t);
#pragma unroll
    for (int n = 0; n < 3; ++n) *(u32x2_t *)(p + n * plane) = t[n];
}

// The weights of what K has past its last whole group, stretch k of the rows row_of(part,
// the lane's row).
template <int FMT, int PARTS, typename RowOf>
__device__ __forceinline__ void load_tails(const uint8_t *codes, const uint8_t *scales, int k, int K,
                                           const RowOf &row_of, W4Unit (&w)[PARTS]) {
    constexpr int BLK = FMT == 0 ? 32 : 16;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        const int64_t row = row_of(p, threadIdx.x & 15);
        w[p] = load_tail<FMT>(codes + row * (K / 2), scales + row * (K / BLK), k, K);
    }
}

constexpr int UP_WAVES = 4;

// Gate and up: a workgroup has 16 rows of each of one expert and the tokens of a
// block that go there, up to TOKENS of them at a time; its waves share K = hidden (four:
// each has several groups, whose loads overlap; with more, 16 tokens of 128 experts, 4096 x
// 1536, took 30 us more).  The weights' bytes bound it: there 107 us, 5.1 TB/s.
template <int FMT, bool X_F32, int TOKENS>
__global__ __launch_bounds__(UP_WAVES *WAVE, TOKENS <= 4 ? 4 : 2) void moe_up_kernel(MoeArgs A,
                                                                                    int32_t *status) {
    using XT = std::conditional_t<X_F32, float, uint16_t>;
    using X = XPart<X_F32, TOKENS>;
    using W = RowsAt<FMT, 2>;
    using G = Gated<X_F32, TOKENS>;
    constexpr int BLK = FMT == 0 ? 32 : 16;
    extern __shared__ u32x4_t lds[];
    __shared__ uint16_t lists[UP_WAVES][MOE_BLOCK];
    __shared__ int count;
    const int lane = threadIdx.x & (WAVE - 1);
    // (waves as a constant: loops unrolled, and 16 tokens of 128 experts 195 us, not 169)
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), waves = blockDim.x / WAVE;
    const int r = lane & 15, g = lane >> 4;
    const int64_t token0 = (int64_t)blockIdx.z * MOE_BLOCK;
    const int block = (int)min((int64_t)MOE_BLOCK, A.tokens - token0);
    const int pairs = block * A.top_k;
    const int32_t *ids = A.ids + token0 * A.top_k;
    // the workgroup's expert: one each, or one for every slot (its first of an expert);
    // up to 64 pairs every wave looks at all of them by itself, in one load
    const bool few = pairs <= WAVE;
    int e = blockIdx.y;
    if (A.slots && e >= pairs) return;
    uint16_t *list = lists[few ? wave : 0];
    int n = 0;
    if (few) {
        const int id = lane < pairs ? ids[lane] : -1;
        if (A.slots) e = __builtin_amdgcn_readlane(id, blockIdx.y);
        if (blockIdx.x == 0 && wave == 0 && (A.slots || e == 0) &&
            __ballot(id < -1 || id >= A.W.experts) != 0 && lane == 0)
            flag(status, FLAG_EXPERT_INDEX);
        if (e < 0 || e >= A.W.experts) return;
        const uint64_t all = __ballot(id == e);
        if (A.slots && (all & ((1ull << blockIdx.y) - 1)) != 0) return;
        const uint64_t mine = all & own_slots(lane, A.top_k) & ((1ull << lane) - 1);
        const uint64_t firsts = __ballot((all >> lane & 1) != 0 && mine == 0);
        n = __builtin_popcountll(firsts);
        if (firsts >> lane & 1)
            list[__builtin_popcountll(firsts & ((1ull << lane) - 1))] = (uint16_t)lane;
        wave_order();
    } else {
        if (A.slots) {
            const int slot = e;
            e = ids[slot];
            if (e < 0 || e >= A.W.experts) {
                if (e != -1 && threadIdx.x == 0) flag(status, FLAG_EXPERT_INDEX);
                return;
            }
            bool earlier = false;
            for (int p = threadIdx.x; p < slot; p += blockDim.x) earlier = earlier || ids[p] == e;
            if (__syncthreads_or(earlier)) return;
        } else if (blockIdx.x == 0 && e == 0) {
            for (int p = threadIdx.x; p < pairs; p += blockDim.x)
                if (ids[p] < -1 || ids[p] >= A.W.experts) flag(status, FLAG_EXPERT_INDEX);
        }
        if (wave == 0) {
            const int found = expert_pairs(ids, pairs, A.top_k, e, list);
            if (lane == 0) count = found;
        }
        __syncthreads();
        n = __builtin_amdgcn_readfirstlane(count);
    }
    if (n == 0) return;

    const int K = (int)A.W.hidden, inner = (int)A.W.inner, row0 = blockIdx.x * 16;
    const int64_t base = (int64_t)e * 2 * inner + row0;
    const uint8_t *codes = A.W.up_codes + base * (K / 2), *scales = A.W.up_scales + base * (K / BLK);
    const XT *x0 = (const XT *)A.x + token0 * K;
    const Rsrc x = span(x0, block * K * (int)sizeof(XT));
    u32x4_t *mine = lds + wave * (X::PIECES + W::LDS);
    const W weights(codes, scales, inner + 16, inner, K, mine + X::PIECES);
    const float s_g = FMT == 0 ? 1.0f : A.W.up_global[(int64_t)e * A.W.global_stride];
    const int groups = K / W4_GROUP;
    for (int c0 = 0; c0 < n; c0 += TOKENS) {
        const int rows = min(n - c0, TOKENS);
        Group<W, X> a = {weights, 0, {}};
#pragma unroll
        for (int i = 0; i < X::LOADS; ++i) {
            const auto p = X::place(i);
            a.x_at[i] = p.row < rows ? (uint32_t)(list[c0 + p.row] / A.top_k * K + p.k) * (uint32_t)sizeof(XT)
                                     : NOWHERE;
        }
        f32x4_t acc[2][1] = {};
        uint32_t top[2] = {0, 0};
        multiply_groups<FMT, false, W, X>(
            [&](int q) {
                a.k = q * W4_GROUP;
                return a;
            },
            x, mine, wave, waves, groups, acc, top, [](int) {});
        const int t = (wave - groups % waves + waves) % waves;
        for (int k = groups * W4_GROUP + W4_STRETCH * t; k < K; k += W4_STRETCH * waves) {
            W4Unit w[2];
            load_tails<FMT>(codes, scales, k, K,
                            [&](int p, int row) { return (int64_t)p * inner + row; }, w);
            Terms<X::TERMS> b[4] = {};
            const int at = k + 32 * g;
            if (r < rows)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + 8 * i < K)
                        b[i] = load_terms(x0 + list[c0 + r] / A.top_k * (int64_t)K + at + 8 * i);
            w4_multiply<FMT, X::TERMS>(w, [&](int, int i, int n) { return b[i].p[n]; }, acc, top);
        }
        if constexpr (FMT == 0) w4_nan_rows(top, acc);
        __syncthreads();
        f32x4_t *sums = (f32x4_t *)lds;  // [waves][2][64]
#pragma unroll
        for (int p = 0; p < 2; ++p) sums[(wave * 2 + p) * WAVE + lane] = acc[p][0];
        __syncthreads();
        if (wave == 0 && r < rows) {
            f32x4_t gate = sums[lane], up = sums[WAVE + lane];
            for (int v = 1; v < waves; ++v) {
                gate += sums[v * 2 * WAVE + lane];
                up += sums[(v * 2 + 1) * WAVE + lane];
            }
            const int64_t pair = token0 * A.top_k + list[c0 + r];
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float gj = gate[j] * s_g, uj = up[j] * s_g;
                v[j] = gj / (1.0f + expf(-gj)) * uj;
            }
            store_gated((typename G::Value *)A.act + pair * G::PLANES * inner + row0 + 4 * g, inner, v);
        }
        __syncthreads();
    }
}

// What a block's tokens want, in LDS: its (token, expert) pairs sorted by expert, a
// token that names an expert twice once, in its first slot, with both weights; and
// items, an expert and up to TOKENS of its pairs each.
struct MoeItem {
    uint16_t expert, first, count, pad;
};
struct MoePlan {
    MoeItem *items;     // [pairs]
    float *share;       // [pairs]
    uint16_t *pair;     // [pairs]
    uint32_t *used;     // [experts]: pairs of an expert; later where its next one goes
    __host__ __device__ static size_t bytes(int pairs) {
        return ((size_t)pairs * (sizeof(MoeItem) + 4 + 2) + 15) / 16 * 16;
    }
    // scratch: 4 bytes an expert, until the plan is made
    __device__ MoePlan(void *p, int pairs, void *scratch)
        : items((MoeItem *)p), share((float *)(items + pairs)), pair((uint16_t *)(share + pairs)),
          used((uint32_t *)scratch) {}
};

// Tokens of an item, a pass over an expert's weights: 4, or 8 where a block's tokens go to
// an expert 4 times on average (64 tokens of 8 experts, top 2, through 2048 x 2816: 123 and
// 98 us; of 64, top 6, 1408 in NVFP4: 237 and 203; but 32 of 128, top 8, 768: 119 and 140).
// 16 win another tenth from 16 times on, and lose as much at 6.
constexpr bool dense(int pairs, int experts) { return pairs >= 4 * experts; }

// Waves of a workgroup of moe_down_kernel: 16, or 8 where more tokens take the LDS of two.
// The plan has a thread for each expert.
template <int TOKENS>
constexpr int DOWN_WAVES = TOKENS > 4 ? 8 : 16;
static_assert(DOWN_WAVES<4> * WAVE >= MOE_EXPERTS);
static_assert(!dense(MOE_BLOCK * MOE_TOP_K, DOWN_WAVES<8> * WAVE + 1));

// The plan of up to 64 pairs, by one wave, experts in the order they are named first:
// no barriers but the one after it (the other way took a third of the kernel's time for
// a single token).  Returns the items.
template <int TOKENS>
__device__ int make_small_plan(const MoePlan &plan, const int32_t *ids, const float *weights,
                               int pairs, int top_k, int experts) {
    const int lane = threadIdx.x & (WAVE - 1);
    const int e = lane < pairs ? ids[lane] : -1;
    const float w = lane < pairs ? weights[lane] : 0.0f;
    const uint64_t token = own_slots(lane, top_k), below = (1ull << lane) - 1;
    uint64_t left = __ballot(e >= 0 && e < experts);
    int items = 0, at = 0;
    while (left != 0) {
        const int expert = __builtin_amdgcn_readlane(e, __builtin_ctzll(left));
        const uint64_t all = __ballot(e == expert);
        left &= ~all;
        const bool first = (all >> lane & 1) != 0 && (all & token & below) == 0;
        const uint64_t firsts = __ballot(first);
        float share = w;
        if (firsts != all)
            for (int j = 1; j < top_k; ++j) {  // the token's other slots of this expert
                const int other = lane + j;
                const float more = __shfl(w, other & (WAVE - 1), WAVE);
                if (other < WAVE && (all & token) >> other & 1) share += more;
            }
        const int n = __builtin_popcountll(firsts);
        if (first) {
            const int place = at + __builtin_popcountll(firsts & below);
            plan.pair[place] = (uint16_t)lane;
            plan.share[place] = share;
        }
        for (int i = 0; i < n; i += TOKENS, ++items)
            if (lane == 0)
                plan.items[items] = {(uint16_t)expert, (uint16_t)(at + i),
                                     (uint16_t)min(n - i, TOKENS), 0};
        at += n;
    }
    return items;
}

// Returns the items.
template <int TOKENS>
__device__ int make_plan(const MoePlan &plan, const int32_t *ids, const float *weights, int pairs,
                         int top_k, int experts) {
    __shared__ uint32_t wave_sum[DOWN_WAVES<TOKENS>];
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE, me = threadIdx.x;
    if (me < experts) plan.used[me] = 0;
    __syncthreads();
    const auto first_of = [&](int p, int e) {
        for (int q = p / top_k * top_k; q < p; ++q)
            if (ids[q] == e) return false;
        return e >= 0 && e < experts;
    };
    for (int p = me; p < pairs; p += DOWN_WAVES<TOKENS> * WAVE) {
        const int e = ids[p];
        if (first_of(p, e)) atomicAdd(&plan.used[e], 1u);
    }
    __syncthreads();
    // pairs (low half) and items (high half) of the experts before: both below 2^16
    const uint32_t n = me < experts ? plan.used[me] : 0;
    const uint32_t own = n | (n + TOKENS - 1) / TOKENS << 16;
    uint32_t before = own;
    for (int off = 1; off < WAVE; off <<= 1) {
        const uint32_t below = __shfl_up(before, off, WAVE);
        if (lane >= off) before += below;
    }
    if (lane == WAVE - 1) wave_sum[wave] = before;
    before -= own;
    __syncthreads();
    uint32_t all = 0;
    for (int w = 0; w < DOWN_WAVES<TOKENS>; ++w) {
        if (w < wave) before += wave_sum[w];
        all += wave_sum[w];
    }
    const uint32_t start = before & 0xFFFFu, item = before >> 16;
    if (me < experts) {
        plan.used[me] = start;
        for (uint32_t i = 0; i * TOKENS < n; ++i)
            plan.items[item + i] = {(uint16_t)me, (uint16_t)(start + i * TOKENS),
                                    (uint16_t)min(n - i * TOKENS, (uint32_t)TOKENS), 0};
    }
    __syncthreads();
    for (int p = me; p < pairs; p += DOWN_WAVES<TOKENS> * WAVE) {
        const int e = ids[p];
        if (first_of(p, e)) plan.pair[atomicAdd(&plan.used[e], 1u)] = (uint16_t)p;
    }
    __syncthreads();
    // in order, whatever order the pairs came in, and each with its weights' sum
    if (me < experts && n > 0) {
        for (uint32_t i = 1; i < n; ++i) {
            const uint16_t p = plan.pair[start + i];
            uint32_t j = i;
            for (; j > 0 && plan.pair[start + j - 1] > p; --j) plan.pair[start + j] = plan.pair[start + j - 1];
            plan.pair[start + j] = p;
        }
        for (uint32_t i = 0; i < n; ++i) {
            const int p = plan.pair[start + i], end = (p / top_k + 1) * top_k;
            float s = weights[p];
            for (int q = p + 1; q < end; ++q)
                if (ids[q] == me) s += weights[q];
            plan.share[start + i] = s;
        }
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(all >> 16);
}

// Down and the weighted sum.  A workgroup has 16 rows and a block's tokens; its waves, or
// those of gridDim.z workgroups, go through the items' groups of K = inner in turn.  A
// wave adds each group's sums, weighted, to its own of the tokens, in LDS: a token that an
// expert does not have takes nothing of it, not a zero times its values, and no order of
// arrival changes a sum.  16 tokens of 128 experts, 4096 x 1536: 74 us, 3.7 TB/s, vector
// instructions 52 % of the cycles (half of them split the gated values), LDS busy for 46 %;
// one token of 64, 2048 x 768: 6.4 us of latency.
template <int FMT, bool X_F32, int TOKENS>
__global__ __launch_bounds__(DOWN_WAVES<TOKENS> *WAVE) void moe_down_kernel(MoeArgs A, int block_tokens) {
    using G = Gated<X_F32, TOKENS>;
    using X = typename G::X;
    using Value = typename G::Value;
    constexpr int PLANES = G::PLANES, BLK = FMT == 0 ? 32 : 16;
    using W = RowsAt<FMT, 1>;
    extern __shared__ u32x4_t lds[];
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int r = lane & 15, g = lane >> 4;
    const int64_t token0 = (int64_t)blockIdx.y * block_tokens;
    const int block = (int)min((int64_t)block_tokens, A.tokens - token0);
    const int pairs = block * A.top_k;
    const int K = (int)A.W.inner, hidden = (int)A.W.hidden, row0 = blockIdx.x * 16;
    f32x4_t *sums = (f32x4_t *)lds;  // [waves][tokens][4]: 16 rows
    u32x4_t *pieces = lds + DOWN_WAVES<TOKENS> * block_tokens * 4;  // the waves' own
    u32x4_t *mine = pieces + wave * (X::PIECES + W::LDS);
    static_assert(DOWN_WAVES<TOKENS> * X::PIECES * 16 >= MOE_EXPERTS * 4);
    const MoePlan plan(pieces + DOWN_WAVES<TOKENS> * (X::PIECES + W::LDS), block_tokens * A.top_k,
                       pieces);

    for (int i = threadIdx.x; i < DOWN_WAVES<TOKENS> * block_tokens * 4; i += DOWN_WAVES<TOKENS> * WAVE)
        sums[i] = {0, 0, 0, 0};
    const int32_t *ids = A.ids + token0 * A.top_k;
    const float *weights = A.weights + token0 * A.top_k;
    int items;
    if (pairs <= WAVE) {
        __shared__ int found;
        if (wave == 0) {
            const int n = make_small_plan<TOKENS>(plan, ids, weights, pairs, A.top_k, A.W.experts);
            if (lane == 0) found = n;
        }
        __syncthreads();
        items = __builtin_amdgcn_readfirstlane(found);
    } else {
        items = make_plan<TOKENS>(plan, ids, weights, pairs, A.top_k, A.W.experts);
    }

    const Value *act0 = (const Value *)A.act + token0 * A.top_k * PLANES * K;
    const Rsrc act = span(act0, pairs * PLANES * K * (int)sizeof(Value));
    const int per = K / W4_GROUP;
    const int splits = gridDim.z, step = splits * DOWN_WAVES<TOKENS>;
    const int turn = blockIdx.z * DOWN_WAVES<TOKENS> + wave;
    f32x4_t acc[1][X::TILES] = {};
    uint32_t top[1] = {0};
    // the sums of an item's products so far go to its tokens
    const auto add = [&](const MoeItem &it) {
        if constexpr (FMT == 0) w4_nan_rows(top, acc);
        const f32x4_t sum = X::sum_columns(acc[0]);
        if (r < it.count) {
            const float s_g = FMT == 0 ? 1.0f : A.W.down_global[(int64_t)it.expert * A.W.global_stride];
            f32x4_t *to = sums + (wave * block_tokens + plan.pair[it.first + r] / A.top_k) * 4 + g;
            *to += sum * (plan.share[it.first + r] * s_g);
        }
#pragma unroll
        for (int t = 0; t < X::TILES; ++t) acc[0][t] = {0, 0, 0, 0};
        top[0] = 0;
    };
    const auto item_of = [&](int i) {
        MoeItem it = plan.items[i];
        it.expert = __builtin_amdgcn_readfirstlane(it.expert);
        return it;
    };
    // where the lane's load i has an item's values, of the stretch at 0
    const auto x_at = [&](const MoeItem &it, int i) {
        const auto p = X::place(i);
        return p.row < it.count
                   ? (uint32_t)((plan.pair[it.first + p.row] * PLANES + p.plane) * K + p.k) *
                         (uint32_t)sizeof(Value)
                   : NOWHERE;
    };
    multiply_groups<FMT, false, W, X>(
        [&](int n) {
            const MoeItem it = item_of(n / per);
            const int64_t row = (int64_t)it.expert * hidden + row0;
            Group<W, X> a = {W(A.W.down_codes + row * (K / 2), A.W.down_scales + row * (K / BLK), 16, 16,
                               K, mine + X::PIECES),
                             (uint32_t)(n % per * W4_GROUP), {}};
#pragma unroll
            for (int i = 0; i < X::LOADS; ++i) a.x_at[i] = x_at(it, i);
            return a;
        },
        act, mine, turn, step, items * per, acc, top, [&](int n) { add(item_of(n / per)); });
    // and stretches past the last whole group, by the waves that have fewer groups
    const int rest = (K - per * W4_GROUP + W4_STRETCH - 1) / W4_STRETCH;
    for (int n = (turn - items * per % step + step) % step; n < items * rest; n += step) {
        const MoeItem it = item_of(n / rest);
        const int64_t row = (int64_t)it.expert * hidden + row0;
        const int k = per * W4_GROUP + n % rest * W4_STRETCH;
        W4Unit w[1];
        load_tails<FMT>(A.W.down_codes + row * (K / 2), A.W.down_scales + row * (K / BLK), k, K,
                        [](int, int rr) { return (int64_t)rr; }, w);
        X xs;
        uint32_t at[X::LOADS];
#pragma unroll
        for (int i = 0; i < X::LOADS; ++i) at[i] = k + X::place(i).k < K ? x_at(it, i) : NOWHERE;
        xs.load(act, at, k);
        wave_order();
        xs.store(mine);
        wave_order();
        w4_multiply<FMT, X::TERMS>(
            w, [&](int t, int i, int m) { return X::piece(mine, g, t, i, m); }, acc, top);
        add(it);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < block * 4; i += DOWN_WAVES<TOKENS> * WAVE) {
        f32x4_t s = sums[i];
        for (int w = 1; w < DOWN_WAVES<TOKENS>; ++w) s += sums[w * block_tokens * 4 + i];
        const int64_t at = (token0 + i / 4) * hidden + row0 + 4 * (i & 3);
        if (splits > 1) {
            *(f32x4_t *)(A.partial + blockIdx.z * A.tokens * hidden + at) = s;
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (A.out_bf16) ((__bf16 *)A.out)[at + j] = (__bf16)s[j];
            else ((float *)A.out)[at + j] = s[j];
        }
    }
}

// The splits' sums, in their order.
__global__ __launch_bounds__(256) void moe_join_kernel(const f32x4_t *partial, int splits, int64_t n,
                                                       void *out, bool out_bf16) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    f32x4_t s = partial[i];
    for (int z = 1; z < splits; ++z) s += partial[z * n + i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (out_bf16) ((__bf16 *)out)[4 * i + j] = (__bf16)s[j];
        else ((float *)out)[4 * i + j] = s[j];
    }
}

// Workgroups that share the down product of 16 rows and a block's tokens: as many as there
// are CUs for, where each still has some 32 groups of K to go through (64 tokens of 128
// experts, 2048 x 768: 169 us in one, 137 in two; 32 of 64, 1408 in NVFP4: 152 and 122; but
// 2 of 128: 28.0 and 28.8, the launch that joins them).
int down_splits(int64_t tokens, int top_k, int64_t hidden, int64_t inner) {
    const int64_t groups = hidden / 16 * ((tokens + MOE_BLOCK - 1) / MOE_BLOCK);
    const int64_t pairs = (tokens < MOE_BLOCK ? tokens : MOE_BLOCK) * top_k;
    const int64_t work = pairs * ((inner + W4_GROUP - 1) / W4_GROUP);
    const int64_t splits = 256 / groups < work / 32 ? 256 / groups : work / 32;
    return splits < 1 ? 1 : splits > 8 ? 8 : (int)splits;
}

template <int FMT, bool X_F32, int TOKENS>
hipError_t launch_tile(MoeArgs A, int32_t *status, hipStream_t s) {
    const int block = (int)(A.tokens < MOE_BLOCK ? A.tokens : MOE_BLOCK);
    A.slots = (int64_t)block * A.top_k < A.W.experts;
    const uint32_t blocks = (uint32_t)((A.tokens + MOE_BLOCK - 1) / MOE_BLOCK);
    const dim3 up_grid((uint32_t)(A.W.inner / 16),
                       (uint32_t)(A.slots ? block * A.top_k : A.W.experts), blocks);
    const size_t up_lds = UP_WAVES * (XPart<X_F32, TOKENS>::PIECES + RowsAt<FMT, 2>::LDS) * 16;
    moe_up_kernel<FMT, X_F32, TOKENS><<<up_grid, UP_WAVES * WAVE, up_lds, s>>>(A, status);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const auto down_lds = [&](int tokens) {
        return (size_t)DOWN_WAVES<TOKENS> *
                   (tokens * 4 + Gated<X_F32, TOKENS>::X::PIECES + RowsAt<FMT, 1>::LDS) * 16 +
               MoePlan::bytes(tokens * A.top_k);
    };
    int down_block = block;  // fewer tokens where a plan of many pairs leaves no room for them
    while (down_block > 16 && down_lds(down_block) > LDS_BYTES) down_block = (down_block + 1) / 2;
    const int splits = down_splits(A.tokens, A.top_k, A.W.hidden, A.W.inner);
    const dim3 grid((uint32_t)(A.W.hidden / 16), (uint32_t)((A.tokens + down_block - 1) / down_block),
                    (uint32_t)splits);
    moe_down_kernel<FMT, X_F32, TOKENS>
        <<<grid, DOWN_WAVES<TOKENS> * WAVE, down_lds(down_block), s>>>(A, down_block);
    e = hipGetLastError();
    if (e != hipSuccess || splits == 1) return e;
    const int64_t n = A.tokens * A.W.hidden / 4;
    moe_join_kernel<<<(uint32_t)((n + 255) / 256), 256, 0, s>>>((const f32x4_t *)A.partial, splits, n,
                                                                 A.out, A.out_bf16);
    return hipGetLastError();
}

template <int FMT, bool X_F32>
hipError_t launch_experts(const MoeArgs &A, int32_t *status, hipStream_t s) {
    const int block = (int)(A.tokens < MOE_BLOCK ? A.tokens : MOE_BLOCK);
    if (dense(block * A.top_k, A.W.experts)) return launch_tile<FMT, X_F32, 8>(A, status, s);
    return launch_tile<FMT, X_F32, 4>(A, status, s);
}

// Shares of K: so many that there is a workgroup for each CU, and work for its waves.
// Four waves of one step each where there are few tiles (1 x 2048 of 64 experts: 7.4 us in
// all, 7.9 with sixteen), sixteen where there are many, so that loads wait for each other
// less (64 x 4096 of 256: 14.4, with four 15.8).
struct RouteShape {
    int waves, splits;
};
RouteShape route_shape(int64_t tokens, int64_t hidden, int experts) {
    const int64_t tiles = (tokens + 15) / 16 * ((experts + 15) / 16);
    const int waves = tiles < 32 ? 4 : 16;
    const int64_t most = (hidden + 32 * waves - 1) / (32 * waves), want = (256 + tiles - 1) / tiles;
    int splits = 1;
    while (splits < 16 && splits < want && splits < most) splits *= 2;
    return {waves, splits};
}

template <typename XT, typename RT>
hipError_t launch_logits(const void *x, const void *router, double *logits, int64_t tokens,
                         int64_t hidden, int experts, RouteShape shape, hipStream_t s) {
    const int expert_tiles = (experts + 15) / 16;
    const uint32_t groups = (uint32_t)((tokens + 15) / 16 * expert_tiles * shape.splits);
    if (shape.waves == 4)
        route_logits_kernel<XT, RT, 4><<<groups, 4 * WAVE, 0, s>>>(
            (const XT *)x, (const RT *)router, logits, tokens, hidden, experts, expert_tiles,
            shape.splits);
    else
        route_logits_kernel<XT, RT, 16><<<groups, 16 * WAVE, 0, s>>>(
            (const XT *)x, (const RT *)router, logits, tokens, hidden, experts, expert_tiles,
            shape.splits);
    return hipGetLastError();
}

}  // namespace

// The workspaces' sizes do not fall with the tokens: one for the largest batch serves every
// smaller one.  Shares get fewer where tiles of tokens get more, and within a tile the
// largest count needs most, so these are the counts to look at.
size_t route_workspace_bytes(int64_t tokens, int64_t hidden, int experts) {
    const auto rows = [&](int64_t t) { return route_shape(t, hidden, experts).splits * t; };
    int64_t most = rows(tokens);
    for (int64_t t = 16; t < tokens && rows(t) > t; t += 16) most = rows(t) > most ? rows(t) : most;
    return (size_t)most * experts * sizeof(double);
}

hipError_t launch_route(const void *x, bool x_bf16, int64_t tokens, int64_t hidden,
                        const void *router, bool router_bf16, int experts, int top_k,
                        bool renormalize, int32_t *chosen, float *weights, void *workspace,
                        hipStream_t s) {
    double *logits = (double *)workspace;
    const RouteShape shape = route_shape(tokens, hidden, experts);
    hipError_t e;
    if (x_bf16)
        e = router_bf16 ? launch_logits<uint16_t, uint16_t>(x, router, logits, tokens, hidden,
                                                            experts, shape, s)
                        : launch_logits<uint16_t, float>(x, router, logits, tokens, hidden, experts,
                                                         shape, s);
    else
        e = router_bf16 ? launch_logits<float, uint16_t>(x, router, logits, tokens, hidden, experts,
                                                         shape, s)
                        : launch_logits<float, float>(x, router, logits, tokens, hidden, experts,
                                                      shape, s);
    if (e != hipSuccess) return e;
    const int threads = (experts + WAVE - 1) / WAVE * WAVE;
    route_choose_kernel<<<(uint32_t)tokens, threads, 0, s>>>(logits, tokens, experts, shape.splits,
                                                            top_k, renormalize, chosen, weights);
    return hipGetLastError();
}

static size_t act_bytes(int64_t tokens, int top_k, int64_t inner, bool x_bf16) {
    return (size_t)tokens * top_k * inner * (x_bf16 ? sizeof(float) : 3 * sizeof(uint16_t));
}

size_t experts_workspace_bytes(int64_t tokens, int top_k, int64_t hidden, int64_t inner, bool x_bf16) {
    const auto bytes = [&](int64_t t) {
        const int splits = down_splits(t, top_k, hidden, inner);
        return act_bytes(t, top_k, inner, x_bf16) +
               (splits > 1 ? (size_t)splits * t * hidden * sizeof(float) : 0);
    };
    size_t most = bytes(tokens);
    for (int64_t t = MOE_BLOCK; t < tokens && down_splits(t, top_k, hidden, inner) > 1; t += MOE_BLOCK)
        most = bytes(t) > most ? bytes(t) : most;
    return most;
}

hipError_t launch_experts(int fmt, const MoeWeights &W, const void *x, bool x_bf16, int64_t tokens,
                          const int32_t *ids, const float *weights, int top_k, void *out,
                          bool out_bf16, void *workspace, int32_t *status, hipStream_t s) {
    // rows of act are multiples of 32 bytes, so partial is aligned too
    float *partial = (float *)((char *)workspace + act_bytes(tokens, top_k, W.inner, x_bf16));
    const MoeArgs A = {x, ids, weights, W, (uint16_t *)workspace, partial, out, tokens, top_k, 0, out_bf16};
    if (fmt == 0)
        return x_bf16 ? launch_experts<0, false>(A, status, s) : launch_experts<0, true>(A, status, s);
    return x_bf16 ? launch_experts<1, false>(A, status, s) : launch_experts<1, true>(A, status, s);
}

}  // namespace fp4dev

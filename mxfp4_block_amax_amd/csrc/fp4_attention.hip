// fp4_attention.hip - attention over the 8-bit key/value cache.
//
//   S_rj = scale q_r . k_j over the visible keys j of row r,
//   out_r = sum_j exp(S_rj) v_j / sum_j exp(S_rj).
//
// One pass over the keys with a running reference m_r and sum per row, both
// fp32: weights are p = 2^(S log2 e - d - m), d the exponent by which the scale
// of the key's value page is below E, the largest among the workgroup's pages.
// So a weight carries its page's scale: what a row's sums lose is relative to
// its own largest weight, not to pages that other rows see.  Pages of one scale
// have d = 0.  The reference is raised (and the sums rescaled) only when some
// weight passes it by more than 2^15, to 2^-7 of that weight: most steps then need
// no rescaling and no exchange between lanes.  The sum of the probabilities takes
// p 2^d.  d ends at 80, which keeps that sum below 2^122; the values take the rest.
//
// First product, on the bf16 MFMA: keys E4M3(c) 2^e are exact in bf16 (the
// converter applies the scale) and bf16 queries multiply as they are; fp32
// queries are three bf16 terms, all 24 bits.
// Second product, on the fp16 MFMA: p is at most 2^15 and rounded to fp16
// (relative 2^-11, an eighth of what bf16 would lose; a row's largest p is 2^7
// or more, so what is lost below fp16's range is under 2^-32 of it), for fp32
// queries two fp16 terms (22 bits).  Values are E4M3(c) 2^6: at most 28672, and
// from d = 80 on down to fp16's end: exact (its subnormals are multiplied as they
// are) for pages down to 2^-101 of the largest.  The sums take 2^(E - 6) back at
// the end.
#include <algorithm>
#include <type_traits>

#include "fp4_kernels.h"
#include "fp4_kv.h"

namespace fp4dev {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kRaiseAbove = 15.0f;  // a weight this far over its reference raises it ..
constexpr float kRaiseTo = 7.0f;      // .. to this far below that weight
constexpr int kVBias = 6;             // values are scaled by 2^kVBias
constexpr int kCarry = 80;            // the most of a page's distance from E that weights carry

struct AttnArgs {
    const void *q;
    int64_t q_token, q_head;
    void *out;
    float *lse;
    float *part_o;   // [tokens, heads, splits, dim]
    float2 *part_ml;  // [tokens, heads, splits]: reference (base 2), sum
    int32_t heads, group, causal, window;
    int32_t sub, sub_heads;          // pieces of a group, and the query heads of one
    int32_t items, tokens;           // row tiles launched, and the tokens of one
    int32_t splits, split_keys;      // launched splits, keys of one
    float scale2;                    // |scale| log2 e
    uint32_t q_sign;                 // sign bits of two bf16 queries (or of one fp32) if scale < 0
};

// A row tile's tokens and the keys any of them sees.
struct Tile {
    int64_t pos0;       // position of its first token
    int64_t base, end;  // keys [base, end), base a page's first
    int64_t first;      // the first key any of them sees
    int tokens;
};

__device__ __forceinline__ Tile tile_range(const KvCache &C, const KvBatch &B, const AttnArgs &A,
                                           const Item &it, int first_row, int32_t *status) {
    Tile T;
    T.tokens = min(A.tokens, it.count - first_row);
    const int64_t len = it.length;
    T.pos0 = len - it.count + first_row;
    int64_t end = A.causal ? T.pos0 + T.tokens : len;
    const int64_t held = (int64_t)B.width << C.block_shift;
    if (end > held) {
        if (threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
        end = held;
    }
    const int64_t first = A.window > 0 ? max(T.pos0 - A.window + 1, (int64_t)0) : 0;
    T.first = first;
    T.base = first & ~(int64_t)(C.block - 1);
    T.end = max(end, T.base);
    return T;
}

template <typename V, int N>
struct Parts {
    V p[N];
};

// x as N terms of a narrower type: each the nearest to what the ones before
// left, an exact difference.
template <typename V, int N, int COUNT>
__device__ __forceinline__ Parts<V, N> split_parts(const float (&x)[COUNT]) {
    Parts<V, N> r;
    float rest[COUNT];
#pragma unroll
    for (int i = 0; i < COUNT; ++i) rest[i] = x[i];
#pragma unroll
    for (int k = 0; k < N; ++k) {
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            r.p[k][i] = rest[i];
            if (k + 1 < N) rest[i] = rest[i] - (float)r.p[k][i];
        }
    }
    return r;
}

// Eight cache values as bf16, the scale applied: two words of codes in order.
__device__ __forceinline__ bf16x8_t widen_codes(uint32_t a, uint32_t b, float scale) {
    const bf16x2_t r[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true)};
    bf16x8_t v;
    __builtin_memcpy(&v, r, sizeof(v));
    return v;
}

__device__ __forceinline__ f32x4_t mfma16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma16(f16x8_t a, f16x8_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma16(f16x4_t a, f16x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x16f16(a, b, c, 0, 0, 0);
}

// d of a value page of scale byte `byte` where the largest is `top`, the factor
// 2^d, and the converter's scale operand (255, a NaN page, stays NaN).
__device__ __forceinline__ int v_below(uint32_t byte, uint32_t top) {
    return byte == 255u ? 0 : min((int)top - (int)byte, kCarry);
}
__device__ __forceinline__ float v_lift(int below) {
    return u2f((E8M0_ONE + (uint32_t)below) << 23);
}
__device__ __forceinline__ float v_operand(uint32_t byte, uint32_t top) {
    const int e = kVBias + (int)E8M0_ONE - max((int)top - (int)byte - kCarry, 0);
    return u2f(byte == 255u ? 255u << 23 : (uint32_t)max(e, 0) << 23);
}

// A split's reference and sum for the join: the sum's exponent goes into the
// reference, so that products of weights and outputs stay in range.
__device__ __forceinline__ float2 split_weight(float m, float l) {
    const int e = __builtin_amdgcn_frexp_expf(l);
    return make_float2(m + (float)e, __builtin_ldexpf(l, -e));
}

// Launch order: heads, then row tiles, then splits, so that the tiles that read
// the same keys are near each other in time and, for 8 heads, on the same XCD and
// its L2 (8 sequences x 20 tokens over 4096 keys, 8 x 4 heads of 256: 97 us, row
// tiles first 112; 4 tokens, 8 x 8 heads of 128: 32 and 52).  More row tiles than a
// grid's y go first.
constexpr int NARROW_GRID_Y = 65535;
constexpr int NARROW_PAGES = 256;  // pages under a workgroup's keys, at most

template <int D, int WAVES>
struct NarrowShared {
    int page[NARROW_PAGES];
    uint8_t k_scale[NARROW_PAGES], v_scale[NARROW_PAGES];
    uint32_t v_top;  // the largest of v_scale but NaN
    float m[WAVES][16], l[WAVES][16];
    float o[WAVES][16][D + 4];
};

// A lane's values of one token: D / 16 consecutive dimensions.
template <int D>
struct VBytes {
    uint32_t w[D / 64];
};

template <int D>
__device__ __forceinline__ VBytes<D> load_v(const uint8_t *p) {
    VBytes<D> r;
    if constexpr (D == 64) {
        r.w[0] = *(const uint32_t *)p;
    } else if constexpr (D == 128) {
        const uint2 x = *(const uint2 *)p;
        r.w[0] = x.x, r.w[1] = x.y;
    } else if constexpr (D == 192) {
#pragma unroll
        for (int i = 0; i < 3; ++i) r.w[i] = ((const uint32_t *)p)[i];
    } else {
        const uint4 x = *(const uint4 *)p;
        r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    }
    return r;
}

// 16-key halves of a wave's step: two, or one where a step of more dimensions
// would leave no registers to load the next one into (24 sequences x 5 tokens
// over 1024 keys of 256 dimensions, the values of 32 keys loaded as they are
// needed: 33 us; with halves 25).
template <int D>
constexpr int kHalves = D <= 128 ? 2 : 1;

// Waves of a SIMD, by registers, and waves of a workgroup that has a CU for
// itself.  The three terms of an fp32 query of 256 dimensions take 96 registers;
// those of 64 spill with four waves (16 sequences x 2048 keys, 16 heads: 27 us,
// with three 22).
template <int D, bool F32>
constexpr int kNarrowOccupancy = D == 64 ? (F32 ? 3 : 4) : F32 && D == 256 ? 1 : 2;
template <int D, bool F32>
constexpr int kNarrowMany = 4 * kNarrowOccupancy<D, F32>;

// The codes of one step: a lane's keys and values.
template <int D>
struct Step {
    uint4 k[kHalves<D>][D / 64];  // key lane % 16 of a half, dimensions 64 c + 16 (lane / 16) ..
    VBytes<D> v[kHalves<D>][4];   // keys 4 (lane / 16) + i of a half, dimensions D / 16 (lane % 16) ..
};

// Row tiles of up to 16 query rows (tokens x the query heads of one kv head):
// single tokens, drafts, short chunks.
//
// A workgroup has one row tile, one kv head and one range of keys; its waves
// take 32 keys at a time in turn (16 of more than 128 dimensions).  Scores are
// computed transposed,
// S^T = K Q^T, so that a lane's scores are those of one row (lane % 16) and its
// keys, 4 (lane / 16) + i, are the ones the second product wants from this
// lane: probabilities go from the first product to the second without leaving
// their lane.  Out^T = V^T P^T; which keys are which of a product's 32 terms is
// free as long as V follows P, and which dimension is which row of a tile is
// free too, so a lane loads D / 16 consecutive bytes of eight (four) value rows
// and transposes them by byte permutes.  Nothing of keys or values goes through
// LDS: each byte is used by one lane.
//
// Long decoding is bound by HBM: 64 tokens over about 8192 keys each, 8 x 8 heads
// of 128, read 1084 MB in 206 us (5.3 TB/s; 190 at equal lengths), one over 200001
// 410 MB in 76 us (5.4 TB/s).  Short calls are bound by latency, some 2 us a step
// where a CU has one workgroup: a token over 1000 keys takes 14.1 us.
template <int D, bool F32, int WAVES>
__global__ __launch_bounds__(WAVES *WAVE, (kNarrowOccupancy<D, F32>)) void attention_narrow_kernel(
    KvCache C, KvBatch B, AttnArgs A, int32_t *status) {
    constexpr int HALVES = kHalves<D>, KEYS = 16 * HALVES, N = 4 * HALVES;  // keys of a wave, of a lane
    constexpr int STEP = KEYS * WAVES;                                     // of a workgroup
    using Values = std::conditional_t<HALVES == 2, f16x8_t, f16x4_t>;
    constexpr int CH = D / 64, NT = D / 16;
    constexpr int QP = F32 ? 3 : 1, PP = F32 ? 2 : 1;  // terms of a query and a probability
    __shared__ NarrowShared<D, WAVES> sh;
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int r = lane & 15, g = lane >> 4;
    if (threadIdx.x == 0) sh.v_top = 0;
    __syncthreads();
    const bool heads_first = A.items <= NARROW_GRID_Y;
    const int headsub = heads_first ? blockIdx.x : blockIdx.y;
    // a sequence's last tiles, with the most keys, first (6 fp32 chunks of about 700
    // tokens, 8 x 5 heads of 192: 357 us, first tiles first 377)
    const int item = !heads_first ? blockIdx.x
                     : A.tokens > 1 ? gridDim.y - 1 - blockIdx.y : blockIdx.y;
    const Item it = A.tokens > 1 && B.seqs < TILE_SEQS
                        ? find_tile(B, item, A.tokens, status)
                        : find_item(B, item, A.items, A.tokens, A.tokens > 1 ? 1 : 0,
                                    headsub == 0 && blockIdx.z == 0, status);
    const int row0 = it.piece * A.tokens;
    if (it.count <= 0 || row0 >= it.count) {
        if (it.count < 0 && threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
        return;
    }
    const int head = headsub / A.sub, sub = headsub - head * A.sub;
    const int split = blockIdx.z;
    const bool none = it.seq >= B.seqs;
    Tile T;
    if (none) {
        T.tokens = min(A.tokens, it.count - row0);
        T.pos0 = T.base = T.first = T.end = 0;
    } else {
        T = tile_range(C, B, A, it, row0, status);
    }
    // this lane's row: token i, query head h (of the group)
    const int h0 = sub * A.sub_heads;
    const int hn = min(A.sub_heads, A.group - h0);
    const int ri = r / hn, rh = r - ri * hn;
    const bool row_real = ri < T.tokens;
    const int64_t token = it.base + row0 + ri;
    const int hq = head * A.group + h0 + rh;
    const int64_t k0 = T.base + (int64_t)split * A.split_keys;
    const int64_t k1 = min(k0 + A.split_keys, T.end);
    const bool whole = T.end - T.base <= A.split_keys;  // the tile has one split
    if (k0 >= k1 && split > 0) return;

    // the keys this lane's row sees (a row that is none sees all: its sums go
    // nowhere, and its steps need no masks)
    const int64_t pos = T.pos0 + ri;
    const int64_t last = row_real && A.causal ? pos : T.end - 1;
    const int64_t first = row_real && A.window > 0 ? pos - A.window + 1 : 0;
    // positions from here on are relative to k0
    const int keys = (int)max(k1 - k0, (int64_t)0);
    const int last_r = (int)max(min(last - k0, (int64_t)keys - 1), (int64_t)-1);
    const int first_r = (int)max(min(first - k0, (int64_t)keys), (int64_t)0);

    // queries: B operand, lane's row r, dimensions 64 c + 16 g + 8 h ..
    Parts<bf16x8_t, QP> q[CH][2];
    {
        const int64_t at = token * A.q_token + hq * A.q_head + 16 * g;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if constexpr (!F32) {
                    uint4 w = make_uint4(0, 0, 0, 0);
                    if (row_real) w = *(const uint4 *)((const uint16_t *)A.q + at + 64 * c + 8 * h);
                    w.x ^= A.q_sign, w.y ^= A.q_sign, w.z ^= A.q_sign, w.w ^= A.q_sign;
                    q[c][h].p[0] = __builtin_bit_cast(bf16x8_t, w);
                } else {
                    float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                    if (row_real) {
                        const uint4 *p = (const uint4 *)((const float *)A.q + at + 64 * c + 8 * h);
                        widen_f32x8(p[0], p[1], x);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = u2f(f2u(x[i]) ^ A.q_sign);
                    q[c][h] = split_parts<bf16x8_t, QP>(x);
                }
            }
    }

    // The pages under [k0, k1), k0 a page's first.  A wave looks its first step's
    // up by itself, so that the step's codes are on their way while the
    // workgroup's pages and their scales are.
    const int64_t b0 = k0 >> C.block_shift;
    const int pages = (keys + C.block - 1) >> C.block_shift;
    const uint32_t k_lane = (uint32_t)(r * D + 16 * g);
    const uint32_t v_lane = (uint32_t)(4 * g * D + r * (D / 16));
    auto page_at = [&](int j) {  // of the keys from j on; clamped to the last
        return __builtin_amdgcn_readfirstlane(min(j >> C.block_shift, pages - 1));
    };
    auto load = [&](int j, Step<D> &s, const int(&page)[HALVES]) {
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
            const int64_t at = page_offset(C, max(page[half], 0), head) +
                               ((j + 16 * half) & (C.block - 1)) * D;
            const uint8_t *kp = C.k_codes + at, *vp = C.v_codes + at;
#pragma unroll
            for (int c = 0; c < CH; ++c) s.k[half][c] = *(const uint4 *)(kp + k_lane + 64 * c);
#pragma unroll
            for (int i = 0; i < 4; ++i) s.v[half][i] = load_v<D>(vp + v_lane + i * D);
        }
    };
    auto load_held = [&](int j, Step<D> &s) {
        int page[HALVES];
#pragma unroll
        for (int half = 0; half < HALVES; ++half)
            page[half] = __builtin_amdgcn_readfirstlane(sh.page[page_at(j + 16 * half)]);
        load(j, s, page);
    };
    Step<D> now, next;
    // a window may start inside its first page
    const int start = (int)max(min(T.first - k0, (int64_t)keys), (int64_t)0) / STEP * STEP;
    int j = start + KEYS * wave;
    const int busy = min(max((keys - start + KEYS - 1) / KEYS, 1), WAVES);  // waves that have a step
    {
        int page = -1, first_pages[HALVES];
        if ((int)threadIdx.x < pages) page = find_page(B, C, it.seq, b0 + threadIdx.x);
        if (j < keys) {
#pragma unroll
            for (int half = 0; half < HALVES; ++half)
                first_pages[half] = __builtin_amdgcn_readfirstlane(
                    find_page(B, C, it.seq, b0 + page_at(j + 16 * half)));
            load(j, now, first_pages);
        }
        uint32_t v_top = 0;
        auto hold = [&](int i, int page) {
            const int64_t at = (int64_t)max(page, 0) * C.heads + head;
            const uint32_t ks = page < 0 ? 0u : C.k_scales[at], vs = page < 0 ? 0u : C.v_scales[at];
            sh.page[i] = page;
            sh.k_scale[i] = (uint8_t)ks;
            sh.v_scale[i] = (uint8_t)vs;
            if (vs != 255u) v_top = max(v_top, vs);
            if (page < 0) flag(status, FLAG_CACHE_INDEX);
        };
        if ((int)threadIdx.x < pages) hold(threadIdx.x, page);
        if (v_top > 0) atomicMax(&sh.v_top, v_top);
    }
    __syncthreads();
    const uint32_t v_top = __builtin_amdgcn_readfirstlane(sh.v_top);

    f32x4_t o[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n] = f32x4_t{0, 0, 0, 0};
    float m = -__builtin_inff(), l = 0.0f;

    auto compute = [&](int j, Step<D> &st) {
        f32x4_t s[HALVES];
        float vs[HALVES], below[HALVES], lift[HALVES];
        bool held[HALVES], all_held = true;
#pragma unroll
        for (int half = 0; half < HALVES; ++half) {
            const int at = page_at(j + 16 * half);
            held[half] = sh.page[at] >= 0;
            all_held = all_held && held[half];
            const float ks = e8m0_operand(__builtin_amdgcn_readfirstlane(sh.k_scale[at]));
            const uint32_t vb = __builtin_amdgcn_readfirstlane(sh.v_scale[at]);
            vs[half] = v_operand(vb, v_top);
            below[half] = (float)v_below(vb, v_top);
            lift[half] = v_lift(v_below(vb, v_top));
            s[half] = f32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const uint4 w = st.k[half][c];
                const bf16x8_t ka = widen_codes(w.x, w.y, ks), kb = widen_codes(w.z, w.w, ks);
#pragma unroll
                for (int p = QP - 1; p >= 0; --p) {
                    s[half] = mfma16(ka, q[c][0].p[p], s[half]);
                    s[half] = mfma16(kb, q[c][1].p[p], s[half]);
                }
            }
        }
        float x[N];  // base-2 scores: keys 4 g + i, then 16 + 4 g + i
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = s[i / 4][i & 3] * A.scale2;
        // a step that some row does not see whole
        const bool clean = j >= first_r && j + KEYS - 1 <= last_r;
        const bool edge = __ballot(!clean) != 0 || !all_held;
        bool fix = false;
        if (edge) {
            const int top = min(keys, j + KEYS);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int key = j + 16 * (i / 4) + 4 * g + (i & 3);
                if (key < first_r || key > last_r || !held[i / 4]) x[i] = -__builtin_inff();
                // values nothing sees are zeros, whatever the page holds there
                if (key >= top || !held[i / 4])
#pragma unroll
                    for (int c = 0; c < CH; ++c) st.v[i / 4][i & 3].w[c] = 0;
            }
            // NaN values that only some rows see
            uint32_t nan = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    uint32_t &w = st.v[i / 4][i & 3].w[c];
                    if (f2u(vs[i / 4]) == 0x7F800000u && j + 16 * (i / 4) + 4 * g + (i & 3) < top)
                        w = 0x7F7F7F7Fu;
                    nan |= (w & 0x7F7F7F7Fu) + 0x01010101u;
                }
            fix = __ballot((nan & 0x80808080u) != 0) != 0;
        }
        float top = x[0];
#pragma unroll
        for (int i = 1; i < N; ++i) top = __builtin_fmaxf(top, x[i]);
        if (__ballot(top > m + kRaiseAbove) != 0) {  // some weight may (d is not negative)
            top = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < N; ++i) top = __builtin_fmaxf(top, x[i] - below[i / 4]);
            top = __builtin_fmaxf(top, __shfl_xor(top, 16, WAVE));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32, WAVE));
            const float next = __builtin_fmaxf(m, top - kRaiseTo);
            const float keep = m == next ? 1.0f : __builtin_amdgcn_exp2f(m - next);
            m = next;
            l *= keep;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n] *= keep;
        }
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        float p[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            p[i] = __builtin_amdgcn_exp2f(x[i] - (ref + below[i / 4]));
            l = __builtin_fmaf(p[i], lift[i / 4], l);
        }
        const Parts<Values, PP> pb = split_parts<Values, PP>(p);
        // values: tile n has dimensions NT row + n; words of two keys interleaved
        auto codes_of = [&](auto &&word, int n, uint32_t(&w)[N / 2]) {
            // bytes of dimension n, a lane's keys, two to each half word
            const int c = n / 4;
            const uint32_t sel = (n & 2) ? 0x07030602u : 0x05010400u;
#pragma unroll
            for (int k = 0; k < N / 2; ++k)
                w[k] = __builtin_amdgcn_perm(word(2 * k + 1, c), word(2 * k, c), sel);
        };
        auto pair = [&](const uint32_t(&w)[N / 2], bool hi, const float(&scale)[HALVES]) {
            f16x2_t t[N / 2];
#pragma unroll
            for (int k = 0; k < N / 2; ++k)
                t[k] = hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[k], scale[k / 2], true)
                          : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[k], scale[k / 2], false);
            Values v;
            __builtin_memcpy(&v, t, sizeof(v));
            return v;
        };
        if (!fix) {
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t w[N / 2];
                codes_of([&](int i, int c) { return st.v[i / 4][i & 3].w[c]; }, n, w);
                const Values va = pair(w, false, vs), vb = pair(w, true, vs);
#pragma unroll
                for (int k = PP - 1; k >= 0; --k) {
                    o[n] = mfma16(va, pb.p[k], o[n]);
                    o[n + 1] = mfma16(vb, pb.p[k], o[n + 1]);
                }
            }
        } else {
            // The sums without the NaN values, then NaN where a row sees one:
            // a product of where they are with who sees them counts it.
            float see[N];
#pragma unroll
            for (int i = 0; i < N; ++i) see[i] = x[i] == -__builtin_inff() ? 0.0f : 1.0f;
            const Values sb = split_parts<Values, 1>(see).p[0];
            float finite[HALVES], one[HALVES];  // scales: of values that are not NaN; of marks
#pragma unroll
            for (int half = 0; half < HALVES; ++half) {
                finite[half] = f2u(vs[half]) == 0x7F800000u ? 1.0f : vs[half];
                one[half] = 1.0f;
            }
            auto nans = [&](int i, int c) {  // 0x80 in the bytes that are NaN
                return ((st.v[i / 4][i & 3].w[c] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
            };
#pragma unroll
            for (int n = 0; n < NT; n += 2) {
                uint32_t w[N / 2], z[N / 2];
                codes_of([&](int i, int c) {
                    const uint32_t b = nans(i, c);
                    return st.v[i / 4][i & 3].w[c] & ~((b >> 7) * 0xFFu);
                }, n, w);
                codes_of([&](int i, int c) { return (nans(i, c) >> 7) * 0x38u; }, n, z);
                const Values va = pair(w, false, finite), vb = pair(w, true, finite);
#pragma unroll
                for (int k = PP - 1; k >= 0; --k) {
                    o[n] = mfma16(va, pb.p[k], o[n]);
                    o[n + 1] = mfma16(vb, pb.p[k], o[n + 1]);
                }
                const f32x4_t zero = {0, 0, 0, 0};
                const f32x4_t ca = mfma16(pair(z, false, one), sb, zero);
                const f32x4_t cb = mfma16(pair(z, true, one), sb, zero);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (ca[i] > 0.0f) o[n][i] = __builtin_nanf("");
                    if (cb[i] > 0.0f) o[n + 1][i] = __builtin_nanf("");
                }
            }
        }
    };

    while (j < keys) {
        const int after = j + STEP;
        if (after < keys) load_held(after, next);
        compute(j, now);
        now = next;
        j = after;
    }

    // join the waves
    l += __shfl_xor(l, 16, WAVE);
    l += __shfl_xor(l, 32, WAVE);
    if (g == 0) {
        sh.m[wave][r] = m;
        sh.l[wave][r] = l;
    }
    __syncthreads();
    // `count` waves: all, as a constant, or those that had a step
    auto join = [&](auto count) {
        if (wave < count) {
            float top = sh.m[0][r];
#pragma unroll
            for (int w = 1; w < count; ++w) top = __builtin_fmaxf(top, sh.m[w][r]);
            const float own = m == top ? 1.0f : __builtin_amdgcn_exp2f(m - top);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float *to = &sh.o[wave][r][NT * (4 * g + i)];
#pragma unroll
                for (int n = 0; n < NT; n += 4) {
                    f32x4_t y = {o[n][i], o[n + 1][i], o[n + 2][i], o[n + 3][i]};
                    y *= own;
                    *(f32x4_t *)(to + n) = y;
                }
            }
        }
        __syncthreads();
        // 16 lanes a row, four dimensions at a time
        if (threadIdx.x >= 256) return;
        const int rr = threadIdx.x >> 4, part = threadIdx.x & 15;
        const int ti = rr / hn, th = rr - ti * hn;
        if (ti >= T.tokens) return;
        float m_all = sh.m[0][rr], l_all = 0.0f;
#pragma unroll
        for (int w = 1; w < count; ++w) m_all = __builtin_fmaxf(m_all, sh.m[w][rr]);
#pragma unroll
        for (int w = 0; w < count; ++w) {
            const float mw = sh.m[w][rr];
            l_all = __builtin_fmaf(sh.l[w][rr],
                                   mw == m_all ? 1.0f : __builtin_amdgcn_exp2f(mw - m_all), l_all);
        }
        const int64_t row = (it.base + row0 + ti) * (int64_t)A.heads + head * A.group + h0 + th;
        const float inv = l_all == 0.0f ? 0.0f : 1.0f / l_all;
        const int back = (int)v_top - (int)E8M0_ONE - kVBias;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int d = 64 * c + 4 * part;
            f32x4_t y = *(const f32x4_t *)&sh.o[0][rr][d];
#pragma unroll
            for (int w = 1; w < count; ++w) y += *(const f32x4_t *)&sh.o[w][rr][d];
            y *= inv;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = __builtin_ldexpf(y[i], back);
            if (!whole) {
                *(f32x4_t *)(A.part_o + (row * A.splits + split) * D + d) = y;
            } else if constexpr (!F32) {
                const f32x2_t lo = {y.x, y.y}, hi = {y.z, y.w};
                *(uint2 *)((uint16_t *)A.out + row * D + d) =
                    make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2_t)),
                               __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2_t)));
            } else {
                *(f32x4_t *)((float *)A.out + row * D + d) = y;
            }
        }
        if (part == 0) {
            if (!whole)
                A.part_ml[row * A.splits + split] = split_weight(m_all, l_all);
            else if (A.lse != nullptr)
                A.lse[row] = l_all == 0.0f ? -__builtin_inff()
                                           : ((m_all == -__builtin_inff() ? 0.0f : m_all) +
                                              __builtin_amdgcn_logf(l_all)) * kLn2;
        }
    };
    if (busy == WAVES)
        join(std::integral_constant<int, WAVES>{});
    else if (busy == 1)
        join(std::integral_constant<int, 1>{});
    else
        join(busy);
}

// Joins the splits of rows that have more than one: a workgroup a row.  A
// split's output is normalised by its own sum, so its weight is that sum.  D / 4
// lanes have four dimensions each; the groups of lanes take every GROUPS-th split
// and are added in order.
constexpr int JOIN_WG = 256;

template <int D, bool F32>
__global__ __launch_bounds__(JOIN_WG) void attention_join_kernel(KvCache C, KvBatch B, AttnArgs A) {
    constexpr int LANES = D / 4, GROUPS = JOIN_WG / LANES;
    __shared__ float tops[JOIN_WG / WAVE], sums[GROUPS];
    __shared__ f32x4_t outs[GROUPS][LANES];
    const int64_t row = (int64_t)blockIdx.x * A.heads + blockIdx.y;
    const Item it = search_item(B, (int)blockIdx.x, 1, 0);
    if (it.count <= 0 || it.seq >= B.seqs || it.piece >= it.count) return;
    const Tile T = tile_range(C, B, A, it, it.piece / A.tokens * A.tokens, nullptr);
    const int n = (int)((T.end - T.base + A.split_keys - 1) / A.split_keys);
    if (n <= 1) return;
    const float2 *ml = A.part_ml + row * A.splits;
    float top = -__builtin_inff();
    for (int i = threadIdx.x; i < n; i += JOIN_WG) top = __builtin_fmaxf(top, ml[i].x);
    for (int off = 32; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off, WAVE));
    if ((threadIdx.x & (WAVE - 1)) == 0) tops[threadIdx.x / WAVE] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < JOIN_WG / WAVE; ++w) top = __builtin_fmaxf(top, tops[w]);
    const int g = threadIdx.x / LANES, lane = threadIdx.x - g * LANES;
    float l = 0.0f;
    f32x4_t o = {0, 0, 0, 0};
    if (g < GROUPS) {
        const f32x4_t *po = (const f32x4_t *)(A.part_o + row * A.splits * D) + lane;
#pragma unroll 4
        for (int i = g; i < n; i += GROUPS) {
            const float2 w = ml[i];
            const float f = w.y * (w.x == top ? 1.0f : __builtin_amdgcn_exp2f(w.x - top));
            const f32x4_t x = po[(int64_t)i * LANES];
            l += f;
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = __builtin_fmaf(x[k], f, o[k]);
        }
        outs[g][lane] = o;
        if (lane == 0) sums[g] = l;
    }
    __syncthreads();
    if (threadIdx.x >= LANES) return;
    l = sums[0];
    o = outs[0][lane];
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) {
        l += sums[k];
        o += outs[k][lane];
    }
    o *= l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t at = row * D + 4 * lane;
    if constexpr (F32) {
        *(f32x4_t *)((float *)A.out + at) = o;
    } else {
        const f32x2_t lo = {o.x, o.y}, hi = {o.z, o.w};
        *(uint2 *)((uint16_t *)A.out + at) =
            make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2_t)),
                       __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2_t)));
    }
    if (A.lse != nullptr && threadIdx.x == 0)
        A.lse[row] = l == 0.0f ? -__builtin_inff()
                               : ((top == -__builtin_inff() ? 0.0f : top) +
                                  __builtin_amdgcn_logf(l)) * kLn2;
}

// ---- row tiles of 128 and 256 ------------------------------------------------------

typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16_t mfma32(bf16x8_t a, bf16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma32(f16x8_t a, f16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

constexpr int WIDE_SEGMENT = 2048;  // keys whose pages are held in LDS
// a segment's pages, and those a step that ends past it may ask for
constexpr int WIDE_PAGES = (WIDE_SEGMENT + 128) / 16;
constexpr uint32_t PAGE_MISSING = 1, PAGE_NAN = 2;

template <int D, int STEP>
struct WideShared {
    u32x4_t k[2][STEP * D / 8];  // bf16: [key][8 dimensions ^ swizzle]
    u32x4_t v[2][STEP * D / 8];  // fp16: [16 keys t][tile n][half h][lane m]: 8 keys of a dimension
    int64_t offset[WIDE_PAGES];        // a page's codes
    float k_operand[WIDE_PAGES], v_operand[WIDE_PAGES];
    float2 v_below[WIDE_PAGES];        // d and 2^d
    uint8_t bad[WIDE_PAGES];           // PAGE_*
    uint32_t v_top, special;           // special: some page of the segment is bad
    int nan[2];                        // the last step (its end) with NaN values taken out
};

// The chunk of a key row that LDS chunk c of the row holds: rows of D bytes
// that start in the same banks spread their chunks over all of them.
template <int D>
__device__ __forceinline__ int key_swizzle(int row) {
    return D % 128 == 0 ? row & 15 : (row >> 1) & 7;
}

// Row tiles of up to 32 WAVES query rows: chunks and whole prompts, bf16 queries.
//
// As above, but the waves share the keys and have 32 rows each: scores
// S^T = K Q^T and sums out^T = V^T P^T on 32 x 32 tiles, probabilities staying
// in their lanes.  A step of 16 WAVES keys is widened once for all waves on its
// way into LDS, keys to bf16, values transposed (eight keys of a dimension side by
// side) to fp16; its codes were loaded during the step before that.
//
// Bound by MFMA and vector issue of the two waves of a SIMD, and by the power they
// draw: 4 chunks of about 1024 tokens over 6000, 8 x 8 heads of 128, 905 us (930
// TFLOP/s, MFMA busy for 41% of the cycles and vector instructions for 46%, LDS for
// 30%, at a clock that falls to 1.94 GHz); a prompt of 4096, 8 x 4 heads, 151 us
// (910 TFLOP/s).  With the codes of a step loaded and stored in the same step 3 to
// 4% more.  Of 192 and 256 dimensions one wave a SIMD holds the sums in accumulation
// registers, and nothing covers what it waits for; of 256 it also spills 18 of its
// 512 registers.
//
// PAGES is how many pages 64 keys may have, 1 (of 64 tokens and more) or 4: four
// distances d cost the same two calls 2.3% over values that carry all of d
// themselves, one 1%.
template <int D, int WAVES, int PAGES>
__global__ __launch_bounds__(WAVES *WAVE, D <= 128 ? 2 : 1) void attention_wide_kernel(
    KvCache C, KvBatch B, AttnArgs A, int32_t *status) {
    constexpr int WG = WAVES * WAVE;
    constexpr int STEP = 16 * WAVES;         // keys of a step
    constexpr int KC = D / 16;               // 16-byte chunks of a key's codes
    constexpr int NT = D / 32;               // 32-dimension tiles of the output
    constexpr int W4 = D / 128, W2 = D % 128 / 64;  // a lane's words and half words of a value
    constexpr int KL = STEP * KC / WG;       // key chunks a thread loads
    static_assert(KL * WG == STEP * KC, "whole loads");
    __shared__ WideShared<D, STEP> sh;
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int r = lane & 31, h = lane >> 5;
    // workgroups in launch order: head, then row tile (the last, with the most
    // keys, first), then split
    const uint32_t hs = A.sub * C.heads;
    const int headsub = blockIdx.x % hs;
    const uint32_t rest = blockIdx.x / hs;
    const int split = rest / (uint32_t)A.items;
    const int item = A.items - 1 - (int)(rest - (uint32_t)split * A.items);
    const Item it = A.tokens > 1 && B.seqs < TILE_SEQS
                        ? find_tile(B, item, A.tokens, status)
                        : find_item(B, item, A.items, A.tokens, A.tokens > 1 ? 1 : 0,
                                    headsub == 0 && split == 0, status);
    const int row0 = it.piece * A.tokens;
    if (it.count <= 0 || row0 >= it.count) {
        if (it.count < 0 && threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
        return;
    }
    const int head = headsub / A.sub, sub = headsub - head * A.sub;
    Tile T;
    if (it.seq >= B.seqs) {
        T.tokens = min(A.tokens, it.count - row0);
        T.pos0 = T.base = T.first = T.end = 0;
    } else {
        T = tile_range(C, B, A, it, row0, status);
    }
    const int h0 = sub * A.sub_heads;
    const int hn = min(A.sub_heads, A.group - h0);
    const int row = 32 * wave + r;
    const int ri = row / hn, rh = row - ri * hn;
    const bool row_real = ri < T.tokens;
    const int64_t token = it.base + row0 + ri;
    const int hq = head * A.group + h0 + rh;
    const int64_t k0 = T.base + (int64_t)split * A.split_keys;
    const int64_t k1 = min(k0 + A.split_keys, T.end);
    const bool whole = T.end - T.base <= A.split_keys;
    if (k0 >= k1 && split > 0) return;

    // from here on keys count from k0, a page's first
    const int64_t pos = T.pos0 + ri;
    const int64_t last = row_real && A.causal ? pos : T.end - 1;
    const int64_t first = row_real && A.window > 0 ? pos - A.window + 1 : 0;
    const int keys = (int)max(k1 - k0, (int64_t)0);
    const int last_r = (int)max(min(last - k0, (int64_t)keys - 1), (int64_t)-1);
    const int first_r = (int)max(min(first - k0, (int64_t)keys), (int64_t)0);
    // the keys any row of this wave sees
    const int wave_last = (int)wave_max_u32(row_real ? (uint32_t)(last_r + 1) : 0u) - 1;
    const int wave_first = (int)wave_min_u32(row_real ? (uint32_t)first_r : 0x7FFFFFFFu);
    // the keys every row of the tile sees
    const int tile_last = (int)min((A.causal ? T.pos0 : T.end - 1) - k0, (int64_t)keys - 1);
    const int tile_first =
        A.window > 0 ? (int)max(min(T.pos0 + T.tokens - A.window - k0, (int64_t)keys), (int64_t)0) : 0;

    bf16x8_t q[KC];
    {
        const uint16_t *p = (const uint16_t *)A.q + token * A.q_token + hq * A.q_head + 8 * h;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (row_real) w = *(const uint4 *)(p + 16 * c);
            w.x ^= A.q_sign, w.y ^= A.q_sign, w.z ^= A.q_sign, w.w ^= A.q_sign;
            q[c] = __builtin_bit_cast(bf16x8_t, w);
        }
    }

    // the next step's codes, in registers
    u32x4_t kr[KL];
    float k_scale[KL];
    uint32_t vr[W4 + W2][8], any_nan = 0;
    float v_scale = 0.0f;
    const int vt = threadIdx.x >> 6;  // this thread's values: keys of group vt, half h, lane r
    const int slots = C.block - 1;
    bool special = false;
    // key and chunk of it that this thread's load i is
    auto key_of = [&](int i) {
        return WG % KC == 0 ? (int)threadIdx.x / KC + i * (WG / KC) : ((int)threadIdx.x + i * WG) / KC;
    };
    auto chunk_of = [&](int i) {
        return WG % KC == 0 ? (int)threadIdx.x % KC : ((int)threadIdx.x + i * WG) % KC;
    };
    auto load = [&](int j, int seg) {
#pragma unroll
        for (int i = 0; i < KL; ++i) {
            const int key = key_of(i);
            const int page = (j - seg + key) >> C.block_shift;
            const uint8_t *p = C.k_codes + sh.offset[page] +
                               (uint32_t)(((j + key) & slots) * D + 16 * chunk_of(i));
            k_scale[i] = sh.k_operand[page];
            kr[i] = *(const u32x4_t *)p;
        }
        const int page = (j - seg + 16 * vt) >> C.block_shift;
        const uint8_t *vp = C.v_codes + sh.offset[page] +
                            (uint32_t)((((j + 16 * vt) & slots) + 4 * h) * D);
        v_scale = sh.v_operand[page];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int at = (8 * (i / 4) + (i & 3)) * D;  // keys 4 h + 0..3, 8 + 4 h + 0..3
#pragma unroll
            for (int w = 0; w < W4; ++w) vr[w][i] = ((const uint32_t *)(vp + at + 128 * w))[r];
            if constexpr (W2 > 0) vr[W4][i] = ((const uint16_t *)(vp + at + 128 * W4))[r];
        }
        any_nan = 0;
    };
    // a step some of whose keys some row does not see
    auto edge = [&](int j) { return special || j < tile_first || j + STEP - 1 > tile_last; };
    auto clean = [&](int j, int seg) {
        // Values nothing sees are zeros, whatever the page holds there.  NaN
        // values of a step that not every row sees whole would reach rows
        // that do not see them (0 times NaN): they are taken out here and
        // marked afterwards.  Where every row sees them the sums do it by
        // themselves.
        const uint32_t bad = sh.bad[(j - seg + 16 * vt) >> C.block_shift];
        const uint32_t every = bad & PAGE_NAN ? 0x01010101u : 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int key = j + 16 * vt + 4 * h + 8 * (i / 4) + (i & 3);
            const bool none = key >= keys || (bad & PAGE_MISSING);
#pragma unroll
            for (int w = 0; w < W4 + W2; ++w) {
                const uint32_t x = vr[w][i];
                uint32_t z = ((((x & 0x7F7F7F7Fu) + 0x01010101u) >> 7) & 0x01010101u) | every;
                if (none) z = 0;
                vr[w][i] = none ? 0u : x & ~(z * 0xFFu);
                any_nan |= z;
            }
        }
    };
    // A step's way into LDS, in PIECES pieces that a caller puts between products.
    constexpr int PIECES = 2 * KL + 2 * (2 * W4 + W2);
    auto store = [&](int buf, int j, int piece) {
        if (piece < 2 * KL) {  // half a chunk of a key
            const int i = piece / 2, e = piece & 1;
            const int at = ((2 * chunk_of(i)) ^ key_swizzle<D>(key_of(i))) ^ e;
            sh.k[buf][key_of(i) * 2 * KC + at] =
                __builtin_bit_cast(u32x4_t, e ? widen_codes(kr[i].z, kr[i].w, k_scale[i])
                                              : widen_codes(kr[i].x, kr[i].y, k_scale[i]));
            return;
        }
        // a dimension of eight values: of dimensions n and n + 1 the bytes of two
        // keys lie in a half word each
        const int at = piece - 2 * KL, w = at / 4, n = at & 3;
        const uint32_t sel = n & 2 ? 0x07030602u : 0x05010400u;
        u32x4_t a;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t x = __builtin_amdgcn_perm(vr[w][2 * k + 1], vr[w][2 * k], sel);
            a[k] = __builtin_bit_cast(uint32_t,
                                      n & 1 ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, v_scale, true)
                                            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x, v_scale, false));
        }
        sh.v[buf][((vt * NT + 4 * w + n) * 2 + h) * 32 + r] = a;
        if (at == 0 && any_nan) sh.nan[buf] = j + STEP;
    };
    auto store_all = [&](int buf, int j) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) store(buf, j, i);
    };

    f32x16_t o[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n] = f32x16_t{};
    float m = -__builtin_inff(), l = 0.0f;

    // 64 keys, part `part` of the step at j0
    // `between(i)` runs after product i of the scores
    auto compute = [&](int buf, int j0, int part, int seg, auto between) {
        const int j = j0 + 64 * part;
        f32x16_t s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) s[u] = f32x16_t{};
        __builtin_amdgcn_s_setprio(1);
        // product i: dimensions 16 (i / 2) .., keys 32 (i & 1) ..; its keys are read
        // AHEAD products before it.  Their addresses differ in the swizzled bits:
        // computed here, as all of them over the loop take more registers than
        // there are (256 dimensions).
        constexpr int AHEAD = 6;
        constexpr int SPAN = D % 128 == 0 ? 8 : 4;  // products of one row whose addresses differ
        uint32_t k_bits = (uint32_t)(h ^ key_swizzle<D>(r)) * 16;
        const uint32_t k_row = (uint32_t)((buf * STEP + 64 * part + r) * 2 * D);
        asm volatile("" : "+v"(k_bits));
        auto key = [&](int i) {
            const int c = i / 2;
            const uint32_t at = (k_bits ^ (uint32_t)(c % SPAN * 32)) + k_row;
            return *(const u32x4_t *)((const char *)sh.k + at + c / SPAN * SPAN * 32 +
                                      (i & 1) * 32 * 2 * D);
        };
        u32x4_t kf[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) kf[i] = key(i);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 2 * KC; ++i) {
            s[i & 1] = mfma32(__builtin_bit_cast(bf16x8_t, kf[i % AHEAD]), q[i / 2], s[i & 1]);
            if (i + AHEAD < 2 * KC) kf[i % AHEAD] = key(i + AHEAD);
            between(i);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_setprio(0);
        // the base-2 scores are s c2
        float c2 = A.scale2;
        const bool clean = j >= first_r && j + 63 <= last_r && !special;
        if (__ballot(!clean) != 0) {
            c2 = 1.0f;
            uint32_t missing = 0;  // a bit for each 16-key group
            if (special)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    missing |= (uint32_t)(sh.bad[(j - seg + 16 * t) >> C.block_shift] & PAGE_MISSING) << t;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = j + 32 * u + 8 * (i / 4) + 4 * h + (i & 3);
                    const bool in = key >= first_r && key <= last_r && !((missing >> (2 * u + i / 8)) & 1u);
                    s[u][i] = in ? s[u][i] * A.scale2 : -__builtin_inff();
                }
        }
        const u32x4_t *vp = &sh.v[buf][(4 * part * NT * 2 + h) * 32 + r];
        u32x4_t vf[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) vf[n] = vp[n * 64];
        float2 below[PAGES];
#pragma unroll
        for (int t = 0; t < PAGES; ++t)
            below[t] = sh.v_below[(j - seg + 64 / PAGES * t) >> C.block_shift];
        float top = s[0][0];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = __builtin_fmaxf(top, s[u][i]);
        if (__ballot(top * c2 > m + kRaiseAbove) != 0) {  // some weight may (d is not negative)
            top = -__builtin_inff();
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    top = __builtin_fmaxf(
                        top, __builtin_fmaf(s[t / 2][8 * (t & 1) + i], c2, -below[t * PAGES / 4].x));
            top = __builtin_fmaxf(top, __shfl_xor(top, 32, WAVE));
            const float next = __builtin_fmaxf(m, top - kRaiseTo);
            const float keep = m == next ? 1.0f : __builtin_amdgcn_exp2f(m - next);
            m = next;
            l *= keep;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n] *= keep;
        }
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        // The probabilities of 16 keys are computed between the products of the
        // 16 before, and a product's values are read as soon as the last one
        // has taken its own.
        float p[8];
        auto probability = [&](int t, int i) {
            p[i] = __builtin_amdgcn_exp2f(
                __builtin_fmaf(s[t / 2][8 * (t & 1) + i], c2, -(ref + below[t * PAGES / 4].x)));
            l = __builtin_fmaf(p[i], below[t * PAGES / 4].y, l);
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) probability(0, i);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const f16x8_t pb = split_parts<f16x8_t, 1>(p).p[0];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                o[n] = mfma32(__builtin_bit_cast(f16x8_t, vf[n]), pb, o[n]);
                if (t < 3) {
                    vf[n] = vp[(t + 1) * NT * 64 + n * 64];
#pragma unroll
                    for (int i = 8 * n / NT; i < 8 * (n + 1) / NT; ++i) probability(t + 1, i);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    // A step whose NaN values were taken out: NaN where a row sees one.  A
    // product of where they are with who sees them counts them.
    auto mark_nan = [&](int j, int seg) {
#pragma unroll 1
        for (int t = 0; t < WAVES; ++t) {
            const int page = (j - seg + 16 * t) >> C.block_shift;
            if (j + 16 * t >= keys || (sh.bad[page] & PAGE_MISSING)) continue;
            const bool every = sh.bad[page] & PAGE_NAN;
            const uint8_t *codes = C.v_codes + sh.offset[page] + ((j + 16 * t) & slots) * D;
            float seen[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int key = j + 16 * t + 8 * (i / 4) + 4 * h + (i & 3);
                seen[i] = key >= first_r && key <= last_r ? 1.0f : 0.0f;
            }
            const f16x8_t sb = split_parts<f16x8_t, 1>(seen).p[0];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int d = n < 4 * W4 ? 128 * (n / 4) + 4 * r + (n & 3) : 128 * W4 + 2 * r + (n & 1);
                f16x8_t a;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int c = codes[(8 * (i / 4) + 4 * h + (i & 3)) * D + d];
                    a[i] = every || (c & 127) == 127 ? 1.0f : 0.0f;
                }
                const f32x16_t count = mfma32(a, sb, f32x16_t{});
#pragma unroll
                for (int i = 0; i < 16; ++i)  // a count is 0 or positive: its negated bits' sign
                    o[n][i] = u2f(f2u(o[n][i]) | ((uint32_t)((int)-f2u(count[i]) >> 31) & 0x7FC00000u));
            }
        }
    };

    // the largest value scale (of one segment it is found with its pages)
    uint32_t v_top = 0;
    if (keys > WIDE_SEGMENT) {
        if (threadIdx.x == 0) sh.v_top = 0;
        __syncthreads();
        const int pages = (keys + slots) >> C.block_shift;
#pragma unroll 4
        for (int i = threadIdx.x; i < pages; i += WG) {
            const int page = find_page(B, C, it.seq, (k0 >> C.block_shift) + i);
            const uint32_t vb = page < 0 ? 0u : C.v_scales[(int64_t)page * C.heads + head];
            if (vb != 255u) v_top = max(v_top, vb);
        }
        if (v_top > 0) atomicMax(&sh.v_top, v_top);
        __syncthreads();
        v_top = __builtin_amdgcn_readfirstlane(sh.v_top);
    }
    // a window may start inside its first page
    const int start = (int)max(min(T.first - k0, (int64_t)keys), (int64_t)0) / STEP * STEP;
    for (int seg = start / WIDE_SEGMENT * WIDE_SEGMENT; seg < keys; seg += WIDE_SEGMENT) {
        const int seg_end = min(seg + WIDE_SEGMENT, keys);
        const int64_t b0 = (k0 + seg) >> C.block_shift;
        const int pages = (seg_end - seg + slots) >> C.block_shift;
        __syncthreads();  // the last segment's pages are done with
        if (threadIdx.x == 0) {
            sh.v_top = v_top;
            sh.special = sh.nan[0] = sh.nan[1] = 0;
        }
        __syncthreads();
        uint32_t kb = 0, vb = 0;
        if (threadIdx.x < WIDE_PAGES) {  // past the segment's pages, the last again
            const int page = find_page(B, C, it.seq, b0 + min((int)threadIdx.x, pages - 1));
            uint32_t bad = page < 0 ? PAGE_MISSING : 0u;
            if (page >= 0) {
                const int64_t at = (int64_t)page * C.heads + head;
                kb = C.k_scales[at], vb = C.v_scales[at];
                if (vb == 255u) bad = PAGE_NAN, vb = 0;
            }
            sh.offset[threadIdx.x] = page_offset(C, max(page, 0), head);
            sh.k_operand[threadIdx.x] = e8m0_operand(kb);
            sh.bad[threadIdx.x] = (uint8_t)bad;
            if (bad) sh.special = 1;
            if (bad & PAGE_MISSING) flag(status, FLAG_CACHE_INDEX);
            if (vb > v_top) atomicMax(&sh.v_top, vb);
        }
        __syncthreads();
        v_top = __builtin_amdgcn_readfirstlane(sh.v_top);
        special = __builtin_amdgcn_readfirstlane(sh.special) != 0;
        if (threadIdx.x < WIDE_PAGES) {
            const int below = v_below(vb, v_top);
            sh.v_operand[threadIdx.x] = v_operand(vb, v_top);
            sh.v_below[threadIdx.x] = make_float2((float)below, v_lift(below));
        }
        __syncthreads();
        int buf = 0, j = max(seg, start);
        load(j, seg);
        if (edge(j)) clean(j, seg);
        store_all(0, j);
        if (j + STEP < seg_end) load(j + STEP, seg);
        __syncthreads();
        for (; j < seg_end; j += STEP) {
            // The next step's codes are in registers.  They are stored between the
            // products of the last part; then the step after it is on its way, and
            // has until the next step's last part.
            const bool more = j + STEP < seg_end, load_more = j + 2 * STEP < seg_end;
            if (more && edge(j + STEP)) clean(j + STEP, seg);
#pragma unroll 1
            for (int part = 0; part < STEP / 64 - 1; ++part)
                if (j + 64 * part <= wave_last && j + 64 * part + 63 >= wave_first)
                    compute(buf, j, part, seg, [](int) {});
            const int part = STEP / 64 - 1;
            if (j + 64 * part <= wave_last && j + 64 * part + 63 >= wave_first) {
                if (more)
                    compute(buf, j, part, seg, [&](int i) {
                        constexpr int EACH = (PIECES + 2 * KC - 1) / (2 * KC);
#pragma unroll
                        for (int e = EACH * i; e < EACH * (i + 1); ++e)
                            if (e < PIECES) store(buf ^ 1, j + STEP, e);
                        if (i == (PIECES + EACH - 1) / EACH - 1 && load_more)
                            load(j + 2 * STEP, seg);
                    });
                else
                    compute(buf, j, part, seg, [](int) {});
            } else if (more) {
                store_all(buf ^ 1, j + STEP);
                if (load_more) load(j + 2 * STEP, seg);
            }
            if (sh.nan[buf] == j + STEP) mark_nan(j, seg);
            __syncthreads();
            buf ^= 1;
        }
    }

    if (!row_real) return;
    l += __shfl_xor(l, 32, WAVE);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int back = (int)v_top - (int)E8M0_ONE - kVBias;
    const int64_t to = token * A.heads + hq;
#pragma unroll
    for (int w = 0; w < W4 + W2; ++w)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            // 4 (of a half word 2) dimensions side by side
            const int mm = 8 * (i / 4) + 4 * h + (i & 3);
            const int d = 128 * w + (w < W4 ? 4 : 2) * mm;
            f32x4_t y = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < (w < W4 ? 4 : 2); ++k)
                y[k] = __builtin_ldexpf(o[4 * w + k][i] * inv, back);
            const f32x2_t lo = {y.x, y.y}, hi = {y.z, y.w};
            if (!whole) {
                float *p = A.part_o + (to * A.splits + split) * D + d;
                *(f32x2_t *)p = lo;
                if (w < W4) *(f32x2_t *)(p + 2) = hi;
            } else {
                uint32_t *p = (uint32_t *)((uint16_t *)A.out + to * D + d);
                p[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2_t));
                if (w < W4) p[1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2_t));
            }
        }
    if (h == 0) {
        if (!whole)
            A.part_ml[to * A.splits + split] = split_weight(m, l);
        else if (A.lse != nullptr)
            A.lse[to] = l == 0.0f ? -__builtin_inff()
                                  : ((m == -__builtin_inff() ? 0.0f : m) + __builtin_amdgcn_logf(l)) * kLn2;
    }
}

// How a call is laid out: from its shapes alone, which the workspace's size
// needs too.
struct Plan {
    int wide;   // waves of a wide workgroup, 0 for narrow tiles
    int waves;  // of a narrow workgroup
    int sub, sub_heads, tokens, splits, split_keys;
    int64_t items;
};

constexpr int CUS = 256;

Plan make_plan(const KvCache &C, const KvBatch &B, int heads, int window, bool bf16) {
    Plan P;
    const int group = heads / C.heads;
    const int64_t per = (B.tokens + B.seqs - 1) / B.seqs;  // new tokens of a sequence, on average
    int64_t extent = (int64_t)B.width << C.block_shift;
    if (window > 0) extent = std::min<int64_t>(extent, (int64_t)window + per + C.block);
    // Which kernel: narrow tiles for few rows of a sequence and kv head (narrow
    // against wide; of 64 dimensions 96 rows 112 and 156 us, 160 rows 158 and 136;
    // of 128 64 rows 45 and 55, 160 rows 307 and 188; of 256 56 rows 58 and 115, 120
    // rows 191 and 144), and where a CU has up to two of them and 2048 of their keys
    // (2 prompts of 433 tokens, 4 heads: 13 us and 21; 3 chunks of 116 tokens, 8
    // heads, over 1212 keys: 20 and 31; but 119 tokens, 16 x 7 heads, four for each
    // CU: 29 and 18).  Tiles of 256 rows once there are two for
    // each CU (4 chunks of 1024 tokens: 980 us with tiles of 128, 911; 8 of 64 tokens,
    // one tile for each four CUs: 130, 187).  fp32 queries have no wide kernel.
    const int64_t narrow_tiles = (per * group + 15) / 16 * B.seqs * C.heads;
    P.wide = 0;
    if (bf16 && per * group > (C.dim == 64 ? 128 : C.dim == 128 ? 64 : 96) &&
        (narrow_tiles > 2 * CUS || narrow_tiles * extent > 2048 * CUS))
        P.wide = C.dim <= 128 && per * group >= 256 && B.tokens * heads >= 2 * CUS * 256 ? 8 : 4;
    const int rows = P.wide ? 32 * P.wide : 16;
    P.sub = (group + rows - 1) / rows;
    P.sub_heads = (group + P.sub - 1) / P.sub;
    P.tokens = (int)std::min<int64_t>(rows / P.sub_heads, per);
    P.items = P.tokens > 1 ? item_count(B.tokens, B.seqs, P.tokens, 1) : B.tokens;
    if (window > 0) extent = std::min<int64_t>(extent, (int64_t)window + P.tokens + C.block);
    const int64_t tiles = (per + P.tokens - 1) / P.tokens * B.seqs * C.heads * P.sub;
    int64_t keys;
    P.waves = 0;
    if (P.wide) {
        auto split = [&](int64_t slots, int64_t least) {
            const int64_t want = std::max<int64_t>(1, slots / tiles);
            return std::max<int64_t>((extent + want - 1) / want, least);
        };
        // One workgroup a CU down to splits of 512 keys (3 chunks of 116 tokens, 8
        // heads, 1212 keys: 31 us; not below 1024 39, nor below 256 29, but 2 of 285
        // tokens then 30 against 25).  Two a CU, where they fit, down to 1024 (8 x 4
        // tokens x 4096 keys: 41 us, of 512 keys 47).  Those of four waves fit to 128
        // dimensions (4 chunks of 100 tokens of 192 dimensions over 4096 keys, split
        // as if they fitted: 109 us, 82).
        keys = split(CUS, 512);
        if (P.wide == 4 && C.dim <= 128) keys = std::min(keys, split(2 * CUS, 1024));
        keys = (keys + 255) / 256 * 256;  // whole pages and steps
    } else {
        // few tiles: workgroups of 8 waves, one a CU (of 16 where 64 dimensions
        // take half the registers); else of 4, two a CU.  Many tiles are split until
        // three workgroups wait for each place: sequences differ in length.  Splits
        // are as long as that leaves them, up to 16384 keys (64 sequences x 20000
        // keys of 256 dimensions: 494 us; up to 8192 514, up to 4096 539); six steps
        // of a workgroup are not split (1000 keys: 14.1 us, in four 14.8).
        P.waves = tiles > CUS || (!bf16 && C.dim == 256) ? 4 : C.dim == 64 ? (bf16 ? 16 : 12) : 8;
        const int64_t slots = tiles > CUS && (bf16 || C.dim < 256) ? 2 * CUS : CUS;
        const int64_t want = tiles <= slots ? slots / tiles : (3 * slots + tiles - 1) / tiles;
        keys = (extent + want - 1) / want;
        if (extent <= 6 * 32 * P.waves) keys = extent;
        keys = (keys + 255) / 256 * 256;  // whole pages and steps
        keys = std::min<int64_t>(keys, std::min<int64_t>(NARROW_PAGES * C.block, 16384));
    }
    P.split_keys = (int)keys;
    P.splits = (int)((extent + keys - 1) / keys);
    return P;
}

}  // namespace

size_t attention_workspace_bytes(const KvCache &C, const KvBatch &B, int heads, int window,
                                 bool bf16) {
    const Plan P = make_plan(C, B, heads, window, bf16);
    if (P.splits <= 1) return 0;
    // tokens, heads and splits are at most 2^23, 2^16 and 2^15: the last factor
    // may pass 64 bits
    size_t bytes = 0;
    if (__builtin_mul_overflow((size_t)B.tokens * heads * P.splits,
                               (size_t)(C.dim + 2) * sizeof(float), &bytes))
        return SIZE_MAX;
    return bytes;
}

template <int D>
static hipError_t launch_dim(const KvCache &C, const KvBatch &B, const AttnArgs &A, const Plan &P,
                       bool bf16, int32_t *status, hipStream_t s) {
    if (P.wide) {
        void (*kernel)(KvCache, KvBatch, AttnArgs, int32_t *) =
            C.block >= 64 ? attention_wide_kernel<D, 4, 1> : attention_wide_kernel<D, 4, 4>;
        if constexpr (D <= 128)
            if (P.wide == 8)
                kernel = C.block >= 64 ? attention_wide_kernel<D, 8, 1> : attention_wide_kernel<D, 8, 4>;
        const int64_t groups = P.items * C.heads * P.sub * P.splits;
        if (groups * P.wide * WAVE > UINT32_MAX) return hipErrorInvalidConfiguration;
        hipLaunchKernelGGL(kernel, dim3((uint32_t)groups), dim3(P.wide * WAVE), 0, s, C, B, A,
                           status);
    } else {
        void (*kernel)(KvCache, KvBatch, AttnArgs, int32_t *) =
            bf16 ? (P.waves == 4 ? attention_narrow_kernel<D, false, 4>
                                 : attention_narrow_kernel<D, false, kNarrowMany<D, false>>)
                 : (P.waves == 4 ? attention_narrow_kernel<D, true, 4>
                                 : attention_narrow_kernel<D, true, kNarrowMany<D, true>>);
        const uint32_t hs = C.heads * P.sub, items = (uint32_t)P.items;
        hipLaunchKernelGGL(kernel, (items <= NARROW_GRID_Y ? dim3(hs, items, P.splits) : dim3(items, hs, P.splits)),
                           dim3(P.waves * WAVE), 0, s, C, B, A, status);
    }
    if (P.splits > 1)
        hipLaunchKernelGGL((bf16 ? attention_join_kernel<D, false> : attention_join_kernel<D, true>),
                           dim3((uint32_t)B.tokens, A.heads), dim3(JOIN_WG), 0, s, C, B, A);
    return hipGetLastError();
}

hipError_t launch_attention(const KvCache &C, const KvBatch &B, const void *q, int64_t q_token,
                            int64_t q_head, bool bf16, int heads, float scale, bool causal,
                            int window, void *out, float *lse, void *workspace, int32_t *status,
                            hipStream_t s) {
    const Plan P = make_plan(C, B, heads, window, bf16);
    AttnArgs A{};
    A.q = q, A.q_token = q_token, A.q_head = q_head, A.out = out, A.lse = lse;
    A.part_o = (float *)workspace;
    A.part_ml = (float2 *)(A.part_o + (size_t)B.tokens * heads * P.splits * C.dim);
    A.heads = heads, A.group = heads / C.heads, A.causal = causal, A.window = window;
    A.sub = P.sub, A.sub_heads = P.sub_heads, A.items = (int)P.items, A.tokens = P.tokens;
    A.splits = P.splits, A.split_keys = P.split_keys;
    A.scale2 = (scale < 0.0f ? -scale : scale) * kLog2e;
    A.q_sign = scale < 0.0f ? (bf16 ? 0x80008000u : 0x80000000u) : 0u;
    switch (C.dim) {
        case 64: return launch_dim<64>(C, B, A, P, bf16, status, s);
        case 128: return launch_dim<128>(C, B, A, P, bf16, status, s);
        case 192: return launch_dim<192>(C, B, A, P, bf16, status, s);
        default: return launch_dim<256>(C, B, A, P, bf16, status, s);
    }
}

}  // namespace fp4dev

// fp4_w4.h - products of wide activations with FP4 weights on the bf16 MFMA:
// weights decoded in registers, activations exact.  Internal to libfp4.so.
//
// A wave multiplies 16 weight rows at a time with up to 16 activation rows:
// v_mfma_f32_16x16x32_bf16 with the weight as its first operand, so that a lane
// l = 16 g + r of it holds 8 values of K of weight row r (g = l / 16 says which),
// and of activation row r as the second operand, and gets the sums of activation
// row r with weight rows 4 g .. 4 g + 3.  Which 8 values of K a lane holds is free
// as long as both operands agree: a lane takes the 16 bytes of codes of one
// 32-value stretch of its row (one load), and four products use 8 values each.
//
// Values: E2M1 times the block's scale is exact in bf16: MXFP4's converter applies
// its power of two, NVFP4's E4M3 scale makes products of at most six significant
// bits.  bf16 activations multiply as they are; fp32 ones are three bf16 terms of 8
// bits each, all 24 where the last is not below 2^-133, bf16's smallest, so from 2^-110 on.
// Sums are fp32.
#pragma once

#include <type_traits>

#include "fp4_device.h"

namespace fp4dev {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// f(0), .. f(N - 1), the index a constant in each.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void unroll(const F &f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>());
        unroll<N, I + 1>(f);
    }
}

constexpr int W4_STRETCH = 128;  // values of K that a load of 16 rows' codes covers

// A lane's part of 16 rows' stretch: the codes of 32 values of its row, and their
// scale bytes (MXFP4 one, NVFP4 two).
struct W4Unit {
    u32x4_t codes;
    uint32_t scale;
};

// NaN scale bytes of MXFP4 (255) are no operand of the converter: the largest
// byte seen tells whether a lane's row had one.
__device__ __forceinline__ bf16x8_t w4_values(uint32_t codes, float scale) {
    const bf16x2_t r[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2),
                           __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3)};
    bf16x8_t v;
    __builtin_memcpy(&v, r, sizeof(v));
    return v;
}

// Two fp32 values that bf16 holds exactly.
__device__ __forceinline__ uint32_t bf16_exact(float a, float b) {
    return __builtin_amdgcn_perm(f2u(b), f2u(a), 0x07060302u);
}

__device__ __forceinline__ bf16x8_t w4_values_e4m3(uint32_t codes, float s) {
    const f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2),
                          __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = bf16_exact(p[i].x * s, p[i].y * s);
    bf16x8_t v;
    __builtin_memcpy(&v, r, sizeof(v));
    return v;
}

// Values 8 i .. 8 i + 7 of a lane's 32.
template <int FMT>
__device__ __forceinline__ bf16x8_t w4_decode(const W4Unit &u, int i) {
    if constexpr (FMT == 0) {
        return w4_values(u.codes[i], e8m0_operand(u.scale));
    } else {
        return w4_values_e4m3(u.codes[i], i < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)u.scale, 0)
                                                : __builtin_amdgcn_cvt_f32_fp8((int)u.scale, 1));
    }
}

template <int N>
struct Terms {
    bf16x8_t p[N];
};

// Four fp32 values as three bf16 terms each: a value's upper 16 bits, those of what
// they leave, and the rest (differences are exact, and nothing overflows).  Of a value
// that is not finite the first term is right, the others are NaN.
__device__ __forceinline__ void split_finite_f32x4(const float (&x)[4], u32x2_t (&t)[3]) {
    float rest[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) rest[i] = x[i];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        t[k] = {__builtin_amdgcn_perm(f2u(rest[1]), f2u(rest[0]), 0x07060302u),
                __builtin_amdgcn_perm(f2u(rest[3]), f2u(rest[2]), 0x07060302u)};
#pragma unroll
        for (int i = 0; i < 4; ++i) rest[i] = rest[i] - u2f(f2u(rest[i]) & 0xFFFF0000u);
    }
}
// The same of any values: one that is not finite is its first term alone.
__device__ __forceinline__ void split_f32x4(const float (&x)[4], u32x2_t (&t)[3]) {
    split_finite_f32x4(x, t);
    const uint32_t top = max(max(f2u(x[0]) & 0x7FFFFFFFu, f2u(x[1]) & 0x7FFFFFFFu),
                             max(f2u(x[2]) & 0x7FFFFFFFu, f2u(x[3]) & 0x7FFFFFFFu));
    if (top >= 0x7F800000u) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = f2u(x[i]), a = b & 0x7FFFFFFFu, shift = 16 * (i & 1);
            if (a < 0x7F800000u) continue;
            const uint32_t keep = ~(0xFFFFu << shift);
            const uint32_t first = a > 0x7F800000u ? 0x7FC0u : b >> 16;
            t[0][i / 2] = (t[0][i / 2] & keep) | first << shift;
            t[1][i / 2] &= keep;
            t[2][i / 2] &= keep;
        }
    }
}

// Eight activations from memory: bf16 as they are, fp32 in three terms.
__device__ __forceinline__ Terms<1> load_terms(const uint16_t *p) {
    return {__builtin_bit_cast(bf16x8_t, *(const uint4 *)p)};
}
__device__ __forceinline__ Terms<3> load_terms(const float *p) {
    u32x2_t t[2][3];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float4 v = ((const float4 *)p)[h];
        const float x[4] = {v.x, v.y, v.z, v.w};
        split_f32x4(x, t[h]);
    }
    Terms<3> r;
#pragma unroll
    for (int n = 0; n < 3; ++n) {
        const u32x4_t w = {t[0][n].x, t[0][n].y, t[1][n].x, t[1][n].y};
        r.p[n] = __builtin_bit_cast(bf16x8_t, w);
    }
    return r;
}

__device__ __forceinline__ f32x4_t mfma_w4(bf16x8_t w, bf16x8_t x, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
}

// What a wave's lanes put into LDS for each other, in order: those before are there for
// those after.  The hardware keeps the order of a wave's LDS operations; this keeps the
// compiler from changing it, and is no instruction.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// ---- loads ------------------------------------------------------------------
// Buffer loads: past the end of what the resource spans they give zeros and move
// nothing, so that a pipeline's loads need no branches (around which the waits for
// them would lose count).
typedef __amdgpu_buffer_rsrc_t Rsrc;
// Resources are below 2^30 bytes: an offset of 2^31 is past any.
constexpr uint32_t NOWHERE = 0x80000000u;
constexpr int STREAMED = 2;  // cache policy: nontemporal

// bytes, alike in all lanes, is made a scalar: the compiler clamps in vector registers,
// and then every load loops over what it takes for different resources.
__device__ __forceinline__ Rsrc span(const void *p, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0,
                                             __builtin_amdgcn_readfirstlane(bytes),
                                             kBufferRsrcWord3);
}
__device__ __forceinline__ u32x4_t load16(Rsrc r, uint32_t at) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, 0);
}
__device__ __forceinline__ u32x4_t load16_streamed(Rsrc r, uint32_t at) {
    return __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, STREAMED);
}

// A wave takes K in groups of 512 values, four stretches; it loads weights by pairs of
// stretches, 128 bytes of a row, and a group's scales at once.  Loads are laid out for
// the memory: lanes next to each other have what is next to each other, a load has whole
// lines, and a line is loaded by one wave.  (With lanes in the products' order, where
// neighbours have different rows, 16 tokens through 8192 x 28672 in NVFP4 took 70 us, not
// 39; with stretches of 64 bytes and scales a stretch at a time, lines that several waves
// wait for, 50.)  What K has past its last whole group is load_tail's: groups cut by the
// rows' end cost K of whole groups 2 to 25 %, and as an instantiation of their own gained
// as often as they lost.
constexpr int W4_GROUP = 4 * W4_STRETCH;

// PARTS parts of 16 rows of row-major weights, codes [rows, K/2] and scales [rows,
// K/block].  A pair's load n has rows 8 n .. 8 n + 7, eight lanes a row.
template <int FMT, int PARTS>
struct RowsAt {
    static constexpr int LDS = 128 + PARTS * (FMT == 0 ? 16 : 32);  // pieces of a wave
    struct Pair {
        u32x4_t v[2 * PARTS];
    };
    static constexpr int EACH = FMT == 0 ? 1 : 2;                       // scale pieces of a row
    static constexpr int SCALE_LOADS = (16 * PARTS * EACH + WAVE - 1) / WAVE;
    struct Scales {
        u32x4_t v[SCALE_LOADS];
    };
    Rsrc codes, scales;
    uint32_t code[2 * PARTS], scale[SCALE_LOADS];
    u32x4_t *lds;  // the wave's: [row][8 pieces of a pair], [part][row] scales

    // rows: of those from row0 on, how many there are; part p has rows row0 + p *
    // part_rows + 0 .. 15; base: of row row0.
    __device__ __forceinline__ RowsAt(const uint8_t *code_base, const uint8_t *scale_base, int rows,
                                      int part_rows, int K, u32x4_t *wave_lds)
        : lds(wave_lds) {
        constexpr int BLK = FMT == 0 ? 32 : 16;
        const int lane = threadIdx.x & (WAVE - 1);
        const int code_row = (uint32_t)K / 2, scale_row = (uint32_t)K / BLK;
        const int have = min(rows, (PARTS - 1) * part_rows + 16);
        codes = span(code_base, have * code_row);
        scales = span(scale_base, have * scale_row);
#pragma unroll
        for (int n = 0; n < 2 * PARTS; ++n)
            code[n] = (uint32_t)(n / 2 * part_rows + n % 2 * 8 + (lane >> 3)) * (uint32_t)code_row +
                      16 * (lane & 7);
#pragma unroll
        for (int n = 0; n < SCALE_LOADS; ++n) {
            const int row = (n * WAVE + lane) / EACH;
            scale[n] = row < 16 * PARTS
                           ? (uint32_t)(row / 16 * part_rows + row % 16) * (uint32_t)scale_row +
                                 16 * (lane % EACH)
                           : NOWHERE;
        }
    }
    // of the group or pair at k (a group past the end: NOWHERE)
    __device__ __forceinline__ Scales load_scales(uint32_t k) const {
        Scales s;
#pragma unroll
        for (int n = 0; n < SCALE_LOADS; ++n)
            s.v[n] = load16(scales, scale[n] + (k == NOWHERE ? k / 2 : k / (FMT == 0 ? 32 : 16)));
        return s;
    }
    __device__ __forceinline__ Pair load_pair(uint32_t k) const {
        Pair r;
#pragma unroll
        for (int n = 0; n < 2 * PARTS; ++n)
            r.v[n] = load16_streamed(codes, code[n] + (k == NOWHERE ? k : k / 2));
        return r;
    }
    __device__ __forceinline__ void put(const Scales &s) const {
        const int lane = threadIdx.x & (WAVE - 1);
#pragma unroll
        for (int n = 0; n < SCALE_LOADS; ++n)
            if (n * WAVE + lane < 16 * PARTS * EACH) lds[128 + n * WAVE + lane] = s.v[n];
    }
    // to the products' order, v[PARTS * stretch + part]: piece v of row r goes through
    // 8 r + (v ^ r), which spreads what is written and what is read over the banks.  Also
    // orders scales that were put before it; the next pair's spread, and the next put, want
    // a barrier or wave_order after the last use of this one's.
    __device__ __forceinline__ void spread(Pair &pair) const {
        const int lane = threadIdx.x & (WAVE - 1), r = lane & 15, g = lane >> 4;
        u32x4_t in[2 * PARTS];
#pragma unroll
        for (int n = 0; n < 2 * PARTS; ++n) in[n] = pair.v[n];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
#pragma unroll
            for (int n = 0; n < 2; ++n) lds[64 * n + (lane ^ (lane >> 3))] = in[2 * p + n];
            wave_order();
#pragma unroll
            for (int h = 0; h < 2; ++h) pair.v[PARTS * h + p] = lds[8 * r + ((4 * h + g) ^ (r & 7))];
            if (p + 1 < PARTS) wave_order();
        }
    }
    // stretch j of the group, of a spread pair
    __device__ __forceinline__ void units(const Scales &, const Pair &pair, int j,
                                          W4Unit (&w)[PARTS]) const {
        const int lane = threadIdx.x & (WAVE - 1), r = lane & 15, g = lane >> 4;
        const uint8_t *s = (const uint8_t *)(lds + 128);
#pragma unroll
        for (int p = 0; p < PARTS; ++p) {
            w[p].codes = pair.v[PARTS * (j & 1) + p];
            if constexpr (FMT == 0) w[p].scale = s[(16 * p + r) * 16 + 4 * j + g];
            else w[p].scale = ((const uint16_t *)s)[(16 * p + r) * 16 + 4 * j + g];
        }
    }
};

// Row tiles of 32, two parts each, of a packed operand: a load has 32 rows, 32 values of
// each of two, rows l % 32 and values 32 (l / 32) .. of a K step.  Exchanging odd groups
// of 16 lanes of one step with even ones of the next gives a register rows 0 .. 15 and
// another rows 16 .. 31, with the 32s 0, 2, 1, 3 of the stretch in lane groups 0 .. 3.
__device__ __forceinline__ int packed_group(int g) { return (g & 1) * 2 + (g >> 1); }

__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

template <int FMT, int PARTS>
struct PackedAt {
    static constexpr int LDS = 0, TILES = PARTS / 2;
    struct Pair {
        u32x4_t v[2 * PARTS];  // [tile][K step], spread [stretch][part]
    };
    struct Scales {
        std::conditional_t<FMT == 0, u32x2_t, u32x4_t> v[TILES];
    };
    Rsrc codes, scales;
    uint32_t code_tile, scale_tile;

    // rows: of those from the base on, how many there are
    __device__ __forceinline__ PackedAt(const uint8_t *code_base, const uint8_t *scale_base, int rows,
                                        int K)
        : code_tile(16 * K), scale_tile(FMT == 0 ? K : 2 * K) {
        const int have = min((rows + 31) / 32, TILES);
        codes = span(code_base, have * (int)code_tile);
        scales = span(scale_base, have * (int)scale_tile);
    }
    __device__ __forceinline__ Scales load_scales(uint32_t k) const {
        const int lane = threadIdx.x & (WAVE - 1);
        Scales s;
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            if constexpr (FMT == 0)
                s.v[t] = __builtin_bit_cast(
                    u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(
                                 scales, (int)(k + t * scale_tile + 8 * lane), 0, 0));
            else
                s.v[t] = load16(scales, (k == NOWHERE ? k : 2 * k) + t * scale_tile + 16 * lane);
        }
        return s;
    }
    __device__ __forceinline__ Pair load_pair(uint32_t k) const {
        const int lane = threadIdx.x & (WAVE - 1);
        Pair r;
#pragma unroll
        for (int n = 0; n < 2 * PARTS; ++n)
            r.v[n] = load16_streamed(codes, (k == NOWHERE ? k : 16 * k) + n / 4 * code_tile +
                                                1024 * (n & 3) + 16 * lane);
        return r;
    }
    __device__ __forceinline__ void put(const Scales &) const {}
    __device__ __forceinline__ void spread(Pair &pair) const {
        u32x4_t out[2 * PARTS];
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t x = pair.v[4 * t + 2 * h][i], y = pair.v[4 * t + 2 * h + 1][i];
                    swap16(x, y);
                    out[PARTS * h + 2 * t][i] = x;
                    out[PARTS * h + 2 * t + 1][i] = y;
                }
#pragma unroll
        for (int n = 0; n < 2 * PARTS; ++n) pair.v[n] = out[n];
    }
    __device__ __forceinline__ void units(const Scales &s, const Pair &pair, int j,
                                          W4Unit (&w)[PARTS]) const {
        const int odd = (threadIdx.x >> 4) & 1, by = FMT == 0 ? 16 * (j & 1) + 8 * odd : 16 * odd;
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            uint32_t s0 = s.v[t][FMT == 0 ? j / 2 : j], s1 = s0;
            swap16(s0, s1);
            w[2 * t] = {pair.v[PARTS * (j & 1) + 2 * t], FMT == 0 ? (s0 >> by) & 0xFFu : s0 >> by};
            w[2 * t + 1] = {pair.v[PARTS * (j & 1) + 2 * t + 1],
                            FMT == 0 ? (s1 >> by) & 0xFFu : s1 >> by};
        }
    }
};

// A lane's unit of the stretch from k on, for what K has past its last whole group:
// zeros past the row's end, which may be inside the lane's 32 values (NVFP4).
template <int FMT>
__device__ __forceinline__ W4Unit load_tail(const uint8_t *codes, const uint8_t *scales, int k,
                                            int K) {
    const int at = k + 32 * ((threadIdx.x & (WAVE - 1)) >> 4);
    W4Unit u = {{0, 0, 0, 0}, 0};
    if (at >= K) return u;
    const uint32_t *c = (const uint32_t *)(codes + at / 2);
    u.codes.x = c[0], u.codes.y = c[1];
    if constexpr (FMT == 0) {
        u.codes.z = c[2], u.codes.w = c[3];
        u.scale = scales[at / 32];
    } else {
        u.scale = scales[at / 16];
        if (at + 16 < K) {
            u.codes.z = c[2], u.codes.w = c[3];
            u.scale |= (uint32_t)scales[at / 16 + 1] << 8;
        }
    }
    return u;
}

// ---- products ----------------------------------------------------------------
// A stretch: its products with activations are added to acc; top takes part in
// w4_nan_rows.  x(t, i, n) is term n of values 8 i .. 8 i + 7 of the lane's 32 for
// its row of activation tile t.
template <int FMT, int TERMS, int PARTS, int TILES, typename X>
__device__ __forceinline__ void w4_multiply(const W4Unit (&w)[PARTS], const X &x,
                                            f32x4_t (&acc)[PARTS][TILES], uint32_t (&top)[PARTS]) {
#pragma unroll
    for (int p = 0; p < PARTS; ++p) top[p] = max(top[p], w[p].scale);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        bf16x8_t v[PARTS];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) v[p] = w4_decode<FMT>(w[p], i);
#pragma unroll
        for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int n = 0; n < TERMS; ++n) {
                const bf16x8_t b = x(t, i, n);
#pragma unroll
                for (int p = 0; p < PARTS; ++p) acc[p][t] = mfma_w4(v[p], b, acc[p][t]);
            }
    }
}

// A scale byte of 255 in any lane of a row makes the row's sums NaN (MXFP4).  No branch:
// behind one that joins again before a product's result is read, the compiler counts the
// waits that it needs along one way only, and on the shorter one the result may come too
// late.
template <int PARTS, int TILES>
__device__ __forceinline__ void w4_nan_rows(const uint32_t (&top)[PARTS],
                                            f32x4_t (&acc)[PARTS][TILES]) {
    const int g = (threadIdx.x & (WAVE - 1)) >> 4;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        const uint64_t lanes = __ballot(top[p] == 255u);
        uint32_t bad = (uint32_t)lanes | (uint32_t)(lanes >> 32);
        bad = (bad | bad >> 16) >> (4 * g);  // bit i: row 4 g + i
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int t = 0; t < TILES; ++t)
                acc[p][t][i] = (bad >> i & 1) != 0 ? __builtin_nanf("") : acc[p][t][i];
    }
}

// ---- activations of one stretch, up to 16 rows ---------------------------------
// A wave brings the activations of its stretch into LDS of its own, as 16-byte pieces
// of 8 values, and reads them as its products want them.  Lanes next to each other load
// what is next to each other in memory (of 64 lanes in as many lines, a load takes four
// times as long), every lane has a share of the rows there are (from a lane's row alone,
// 16 - ROWS of 16 lanes would load nothing), and fp32 is split into its terms once a
// value, not once for each row of a tile.  Rows that are not there are others' or
// whatever LDS held: they end in sums that nothing stores.  A wave's LDS operations keep
// their order, so there is no barrier but wave_order.
//
// Piece of values 8 v .. of row `row`, term n: at [v % 4][n][v / 4][row ^ v].  What lanes
// write at a time (a row's v) and what they read (all rows of v / 4 = 0 .. 3, the four
// lane groups) are both next to each other, so over all banks (with [v][n][row ^ v] the
// lane groups' reads shared banks: 16 tokens of 128 experts 180 us, not 170).
//
// COLUMNS: a product has 16 columns, of which ROWS tokens leave some without use; the
// terms are then columns of their own, token r's term n in column ROWS n + r, TILES
// products of 16 hold them all, and sum_columns adds them up.  (Three terms of four
// tokens are one product instead of three, with a third of the reads.)  Pieces are at
// [v % 4][v / 4][n][row ^ v].
template <bool F32, int ROWS, int PLANES = 1, bool COLUMNS = false>
struct XPart {
    static constexpr int SPLIT = F32 ? 3 : PLANES;                        // terms of a value
    static constexpr int TERMS = COLUMNS ? 1 : SPLIT;          // products of a tile
    static constexpr int TILES = COLUMNS ? (SPLIT * ROWS + 15) / 16 : 1;
    static constexpr int PIECES = ROWS * 16 * SPLIT;           // in LDS
    static constexpr int HALVES = F32 ? 2 : 1;                            // loads of a piece
    static constexpr int LOADS = ROWS * 16 * HALVES * PLANES / WAVE;      // of a lane
    static_assert(ROWS * 16 * HALVES * PLANES % WAVE == 0, "every lane loads");
    u32x4_t v[LOADS];

    // Load n of a lane: its row and plane, and the value of the stretch it starts at.
    struct Place {
        int row, k, plane;
    };
    static __device__ __forceinline__ Place place(int n) {
        const int p = n * WAVE + (threadIdx.x & (WAVE - 1));
        const int q = p / (16 * HALVES);
        return {q / PLANES, p % (16 * HALVES) * (8 / HALVES), q % PLANES};
    }

    // at[n]: the lane's byte offset of load n in the activations, of the stretch at 0
    // (NOWHERE: no such row); k: the stretch's offset in values, or NOWHERE.
    __device__ __forceinline__ void load(Rsrc x, const uint32_t (&at)[LOADS], uint32_t k) {
#pragma unroll
        for (int n = 0; n < LOADS; ++n)
            v[n] = load16(x, at[n] + (k == NOWHERE ? NOWHERE / 2 : k * (F32 ? 4 : 2)));
    }

    static __device__ __forceinline__ int at(int v, int n, int row) {
        const int place = row ^ (v & (ROWS - 1));
        if constexpr (COLUMNS) return (((v & 3) * 4 + (v >> 2)) * SPLIT + n) * ROWS + place;
        else return (((v & 3) * SPLIT + n) * 4 + (v >> 2)) * ROWS + place;
    }

    __device__ __forceinline__ void store(u32x4_t *lds) const {
#pragma unroll
        for (int n = 0; n < LOADS; ++n) {
            const auto from = place(n);
            const int piece = from.k / 8;
            if constexpr (F32) {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = u2f(v[n][j]);
                u32x2_t t[3];
                if constexpr (COLUMNS) split_finite_f32x4(x, t);
                else split_f32x4(x, t);
                u32x2_t *to = (u32x2_t *)(lds + at(piece, 0, from.row)) + (from.k / 4 & 1);
#pragma unroll
                for (int m = 0; m < 3; ++m) to[m * (COLUMNS ? 2 : 8) * ROWS] = t[m];
            } else {
                lds[at(piece, from.plane, from.row)] = v[n];
            }
        }
    }

    // The term and row of the lane's column of tile t (COLUMNS).  Columns past the last
    // term have the last one again: nothing reads their sums.
    static __device__ __forceinline__ int column_term(int t) {
        return min((16 * t + (int)(threadIdx.x & 15)) / ROWS, SPLIT - 1);
    }
    static __device__ __forceinline__ int column_row() { return threadIdx.x & (ROWS - 1); }

    // Values 8 i .. 8 i + 7 of the lane's 32 for its row, term n of them, or that of its
    // column of tile t; the 32 values of lane group g are the stretch's group_of(g)-th.
    static __device__ __forceinline__ bf16x8_t piece(const u32x4_t *lds, int group, int t, int i,
                                                     int n) {
        const int term = COLUMNS ? column_term(t) : n;
        return __builtin_bit_cast(bf16x8_t, lds[at(4 * group + i, term, column_row())]);
    }

    // The sums of the lane's token, in the columns of its first term (COLUMNS, three
    // terms of 4 or 8 tokens): the small terms' first.  A first term that is not finite
    // makes a sum that is not either, and then it is the sum: the other terms may be NaN.
    static __device__ __forceinline__ f32x4_t sum_columns(const f32x4_t (&acc)[TILES]) {
        static_assert(COLUMNS && SPLIT == 3 && (ROWS == 4 || ROWS == 8));
        f32x4_t s;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float second = dppf<DPP_ROW_SHL + ROWS>(acc[0][j]);
            const float third = ROWS == 4 ? dppf<DPP_ROW_SHL + 8>(acc[0][j]) : acc[TILES - 1][j];
            s[j] = __builtin_fabsf(acc[0][j]) < __builtin_inff() ? acc[0][j] + (second + third)
                                                                 : acc[0][j];
        }
        return s;
    }
};

// A barrier for what the workgroup has in LDS: loads from memory stay on their way.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A group of K that a wave multiplies: the weights that have it, its place k in them
// and in the activations (NOWHERE: none), and the lane's rows of the activations.
template <typename W, typename X>
struct Group {
    W w;
    uint32_t k;
    uint32_t x_at[X::LOADS];
};

// A wave's groups group(first), group(first + step), .. up to `groups`: their products
// are added to acc, and done(n) is called after each.  Weights are loaded two pairs
// ahead, activations two stretches.  The loop is short on purpose: instructions that run
// once have to come from memory first (four groups unrolled: 1 x 512 x 2048 9 us, not 4).
template <int FMT, bool PACKED, typename W, typename X, int PARTS, typename GroupAt, typename Done>
__device__ __forceinline__ void multiply_groups(const GroupAt &group, Rsrc x, u32x4_t *x_lds,
                                                int first, int step, int groups,
                                                f32x4_t (&acc)[PARTS][X::TILES],
                                                uint32_t (&top)[PARTS], const Done &done) {
    const int g = (threadIdx.x & (WAVE - 1)) >> 4, part = PACKED ? packed_group(g) : g;
    const auto from = [](uint32_t k, int more) { return k == NOWHERE ? k : k + more; };
    if (first >= groups) return;
    Group<W, X> here = group(first);
    typename W::Scales scales = here.w.load_scales(here.k);
    typename W::Pair pair[2];
    X xs[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        pair[j] = here.w.load_pair(here.k + 2 * W4_STRETCH * j);
        if (j == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i) xs[i].load(x, here.x_at, here.k + W4_STRETCH * i);
        __builtin_amdgcn_sched_barrier(0);  // in the order that they are waited for
    }
    for (int n = first; n < groups; n += step) {
        Group<W, X> next = group(n + step < groups ? n + step : n);
        if (n + step >= groups) next.k = NOWHERE;
        const typename W::Scales s = scales;
        here.w.put(s);
        scales = next.w.load_scales(next.k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j % 2 == 0) here.w.spread(pair[j / 2]);
            xs[j & 1].store(x_lds);
            wave_order();
            if (j < 2) xs[j].load(x, here.x_at, here.k + W4_STRETCH * (j + 2));
            else xs[j & 1].load(x, next.x_at, from(next.k, W4_STRETCH * (j - 2)));
            __builtin_amdgcn_sched_barrier(0);
            W4Unit u[PARTS];
            here.w.units(s, pair[j / 2], j, u);
            w4_multiply<FMT, X::TERMS>(
                u, [&](int t, int i, int m) { return X::piece(x_lds, part, t, i, m); }, acc, top);
            if (j % 2 == 1) pair[j / 2] = next.w.load_pair(from(next.k, W4_STRETCH * (j - 1)));
            wave_order();  // before the next stretch's stores
            __builtin_amdgcn_sched_barrier(0);
        }
        done(n);
        here = next;
    }
}

}  // namespace fp4dev

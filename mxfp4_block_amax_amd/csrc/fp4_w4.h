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
// bits each, all 24.  Sums are fp32.
#pragma once

#include "fp4_device.h"

namespace fp4dev {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
// vectors in memory that start where their first element may
typedef u32x4_t u32x4_at4_t __attribute__((aligned(4)));
typedef u32x4_t u32x4_at1_t __attribute__((aligned(1)));
typedef u32x2_t u32x2_at1_t __attribute__((aligned(1)));

constexpr int W4_UNIT = 256;  // values of K that a lane group's two loads of a row cover

// The scale bytes of a lane's two 32-value stretches of a unit: MXFP4 one byte
// each, NVFP4 two.
template <int FMT>
struct W4Unit {
    u32x4_t codes[2];
    uint32_t scale[2];
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

// Values 8 i .. 8 i + 7 of a lane's stretch h of a unit.
template <int FMT>
__device__ __forceinline__ bf16x8_t w4_decode(const W4Unit<FMT> &u, int h, int i) {
    if constexpr (FMT == 0) {
        return w4_values(u.codes[h][i], e8m0_operand(u.scale[h]));
    } else {
        return w4_values_e4m3(u.codes[h][i],
                              i < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)u.scale[h], 0)
                                    : __builtin_amdgcn_cvt_f32_fp8((int)u.scale[h], 1));
    }
}

template <int N>
struct Terms {
    bf16x8_t p[N];
};

// Eight fp32 values as three bf16 terms: a value's upper 16 bits, those of what
// they leave, and the rest (differences are exact, and nothing overflows).  A
// value that is not finite is its first term alone.
__device__ __forceinline__ Terms<3> split_f32x8(const float (&x)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, f2u(x[i]) & 0x7FFFFFFFu);
    float rest[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) rest[i] = x[i];
    Terms<3> t;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = __builtin_amdgcn_perm(f2u(rest[2 * i + 1]), f2u(rest[2 * i]), 0x07060302u);
        __builtin_memcpy(&t.p[k], w, sizeof(w));
#pragma unroll
        for (int i = 0; i < 8; ++i) rest[i] = rest[i] - u2f(f2u(rest[i]) & 0xFFFF0000u);
    }
    if (top >= 0x7F800000u) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = f2u(x[i]), a = b & 0x7FFFFFFFu;
            if (a >= 0x7F800000u) {
                t.p[0][i] = a > 0x7F800000u ? (__bf16)__builtin_nanf("") : (__bf16)x[i];
                t.p[1][i] = t.p[2][i] = (__bf16)0.0f;
            }
        }
    }
    return t;
}

// Eight activations from memory: bf16 as they are, fp32 in three terms.
__device__ __forceinline__ Terms<1> load_terms(const uint16_t *p) {
    return {__builtin_bit_cast(bf16x8_t, *(const uint4 *)p)};
}
__device__ __forceinline__ Terms<3> load_terms(const float *p) {
    float x[8];
    widen_f32x8(((const uint4 *)p)[0], ((const uint4 *)p)[1], x);
    return split_f32x8(x);
}

__device__ __forceinline__ f32x4_t mfma_w4(bf16x8_t w, bf16x8_t x, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x, c, 0, 0, 0);
}

// Where a lane's weight row lies: codes [rows, K/2] and scales [rows, K/block].
template <int FMT>
struct W4Row {
    const uint8_t *codes, *scales;
};

// Unit u of a row, all of it inside the row.
template <int FMT>
__device__ __forceinline__ W4Unit<FMT> w4_load(const W4Row<FMT> &row, int64_t u, int g) {
    W4Unit<FMT> r;
    const uint8_t *c = row.codes + u * (W4_UNIT / 2) + 16 * g;
    r.codes[0] = *(const u32x4_at4_t *)c;
    r.codes[1] = *(const u32x4_at4_t *)(c + 64);
    if constexpr (FMT == 0) {
        const u32x2_t s = *(const u32x2_at1_t *)(row.scales + u * (W4_UNIT / 32));
        r.scale[0] = (s.x >> (8 * g)) & 0xFFu;
        r.scale[1] = (s.y >> (8 * g)) & 0xFFu;
    } else {
        const u32x4_t s = *(const u32x4_at1_t *)(row.scales + u * (W4_UNIT / 16));
        r.scale[0] = (g & 2 ? s.y : s.x) >> (16 * (g & 1));
        r.scale[1] = (g & 2 ? s.w : s.z) >> (16 * (g & 1));
    }
    return r;
}

// The last unit of a row whose K is no multiple of a unit: stretches past the
// row's end are zero, and so is the half past it of one that NVFP4's K ends in.
template <int FMT>
__device__ __forceinline__ W4Unit<FMT> w4_load_tail(const W4Row<FMT> &row, int64_t u, int g,
                                                    int64_t K) {
    W4Unit<FMT> r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t k = u * W4_UNIT + 128 * h + 32 * g;
        r.codes[h] = {0, 0, 0, 0};
        r.scale[h] = 0;
        if (k >= K) continue;
        if constexpr (FMT == 0) {
            r.codes[h] = *(const u32x4_at4_t *)(row.codes + k / 2);
            r.scale[h] = row.scales[k / 32];
        } else {
            const uint32_t *c = (const uint32_t *)(row.codes + k / 2);
            r.codes[h].x = c[0], r.codes[h].y = c[1];
            r.scale[h] = row.scales[k / 16];
            if (k + 16 < K) {
                r.codes[h].z = c[2], r.codes[h].w = c[3];
                r.scale[h] |= (uint32_t)row.scales[k / 16 + 1] << 8;
            }
        }
    }
    return r;
}

// The same unit of a packed operand's row tile of 32 rows: a lane's loads are of
// rows l % 32 and 32-value stretches 2 ks + l / 32 of four K steps ks.  Exchanging
// odd groups of 16 lanes of one step with even ones of the next gives a register
// rows 0 .. 15 and another rows 16 .. 31, with the stretches 0, 2, 1, 3 in lane
// groups 0 .. 3.
__device__ __forceinline__ int packed_stretch(int g) { return (g & 1) * 2 + (g >> 1); }

__device__ __forceinline__ void swap16(uint32_t &a, uint32_t &b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

template <int FMT>
__device__ __forceinline__ void w4_load_packed(const uint8_t *codes, const uint8_t *scales,
                                               int64_t u, int lane, W4Unit<FMT> (&r)[2]) {
    const u32x4_t *c = (const u32x4_t *)(codes + u * 4096) + lane;
    const int odd = (lane >> 4) & 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        u32x4_t a = c[128 * h], b = c[128 * h + 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t x = a[i], y = b[i];
            swap16(x, y);
            r[0].codes[h][i] = x;
            r[1].codes[h][i] = y;
        }
    }
    if constexpr (FMT == 0) {
        uint32_t s0 = *(const uint32_t *)(scales + (u >> 1) * 512 + 8 * lane + 4 * (u & 1)), s1 = s0;
        swap16(s0, s1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            r[0].scale[h] = (s0 >> (16 * h + 8 * odd)) & 0xFFu;
            r[1].scale[h] = (s1 >> (16 * h + 8 * odd)) & 0xFFu;
        }
    } else {
        const u32x2_t s = *(const u32x2_t *)(scales + (u >> 1) * 1024 + 16 * lane + 8 * (u & 1));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t s0 = h ? s.y : s.x, s1 = s0;
            swap16(s0, s1);
            r[0].scale[h] = s0 >> (16 * odd);
            r[1].scale[h] = s1 >> (16 * odd);
        }
    }
}

// One unit: its products with X's activations are added to acc; top takes part in
// w4_nan_rows.  x(t, k) gives the terms of values k .. k + 7 of the unit for the
// lane's row of activation tile t.
template <int FMT, int ROWS, int TILES, typename X>
__device__ __forceinline__ void w4_multiply(const W4Unit<FMT> (&w)[ROWS], const X &x,
                                            f32x4_t (&acc)[ROWS][TILES], uint32_t (&top)[ROWS]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int p = 0; p < ROWS; ++p) top[p] = max(top[p], w[p].scale[h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            bf16x8_t v[ROWS];
#pragma unroll
            for (int p = 0; p < ROWS; ++p) v[p] = w4_decode<FMT>(w[p], h, i);
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                const auto b = x(t, 128 * h + 8 * i);
#pragma unroll
                for (auto &term : b.p)
#pragma unroll
                    for (int p = 0; p < ROWS; ++p) acc[p][t] = mfma_w4(v[p], term, acc[p][t]);
            }
        }
    }
}

// A scale byte of 255 in any lane of a row makes the row's sums NaN (MXFP4).
template <int ROWS, int TILES>
__device__ __forceinline__ void w4_nan_rows(const uint32_t (&top)[ROWS],
                                            f32x4_t (&acc)[ROWS][TILES]) {
    const int g = (threadIdx.x & (WAVE - 1)) >> 4;
#pragma unroll
    for (int p = 0; p < ROWS; ++p) {
        uint64_t bad = __ballot(top[p] == 255u);
        if (bad == 0) continue;
        bad |= bad >> 32;
        bad |= bad >> 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (bad >> (4 * g + i) & 1)
#pragma unroll
                for (int t = 0; t < TILES; ++t) acc[p][t][i] = __builtin_nanf("");
    }
}

}  // namespace fp4dev

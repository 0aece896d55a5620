// fp4_linear.hip - linear layers of few tokens with an FP4 weight and
// activations that keep their precision:
//
//   c_mn = s_g sum_b s_nb sum_{k in b} E2M1(code_nk) x_mk,
//
// s_g = 1 for MXFP4.  What it cannot do without is reading the weight once: a
// token's 2 N K operations are far below the MFMA's rate up to some 64 tokens.
#include "fp4_kernels.h"
#include "fp4_linear.h"
#include "fp4_w4.h"

namespace fp4dev {
namespace {

struct LinearArgs {
    const void *x;
    const uint8_t *codes, *scales;  // packed: of the row tiles
    const float *s_g;
    void *c;
    int32_t M, N, K;
    bool out_bf16;
};

constexpr int LINEAR_WAVES = 16;

// Waves of a workgroup: 16, or 8 where more tokens leave registers or LDS for no more.
template <bool X_F32, int TOKENS>
constexpr int tile_waves() {
    return TOKENS > 8 || (X_F32 && TOKENS > 4) ? 8 : LINEAR_WAVES;
}

// Up to TOKENS (16 at most) tokens and 32 weight rows a workgroup: its waves take
// groups of K in turn, and add their sums in LDS in the order of the waves.  Two parts of
// 16 rows a wave, so that a fragment of the activations serves two products; and with 32
// rows 8192 of them fill the CUs.  The weight's bytes bound it: captured, with inputs from
// memory, 1 x 8192 x 8192 packed takes 9.8 us (3.6 TB/s; 2 us are a node's start), 1 x 8192
// x 28672 23.8 (5.3 TB/s), 16 x 8192 x 28672 in NVFP4 38.5 (3.4 TB/s, vector instructions
// 35 % of the cycles), and 1 x 512 x 2048 3.9, a chain of load, decode and join.
template <int FMT, bool X_F32, bool PACKED, int TOKENS, int WAVES>
__global__ __launch_bounds__(WAVES *WAVE) void linear_w4_kernel(LinearArgs A) {
    using XT = std::conditional_t<X_F32, float, uint16_t>;
    using X = XPart<X_F32, TOKENS>;
    extern __shared__ u32x4_t lds[];
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    constexpr int waves = WAVES;
    const int m0 = blockIdx.y * TOKENS, row0 = blockIdx.x * LINEAR_ROWS, K = A.K;
    const int tokens = min(TOKENS, A.M - m0);

    const Rsrc x = span((const XT *)A.x + (int64_t)m0 * K, tokens * K * (int)sizeof(XT));
    uint32_t x_at[X::LOADS];
#pragma unroll
    for (int n = 0; n < X::LOADS; ++n) {
        const auto p = X::place(n);
        x_at[n] = (uint32_t)(p.row * K + p.k) * (uint32_t)sizeof(XT);
    }
    constexpr int BLK = FMT == 0 ? 32 : 16;
    using W = std::conditional_t<PACKED, PackedAt<FMT, 2>, RowsAt<FMT, 2>>;
    u32x4_t *mine = lds + wave * (X::PIECES + W::LDS);
    const uint8_t *codes = A.codes + (int64_t)row0 * (K / 2);
    const uint8_t *scales = A.scales + (int64_t)row0 * (K / BLK);

    f32x4_t acc[2][1] = {};
    uint32_t top[2] = {0, 0};
    const int groups = (uint32_t)K / W4_GROUP;
    const W weights = [&] {
        if constexpr (PACKED) return W(codes, scales, A.N - row0, K);
        else return W(codes, scales, A.N - row0, 16, K, mine + X::PIECES);
    }();
    multiply_groups<FMT, PACKED, W, X>(
        [&](int n) {
            Group<W, X> a = {weights, (uint32_t)(n * W4_GROUP), {}};
#pragma unroll
            for (int i = 0; i < X::LOADS; ++i) a.x_at[i] = x_at[i];
            return a;
        },
        x, mine, wave, waves, groups, acc, top, [](int) {});
    if constexpr (!PACKED) {
        // the stretches past the last whole group, by the waves that have fewer groups
        const int r = lane & 15, g = lane >> 4;
        int t = (wave - groups % waves + waves) % waves;
        for (int k = groups * W4_GROUP + W4_STRETCH * t; k < K; k += W4_STRETCH * waves) {
            W4Unit w[2];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const int n = min(16 * p + r, A.N - 1 - row0);
                w[p] = load_tail<FMT>(codes + (int64_t)n * (K / 2), scales + (int64_t)n * (K / BLK), k, K);
            }
            Terms<X::TERMS> b[4] = {};
            const int at = k + 32 * g;
            if (r < tokens)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (at + 8 * i < K)
                        b[i] = load_terms((const XT *)A.x + (int64_t)(m0 + r) * K + at + 8 * i);
            w4_multiply<FMT, X::TERMS>(w, [&](int, int i, int n) { return b[i].p[n]; }, acc, top);
        }
    }
    if constexpr (FMT == 0) w4_nan_rows(top, acc);
    __syncthreads();
    f32x4_t *sums = (f32x4_t *)lds;  // [waves][2][64]
#pragma unroll
    for (int p = 0; p < 2; ++p) sums[(wave * 2 + p) * WAVE + lane] = acc[p][0];
    __syncthreads();
    // four sums at a time: a wave has 64 / 4 outputs' quarters
    if (wave >= 2) return;
    f32x4_t s = sums[wave * WAVE + lane];
    for (int v = 1; v < waves; ++v) s += sums[(v * 2 + wave) * WAVE + lane];
    const int m = m0 + (lane & 15), n = row0 + 16 * wave + 4 * (lane >> 4);
    if ((lane & 15) >= tokens) return;
    if constexpr (FMT == 1) s = s * *A.s_g;
    const int64_t to = (int64_t)m * A.N + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= A.N) break;
        if (A.out_bf16) ((__bf16 *)A.c)[to + j] = (__bf16)s[j];
        else ((float *)A.c)[to + j] = s[j];
    }
}

template <int FMT, bool X_F32, bool PACKED, int TOKENS>
hipError_t launch_tile(const LinearArgs &A, hipStream_t s) {
    constexpr int waves = tile_waves<X_F32, TOKENS>();
    const size_t pieces =
        (size_t)waves * (XPart<X_F32, TOKENS>::PIECES + (PACKED ? 0 : RowsAt<FMT, 2>::LDS)) * 16;
    const size_t sums = (size_t)waves * 2 * WAVE * sizeof(f32x4_t);
    const dim3 grid((uint32_t)((A.N + LINEAR_ROWS - 1) / LINEAR_ROWS),
                    (uint32_t)((A.M + TOKENS - 1) / TOKENS));
    linear_w4_kernel<FMT, X_F32, PACKED, TOKENS, waves>
        <<<grid, waves * WAVE, pieces > sums ? pieces : sums, s>>>(A);
    return hipGetLastError();
}

// More tokens, bf16: 16 TILES of them and 64 ROW_WAVES weight rows a workgroup.  A wave
// has 64 rows (what it reads of the activations then serves as many products as the matrix
// units do while LDS gives them); ROW_WAVES waves side by side take a group of K, the
// others of the eight the next ones.  A slab, a stretch of each of these groups, of the
// activations is in LDS for all; the next one is on its way in registers.  With tiles of 4
// the matrix, vector and LDS instructions of a stretch take some 2000 cycles each, one
// after the other, 5900 in all: barriers keep the waves in step, so that little overlaps.
// 64 x 28672 x 8192 packed 47 us, of which the weight's bytes are 26.
constexpr int WIDE_WAVES = 8;
constexpr int WIDE_THREADS = WIDE_WAVES * WAVE;

template <int FMT, bool PACKED, int TILES, int ROW_WAVES>
__global__ __launch_bounds__(WIDE_THREADS, 2) void linear_w4_wide_kernel(LinearArgs A) {
    constexpr int BLK = FMT == 0 ? 32 : 16, PARTS = WIDE_PARTS;
    constexpr int K_WAVES = WIDE_WAVES / ROW_WAVES, ROWS = 16 * PARTS * ROW_WAVES;
    constexpr int SLAB = K_WAVES * TILES * 256;  // pieces: [K wave][tile][v][row ^ v]
    constexpr int LOADS = SLAB / WIDE_THREADS;
    using W = std::conditional_t<PACKED, PackedAt<FMT, PARTS>, RowsAt<FMT, PARTS>>;
    extern __shared__ u32x4_t lds[];  // [2][SLAB], then the waves' own
    const int lane = threadIdx.x & (WAVE - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int k_wave = wave % K_WAVES, row_wave = wave / K_WAVES;
    const int r = lane & 15, g = lane >> 4, part = PACKED ? packed_group(g) : g;
    const int m0 = blockIdx.y * (16 * TILES), K = A.K;
    const int row0 = blockIdx.x * ROWS + 16 * PARTS * row_wave;
    const int tokens = min(16 * TILES, A.M - m0);
    const int groups = (uint32_t)K / W4_GROUP;
    const int slabs = (groups + K_WAVES - 1) / K_WAVES * 4;  // four stretches a group

    // a wave past the last row has the last ones' weights, for sums that are not stored
    const int first = min(row0, (A.N - 1) / 32 * 32);
    const uint8_t *codes = A.codes + (int64_t)first * (K / 2);
    const uint8_t *scales = A.scales + (int64_t)first * (K / BLK);
    const W w = [&] {
        if constexpr (PACKED) return W(codes, scales, A.N - first, K);
        else return W(codes, scales, A.N - first, 16, K, lds + 2 * SLAB + wave * W::LDS);
    }();
    const Rsrc x = span((const uint16_t *)A.x + (int64_t)m0 * K, tokens * K * 2);
    const auto group_k = [&](int n) { return n < groups ? (uint32_t)(n * W4_GROUP) : NOWHERE; };
    const auto from = [](uint32_t k, int more) { return k == NOWHERE ? k : k + more; };

    // a thread's load n of a slab: 16 lanes have a row's stretch
    u32x4_t xs[LOADS];
    const auto load_slab = [&](int s) {
#pragma unroll
        for (int n = 0; n < LOADS; ++n) {
            const int e = n * WIDE_THREADS + threadIdx.x, v = e / 16 % K_WAVES;
            const uint32_t k = group_k(s / 4 * K_WAVES + v);
            xs[n] = load16(x, (uint32_t)(e / (16 * K_WAVES) * K + 8 * (e & 15)) * 2 +
                                  (k == NOWHERE ? NOWHERE / 2 : (k + (s & 3) * W4_STRETCH) * 2));
        }
    };
    const auto store_slab = [&](u32x4_t *to) {
#pragma unroll
        for (int n = 0; n < LOADS; ++n) {
            const int e = n * WIDE_THREADS + threadIdx.x, piece = e & 15, v = e / 16 % K_WAVES;
            const int row = e / (16 * K_WAVES);
            to[((v * TILES + row / 16) * 16 + piece) * 16 + ((row & 15) ^ piece)] = xs[n];
        }
    };
    load_slab(0);
    uint32_t k = group_k(k_wave);
    typename W::Scales scale = w.load_scales(k);
    typename W::Pair pair[2] = {w.load_pair(k), w.load_pair(from(k, 2 * W4_STRETCH))};
    __builtin_amdgcn_sched_barrier(0);
    store_slab(lds);
    lds_barrier();

    f32x4_t acc[PARTS][TILES] = {};
    uint32_t top[PARTS] = {};
    for (int s = 0; s < slabs; s += 4) {
        const uint32_t next = group_k(s / 4 * K_WAVES + K_WAVES + k_wave);
        const typename W::Scales here = scale;
        w.put(here);
        scale = w.load_scales(next);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            load_slab(s + j + 1);
            __builtin_amdgcn_sched_barrier(0);
            if (j % 2 == 0) w.spread(pair[j / 2]);
            W4Unit u[PARTS];
            w.units(here, pair[j / 2], j, u);
            const u32x4_t *mine = lds + (j & 1) * SLAB + k_wave * TILES * 256;
            w4_multiply<FMT, 1>(
                u,
                [&](int t, int i, int) {
                    const int v = 4 * part + i;
                    return __builtin_bit_cast(bf16x8_t, mine[(t * 16 + v) * 16 + (r ^ v)]);
                },
                acc, top);
            if (j % 2 == 1) pair[j / 2] = w.load_pair(from(next, W4_STRETCH * (j - 1)));
            __builtin_amdgcn_sched_barrier(0);
            store_slab(lds + ((j + 1) & 1) * SLAB);
            lds_barrier();
        }
    }
    if constexpr (!PACKED) {
        // the stretches past the last whole group, in turn
        for (int q = groups * W4_GROUP + W4_STRETCH * k_wave; q < K; q += W4_STRETCH * K_WAVES) {
            W4Unit u[PARTS];
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                const int64_t n = min(16 * p + r, A.N - 1 - first);
                u[p] = load_tail<FMT>(codes + n * (K / 2), scales + n * (K / BLK), q, K);
            }
            const int at = q + 32 * g;
            w4_multiply<FMT, 1>(
                u,
                [&](int t, int i, int) {
                    Terms<1> b = {};
                    if (16 * t + r < tokens && at + 8 * i < K)
                        b = load_terms((const uint16_t *)A.x + (int64_t)(m0 + 16 * t + r) * K + at + 8 * i);
                    return b.p[0];
                },
                acc, top);
        }
    }
    if constexpr (FMT == 0) w4_nan_rows(top, acc);
    // the K waves' sums, one part after the other, added in their order
    f32x4_t *sums = (f32x4_t *)lds;  // [K wave][row wave][TILES][64]
    constexpr int EACH = ROW_WAVES * TILES * WAVE;
    static_assert(K_WAVES * EACH <= 2 * SLAB);
    const float s_g = FMT == 0 ? 1.0f : *A.s_g;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        __syncthreads();
#pragma unroll
        for (int t = 0; t < TILES; ++t)
            sums[k_wave * EACH + (row_wave * TILES + t) * WAVE + lane] = acc[p][t];
        __syncthreads();
        for (int i = threadIdx.x; i < EACH; i += WIDE_THREADS) {
            f32x4_t y = sums[i];
#pragma unroll
            for (int v = 1; v < K_WAVES; ++v) y += sums[v * EACH + i];
            if constexpr (FMT == 1) y = y * s_g;
            const int l = i % WAVE, m = m0 + 16 * (i / WAVE % TILES) + (l & 15);
            const int n = blockIdx.x * ROWS + i / (TILES * WAVE) * 16 * PARTS + 16 * p + 4 * (l >> 4);
            if (m >= A.M) continue;
            const int64_t to = (int64_t)m * A.N + n;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (n + j >= A.N) break;
                if (A.out_bf16) ((__bf16 *)A.c)[to + j] = (__bf16)y[j];
                else ((float *)A.c)[to + j] = y[j];
            }
        }
    }
}

template <int FMT, bool PACKED, int TILES, int ROW_WAVES>
hipError_t launch_wide(const LinearArgs &A, hipStream_t s) {
    constexpr int ROWS = 16 * WIDE_PARTS * ROW_WAVES;
    const size_t lds = 2 * (WIDE_WAVES / ROW_WAVES) * TILES * 256 * 16 +
                       (PACKED ? 0 : WIDE_WAVES * RowsAt<FMT, WIDE_PARTS>::LDS * 16);
    const dim3 grid((uint32_t)((A.N + ROWS - 1) / ROWS),
                    (uint32_t)((A.M + 16 * TILES - 1) / (16 * TILES)));
    linear_w4_wide_kernel<FMT, PACKED, TILES, ROW_WAVES><<<grid, WIDE_THREADS, lds, s>>>(A);
    return hipGetLastError();
}

// Tokens of a tile: the smallest that holds them (packed MXFP4, 8192 x 8192, tiles of 4, 8
// and 16: 4 tokens 9.8, 10.5, 10.8 us; 8 tokens 16.5, 10.9, 10.9, in fp32 23, 15, 19).
template <int FMT, bool X_F32, bool PACKED>
hipError_t launch_tokens(const LinearArgs &A, hipStream_t s) {
    if (A.M <= 4) return launch_tile<FMT, X_F32, PACKED, 4>(A, s);
    if (A.M <= 8) return launch_tile<FMT, X_F32, PACKED, 8>(A, s);
    if constexpr (!X_F32) {
        if (A.M > 16) {
            const Wide w = wide_tile(A.M, A.N);
            if (w.row_waves == 1)
                return w.tiles == 1 ? launch_wide<FMT, PACKED, 1, 1>(A, s) : launch_wide<FMT, PACKED, 2, 1>(A, s);
            if (w.tiles == 1) return launch_wide<FMT, PACKED, 1, 2>(A, s);
            if (w.tiles == 2) return launch_wide<FMT, PACKED, 2, 2>(A, s);
            if (w.tiles == 4) return launch_wide<FMT, PACKED, 4, 2>(A, s);
        }
    }
    return launch_tile<FMT, X_F32, PACKED, 16>(A, s);
}

template <int FMT, bool PACKED>
hipError_t launch_types(const LinearArgs &A, bool x_bf16, hipStream_t s) {
    return x_bf16 ? launch_tokens<FMT, false, PACKED>(A, s) : launch_tokens<FMT, true, PACKED>(A, s);
}

}  // namespace

hipError_t launch_linear_w4(int fmt, const void *x, bool x_bf16, int64_t M, int64_t K,
                            const uint8_t *codes, const uint8_t *scales, const float *s_g,
                            bool packed, int64_t N, void *c, bool out_bf16, hipStream_t s) {
    const LinearArgs A = {x, codes, scales, s_g, c, (int32_t)M, (int32_t)N, (int32_t)K, out_bf16};
    if (fmt == 0)
        return packed ? launch_types<0, true>(A, x_bf16, s) : launch_types<0, false>(A, x_bf16, s);
    return packed ? launch_types<1, true>(A, x_bf16, s) : launch_types<1, false>(A, x_bf16, s);
}

}  // namespace fp4dev

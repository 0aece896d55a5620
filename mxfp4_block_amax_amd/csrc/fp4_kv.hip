// fp4_kv.hip - writing and reading the 8-bit key/value cache.
//
// Write.  Per page and head with new values x (and live old codes c where the
// first new slot is not the page's first):
//   A = max |x|,  e = the smallest integer >= -127 with 448 2^e >= A,
//   live codes: e = max(e, e_old), c <- E4M3(c 2^(e_old - e)),
//   new codes:  E4M3(x 2^-e), nearest, ties to the even code.
// The scale is a power of two, so a page that grows moves its old codes
// without a second rounding, but for values that become E4M3 subnormals.
// Read: y = E4M3(c) 2^e.
//
// Both are bound by memory on prompts and by a launch on single tokens.  A
// workgroup has the keys and the values of one page and head: neither needs
// another's amax, a page's codes are contiguous, and the way to the page (the
// batch's prefix sums, then the table, then the page: three loads that wait for
// each other) is gone once for both.
#include <algorithm>
#include <type_traits>

#include "fp4_kernels.h"
#include "fp4_kv.h"

namespace fp4dev {
namespace {

constexpr int KV_HELD = 4;  // 8-value chunks of keys, and of values, a lane holds at once

// Eight values as loaded: 16 bytes of bf16, 32 of fp32.
template <bool BF16>
struct Chunk {
    u32x4_t w[BF16 ? 1 : 2];
};

// ONCE: streamed, nothing reads it again.
template <bool BF16, bool ONCE>
__device__ __forceinline__ Chunk<BF16> load_chunk(const void *x, int64_t at) {
    Chunk<BF16> c;
    const u32x4_t *p = BF16 ? (const u32x4_t *)((const uint16_t *)x + at)
                            : (const u32x4_t *)((const float *)x + at);
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i) c.w[i] = ONCE ? __builtin_nontemporal_load(p + i) : p[i];
    return c;
}

template <bool BF16>
__device__ __forceinline__ void widen(const Chunk<BF16> &c, float (&v)[8]) {
    if constexpr (BF16) {
        widen_bf16x8(make_uint4(c.w[0].x, c.w[0].y, c.w[0].z, c.w[0].w), v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = u2f(c.w[i / 4][i & 3]);
    }
}

// The largest finite magnitude; whether any value was not finite.
template <bool BF16>
__device__ __forceinline__ bool chunk_amax(const Chunk<BF16> &c, float &amax) {
    float v[8];
    widen<BF16>(c, v);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float a = __builtin_fabsf(v[i]);
        const bool fin = a < __builtin_inff();
        amax = fin ? __builtin_fmaxf(amax, a) : amax;
        bad = bad || !fin;
    }
    return bad;
}

// A chunk's codes under 2^-e; values that are not finite become NaN codes.
template <bool BF16>
__device__ __forceinline__ uint2 chunk_codes(const Chunk<BF16> &c, float inv) {
    float v[8], q[8];
    widen<BF16>(c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = __builtin_fabsf(v[i]) < __builtin_inff() ? v[i] * inv : __builtin_nanf("");
    return make_uint2(cvt_e4m3x4(q[0], q[1], q[2], q[3]), cvt_e4m3x4(q[4], q[5], q[6], q[7]));
}

// A launch's workgroups: x heads, then the batch's items of one page over y and
// z.  The heads of a page run side by side: their rows are pieces of the same
// rows of a projection, and of the same DRAM pages (8 x 4096 tokens of 8 heads of
// 128 written: 40.3 us, with the pages of a head side by side 40.9; 16 x 4096 read:
// 79.4 and 80.9).
constexpr int KV_GRID_Y = 32768;

__device__ __forceinline__ Item grid_item(const KvCache &C, const KvBatch &B, int32_t *status) {
    return find_item(B, (int)(blockIdx.z * KV_GRID_Y + blockIdx.y),
                     (int64_t)gridDim.y * gridDim.z, C.block, 2, blockIdx.x == 0, status);
}

dim3 kv_grid(const KvCache &C, const KvBatch &B) {
    const int64_t items = item_count(B.tokens, B.seqs, C.block, 2);
    return dim3((uint32_t)C.heads, (uint32_t)std::min<int64_t>(items, KV_GRID_Y),
                (uint32_t)((items + KV_GRID_Y - 1) / KV_GRID_Y));
}

// One half (keys or values) of the write's source and destination.
struct Half {
    const void *x;
    int64_t token, x0;  // stride of a token; the first new value
    uint8_t *codes, *scale;
};

template <bool BF16>
__global__ __launch_bounds__(256) void kv_write_kernel(KvCache C, KvBatch B, const void *k,
                                                       int64_t k_token, int64_t k_head,
                                                       const void *v, int64_t v_token,
                                                       int64_t v_head, int32_t *status) {
    __shared__ uint32_t part[2][256 / WAVE];
    const Item it = grid_item(C, B, status);
    if (it.seq >= B.seqs || it.count <= 0) {
        if (it.count < 0 && threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
        return;
    }
    const int64_t len = it.length, start = len - it.count;
    const int64_t b = (start < 0 ? 0 : start >> C.block_shift) + it.piece;
    const int64_t p0 = max(max(b << C.block_shift, start), (int64_t)0);
    const int64_t p1 = min((b + 1) << C.block_shift, len);
    if (start < 0 && it.piece == 0 && threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
    if (p0 >= p1) return;
    const int page = find_page(B, C, it.seq, b);
    if (page < 0) {
        if (threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
        return;
    }
    const int head = blockIdx.x;
    const int slot0 = (int)(p0 - (b << C.block_shift)), n = (int)(p1 - p0);
    const int64_t t0 = it.base + (p0 - start);
    const int64_t to = page_offset(C, page, head), at = (int64_t)page * C.heads + head;
    const Half half[2] = {
        {k, k_token, t0 * k_token + head * k_head, C.k_codes + to, C.k_scales + at},
        {v, v_token, t0 * v_token + head * v_head, C.v_codes + to, C.v_scales + at}};
    uint32_t before[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) before[s] = slot0 > 0 ? *half[s].scale : 0u;

    const int per = C.dim >> 3;  // chunks of a token: 8, 16, 24 or 32
    const int chunks = n * per;
    const bool held = chunks <= KV_HELD * (int)blockDim.x;
    auto fetch = [&](auto stream, const Half &f, int c) {
        const int t = c / per;
        return load_chunk<BF16, stream>(f.x, f.x0 + t * f.token + 8 * (c - t * per));
    };
    constexpr std::true_type once{};
    constexpr std::false_type again{};
    Chunk<BF16> x[2][KV_HELD];
    float amax[2] = {0.0f, 0.0f};
    bool bad = false;
    if (held) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < KV_HELD; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c < chunks) x[s][i] = fetch(once, half[s], c);
            }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < KV_HELD; ++i)
                if (threadIdx.x + i * blockDim.x < (uint32_t)chunks)
                    bad |= chunk_amax<BF16>(x[s][i], amax[s]);
    } else {
        // Too many to hold: read again below, for which these loads are ordinary
        // ones (8 x 4096 tokens of 8 heads of 128 in pages of 128, fp32: 109 us,
        // streamed 138; bf16 73 and 74; in pages of 256, bf16: 70 and 68).
        for (int c = threadIdx.x; c < chunks; c += blockDim.x)
#pragma unroll
            for (int s = 0; s < 2; ++s) bad |= chunk_amax<BF16>(fetch(again, half[s], c), amax[s]);
    }
    // non-negative floats order as their bits
    uint32_t top[2] = {wave_max_u32(f2u(amax[0])), wave_max_u32(f2u(amax[1]))};
    if (blockDim.x > WAVE) {
        if ((threadIdx.x & (WAVE - 1)) == 0)
#pragma unroll
            for (int s = 0; s < 2; ++s) part[s][threadIdx.x / WAVE] = top[s];
        __syncthreads();
#pragma unroll
        for (int s = 0; s < 2; ++s)
            top[s] = max(max(part[s][0], part[s][1]), max(part[s][2], part[s][3]));
    }
    if (__ballot(bad) != 0 && (threadIdx.x & (WAVE - 1)) == 0) flag(status, FLAG_NONFINITE);

#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const Half &f = half[s];
        const uint32_t byte = max(kv_scale_byte(u2f(top[s])), before[s]);
        const float inv = byte == 255u ? __builtin_nanf("") : e8m0_value(254u - byte);
        uint8_t *codes = f.codes + slot0 * C.dim;
        if (held) {
#pragma unroll
            for (int i = 0; i < KV_HELD; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c < chunks) *(uint2 *)(codes + 8 * c) = chunk_codes<BF16>(x[s][i], inv);
            }
        } else {
            for (int c = threadIdx.x; c < chunks; c += blockDim.x)
                *(uint2 *)(codes + 8 * c) = chunk_codes<BF16>(fetch(once, f, c), inv);
        }
        if (byte > before[s] && slot0 > 0) {
            // 448 2^-20 rounds to zero, and so does all below
            const float down = u2f((127u - min(byte - before[s], 40u)) << 23);
            for (int c = threadIdx.x; c < slot0 * per; c += blockDim.x) {
                uint2 w = *(const uint2 *)(f.codes + 8 * c);
                const f32x2_t a = e4m3_pair<false>(w.x), d = e4m3_pair<true>(w.x);
                const f32x2_t e = e4m3_pair<false>(w.y), g = e4m3_pair<true>(w.y);
                w.x = cvt_e4m3x4(a.x * down, a.y * down, d.x * down, d.y * down);
                w.y = cvt_e4m3x4(e.x * down, e.y * down, g.x * down, g.y * down);
                *(uint2 *)(f.codes + 8 * c) = w;
            }
        }
        if (threadIdx.x == 0) *f.scale = (uint8_t)byte;
    }
}

// A lane reads the codes of 16 bytes of output at a time, so that a wave's stores
// are whole lines, and streams them out: 16 x 4096 tokens of 8 heads of 128 as
// bf16, 404 MB moved, take 79 us (5.1 TB/s, what a large copy reaches here), 84
// with ordinary stores, 93 with two 16-byte stores side by side a lane.
constexpr int KV_READ = 2;  // such pieces of keys, and of values, a lane has in flight

// y rows are [tokens, heads, dim].
template <bool BF16>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache C, KvBatch B, void *k, void *v,
                                                      int32_t *status) {
    const Item it = grid_item(C, B, status);
    if (it.count <= 0) {
        if (it.count < 0 && threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
        return;
    }
    // rows past the last sequence, positions before 0 and pages that do not
    // exist read as zero
    const bool none = it.seq >= B.seqs;
    const int64_t len = none ? it.count : it.length, start = len - it.count;
    const int64_t b = (start >> C.block_shift) + it.piece;
    const int64_t p0 = max(b << C.block_shift, start);
    const int64_t p1 = min((b + 1) << C.block_shift, len);
    if (p0 >= p1) return;
    const int page = none ? -1 : find_page(B, C, it.seq, b);
    if (page < 0 && !none && threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
    const int head = blockIdx.x;
    const int64_t at = (int64_t)max(page, 0) * C.heads + head;
    const int64_t from = page_offset(C, max(page, 0), head) + (int)(p0 - (b << C.block_shift)) * C.dim;
    const uint8_t *codes[2] = {C.k_codes + from, C.v_codes + from};
    const uint8_t *bytes[2] = {C.k_scales + at, C.v_scales + at};
    void *y[2] = {k, v};
    constexpr int N = BF16 ? 8 : 4;  // codes of 16 bytes of output
    const int per = C.dim / N;
    const int chunks = (int)(p1 - p0) * per;
    const int64_t row = (int64_t)C.heads * C.dim;
    const int64_t y0 = (it.base + (p0 - start)) * row + (int64_t)head * C.dim;
    for (int c0 = threadIdx.x; c0 < chunks; c0 += KV_READ * blockDim.x) {
        uint32_t w[2][KV_READ][N / 4];
        float scale[2];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < KV_READ; ++i) {
                const int c = c0 + i * blockDim.x;
                const bool some = c < chunks && page >= 0;
                if constexpr (BF16) {
                    const uint2 x = some ? *(const uint2 *)(codes[s] + N * c) : make_uint2(0, 0);
                    w[s][i][0] = x.x, w[s][i][N / 4 - 1] = x.y;
                } else {
                    w[s][i][0] = some ? *(const uint32_t *)(codes[s] + N * c) : 0u;
                }
            }
            scale[s] = page < 0 ? 1.0f : e8m0_value(*bytes[s]);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < KV_READ; ++i) {
                const int c = c0 + i * blockDim.x;
                if (c >= chunks) continue;
                const int t = c / per;
                const int64_t to = y0 + t * row + N * (c - t * per);
                u32x4_t z;
#pragma unroll
                for (int j = 0; j < N / 4; ++j) {
                    const f32x2_t lo = e4m3_pair<false>(w[s][i][j]) * scale[s];
                    const f32x2_t hi = e4m3_pair<true>(w[s][i][j]) * scale[s];
                    if constexpr (BF16) {
                        z[2 * j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(lo, bf16x2_t));
                        z[2 * j + 1] = __builtin_bit_cast(uint32_t, __builtin_convertvector(hi, bf16x2_t));
                    } else {
                        z = u32x4_t{f2u(lo.x), f2u(lo.y), f2u(hi.x), f2u(hi.y)};
                    }
                }
                __builtin_nontemporal_store(z, (u32x4_t *)((uint8_t *)y[s] + to * (BF16 ? 2 : 4)));
            }
    }
}

// Threads of a workgroup: one wave where a sequence has a few new tokens.
int kv_threads(const KvBatch &B, const KvCache &C) {
    const int64_t per = B.tokens / B.seqs;  // new tokens of a sequence, on average
    return std::min<int64_t>(per, C.block) * (C.dim / 8) <= KV_HELD * WAVE ? WAVE : 256;
}

}  // namespace

hipError_t launch_kv_write(const KvCache &C, const KvBatch &B, const void *k, const void *v,
                           bool bf16, int64_t k_token, int64_t k_head, int64_t v_token,
                           int64_t v_head, int32_t *status, hipStream_t s) {
    const dim3 grid = kv_grid(C, B), threads(kv_threads(B, C));
    if (bf16)
        hipLaunchKernelGGL(kv_write_kernel<true>, grid, threads, 0, s, C, B, k, k_token, k_head, v,
                           v_token, v_head, status);
    else
        hipLaunchKernelGGL(kv_write_kernel<false>, grid, threads, 0, s, C, B, k, k_token, k_head,
                           v, v_token, v_head, status);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &C, const KvBatch &B, void *k, void *v, bool bf16,
                          int32_t *status, hipStream_t s) {
    const dim3 grid = kv_grid(C, B), threads(kv_threads(B, C));
    if (bf16)
        hipLaunchKernelGGL(kv_read_kernel<true>, grid, threads, 0, s, C, B, k, v, status);
    else
        hipLaunchKernelGGL(kv_read_kernel<false>, grid, threads, 0, s, C, B, k, v, status);
    return hipGetLastError();
}

}  // namespace fp4dev

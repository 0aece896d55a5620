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
// workgroup has one (page, head, half): it needs no other's amax, and the
// page's codes are one contiguous piece.
#include <algorithm>

#include "fp4_kernels.h"
#include "fp4_kv.h"

namespace fp4dev {
namespace {

constexpr int KV_HELD = 4;  // 8-value chunks a lane holds between amax and rounding

template <bool BF16>
__device__ __forceinline__ void load_chunk(const void *x, int64_t at, float (&v)[8]) {
    if constexpr (BF16) {
        widen_bf16x8(*(const uint4 *)((const uint16_t *)x + at), v);
    } else {
        const uint4 *p = (const uint4 *)((const float *)x + at);
        widen_f32x8(p[0], p[1], v);
    }
}

// The largest finite magnitude; whether any value was not finite.
__device__ __forceinline__ bool chunk_amax(const float (&v)[8], float &amax) {
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
__device__ __forceinline__ uint2 chunk_codes(const float (&v)[8], float inv) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = __builtin_fabsf(v[i]) < __builtin_inff() ? v[i] * inv : __builtin_nanf("");
    return make_uint2(cvt_e4m3x4(q[0], q[1], q[2], q[3]), cvt_e4m3x4(q[4], q[5], q[6], q[7]));
}

struct KvStrides {
    int64_t k_token, k_head, v_token, v_head;
};

// Grid: x the batch's items of one page, y heads, z keys or values.
template <bool BF16>
__global__ __launch_bounds__(256) void kv_write_kernel(KvCache C, KvBatch B, const void *k,
                                                       const void *v, KvStrides S,
                                                       int32_t *status) {
    const Item it = find_item(B, (int)blockIdx.x, C.block, 2);
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
    const int head = blockIdx.y;
    const bool values = blockIdx.z != 0;
    const int slot0 = (int)(p0 - (b << C.block_shift)), n = (int)(p1 - p0);
    const int64_t t0 = it.base + (p0 - start);
    const void *x = values ? v : k;
    const int64_t ts = values ? S.v_token : S.k_token;
    const int64_t x0 = t0 * ts + head * (values ? S.v_head : S.k_head);
    uint8_t *codes = (values ? C.v_codes : C.k_codes) + page_offset(C, page, head);
    uint8_t *scale = (values ? C.v_scales : C.k_scales) + (int64_t)page * C.heads + head;
    const uint32_t before = slot0 > 0 ? *scale : 0u;

    const int per = C.dim >> 3;  // chunks of a token: 8, 16, 24 or 32
    const int chunks = n * per;
    const bool held = chunks <= KV_HELD * (int)blockDim.x;
    float amax = 0.0f, x8[KV_HELD][8];
    bool bad = false;
    if (held) {
#pragma unroll
        for (int i = 0; i < KV_HELD; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < chunks) {
                const int t = c / per;
                load_chunk<BF16>(x, x0 + t * ts + 8 * (c - t * per), x8[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < KV_HELD; ++i)
            if (threadIdx.x + i * blockDim.x < (uint32_t)chunks) bad |= chunk_amax(x8[i], amax);
    } else {
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            const int t = c / per;
            load_chunk<BF16>(x, x0 + t * ts + 8 * (c - t * per), x8[0]);
            bad |= chunk_amax(x8[0], amax);
        }
    }
    // non-negative floats order as their bits
    uint32_t top = wave_max_u32(f2u(amax));
    if (blockDim.x > WAVE) {
        __shared__ uint32_t part[256 / WAVE];
        if ((threadIdx.x & (WAVE - 1)) == 0) part[threadIdx.x / WAVE] = top;
        __syncthreads();
        top = max(max(part[0], part[1]), max(part[2], part[3]));
    }
    if (__ballot(bad) != 0 && (threadIdx.x & (WAVE - 1)) == 0) flag(status, FLAG_NONFINITE);

    const uint32_t byte = max(kv_scale_byte(u2f(top)), before);
    const float inv = e8m0_value(254u - min(byte, 254u)) * (byte == 255u ? __builtin_nanf("") : 1.0f);
    if (held) {
#pragma unroll
        for (int i = 0; i < KV_HELD; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c < chunks) *(uint2 *)(codes + slot0 * C.dim + 8 * c) = chunk_codes(x8[i], inv);
        }
    } else {
        for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
            const int t = c / per;
            load_chunk<BF16>(x, x0 + t * ts + 8 * (c - t * per), x8[0]);
            *(uint2 *)(codes + slot0 * C.dim + 8 * c) = chunk_codes(x8[0], inv);
        }
    }
    if (byte > before && slot0 > 0) {
        // 448 2^-20 rounds to zero, and so does all below
        const float down = u2f((127u - min(byte - before, 40u)) << 23);
        for (int c = threadIdx.x; c < slot0 * per; c += blockDim.x) {
            uint2 w = *(const uint2 *)(codes + 8 * c);
            const f32x2_t a = e4m3_pair<false>(w.x), d = e4m3_pair<true>(w.x);
            const f32x2_t e = e4m3_pair<false>(w.y), g = e4m3_pair<true>(w.y);
            w.x = cvt_e4m3x4(a.x * down, a.y * down, d.x * down, d.y * down);
            w.y = cvt_e4m3x4(e.x * down, e.y * down, g.x * down, g.y * down);
            *(uint2 *)(codes + 8 * c) = w;
        }
    }
    if (threadIdx.x == 0) *scale = (uint8_t)byte;
}

// Grid as the write's; y rows are [tokens, heads, dim].
template <bool BF16>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache C, KvBatch B, void *k, void *v,
                                                      int32_t *status) {
    const Item it = find_item(B, (int)blockIdx.x, C.block, 2);
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
    const int head = blockIdx.y;
    const bool values = blockIdx.z != 0;
    const int64_t off = page < 0 ? 0 : page_offset(C, page, head);
    const uint8_t *codes = (values ? C.v_codes : C.k_codes) + off +
                           (int)(p0 - (b << C.block_shift)) * C.dim;
    const uint32_t byte =
        page < 0 ? 127u : (values ? C.v_scales : C.k_scales)[(int64_t)page * C.heads + head];
    const float scale = e8m0_value(byte);
    const int per = C.dim >> 3;
    const int chunks = (int)(p1 - p0) * per;
    void *y = values ? v : k;
    const int64_t row = (int64_t)C.heads * C.dim;
    const int64_t y0 = (it.base + (p0 - start)) * row + (int64_t)head * C.dim;
    for (int c = threadIdx.x; c < chunks; c += blockDim.x) {
        const int t = c / per;
        const int64_t at = y0 + t * row + 8 * (c - t * per);
        const uint2 w = page < 0 ? make_uint2(0, 0) : *(const uint2 *)(codes + 8 * c);
        const f32x2_t a = e4m3_pair<false>(w.x) * scale, d = e4m3_pair<true>(w.x) * scale;
        const f32x2_t e = e4m3_pair<false>(w.y) * scale, g = e4m3_pair<true>(w.y) * scale;
        if constexpr (BF16) {
            const uint4 o = make_uint4(
                __builtin_bit_cast(uint32_t, __builtin_convertvector(a, bf16x2_t)),
                __builtin_bit_cast(uint32_t, __builtin_convertvector(d, bf16x2_t)),
                __builtin_bit_cast(uint32_t, __builtin_convertvector(e, bf16x2_t)),
                __builtin_bit_cast(uint32_t, __builtin_convertvector(g, bf16x2_t)));
            *(uint4 *)((uint16_t *)y + at) = o;
        } else {
            float4 *o = (float4 *)((float *)y + at);
            o[0] = make_float4(a.x, a.y, d.x, d.y);
            o[1] = make_float4(e.x, e.y, g.x, g.y);
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
    const dim3 grid((uint32_t)item_count(B.tokens, B.seqs, C.block, 2), C.heads, 2);
    const KvStrides st{k_token, k_head, v_token, v_head};
    const int threads = kv_threads(B, C);
    if (bf16)
        hipLaunchKernelGGL(kv_write_kernel<true>, grid, dim3(threads), 0, s, C, B, k, v, st, status);
    else
        hipLaunchKernelGGL(kv_write_kernel<false>, grid, dim3(threads), 0, s, C, B, k, v, st, status);
    return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache &C, const KvBatch &B, void *k, void *v, bool bf16,
                          int32_t *status, hipStream_t s) {
    const dim3 grid((uint32_t)item_count(B.tokens, B.seqs, C.block, 2), C.heads, 2);
    const int threads = kv_threads(B, C);
    if (bf16)
        hipLaunchKernelGGL(kv_read_kernel<true>, grid, dim3(threads), 0, s, C, B, k, v, status);
    else
        hipLaunchKernelGGL(kv_read_kernel<false>, grid, dim3(threads), 0, s, C, B, k, v, status);
    return hipGetLastError();
}

}  // namespace fp4dev

// fp4_kv.h - the 8-bit key/value cache: kernel arguments, the batch's map from
// grid to pages, and E4M3 conversion.  Internal to libfp4.so.
//
// A cache page holds `block` tokens.  Per page and kv head it has block x D
// E4M3FN codes (token-major) and one E8M0 byte, for keys and for values; a
// code stands for E4M3(code) 2^(byte - 127).  Pages are far apart in a long
// cache, so every page address is 64-bit; inside a page offsets fit 32 bits.
#pragma once

#include "fp4_device.h"

namespace fp4dev {

constexpr uint32_t FLAG_CACHE_INDEX = 8;

struct KvCache {
    uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
    int32_t pages, heads, block, block_shift, dim;
};

struct KvBatch {
    const int32_t *cu, *lengths, *table;
    int64_t table_stride;
    int32_t seqs, width, tokens;
};

// First code of a page and head.
__device__ __forceinline__ int64_t page_offset(const KvCache &C, int page, int head) {
    return ((int64_t)page * C.heads + head) * (C.block * C.dim);
}

__device__ __forceinline__ void flag(int32_t *status, uint32_t bits) {
    if (status != nullptr) atomicOr(status, (int32_t)bits);
}

// A work item of a launch over (sequence, piece): the host does not know the
// sequences' token counts, so sequence s owns the items from
//   first(s) = cu[s] / unit + extra s
// on, which is at least as many as its pieces of up to `unit` tokens, whatever
// they start at: n tokens from a unit's start make ceil(n / unit) <=
// floor difference + 1 pieces (extra 1), from inside a unit one more (extra
// 2).  Items past a sequence's pieces end at once.  Sequence `seqs` stands for
// the rows past cu[seqs].  The search reads 64 candidates at a time, one per
// lane: one step up to 62 sequences, two up to some 4000.
struct Item {
    int seq, piece, base, count;  // base, count: the sequence's rows [base, base + count)
    int length;                   // the sequence's tokens
};

// cu is prefix sums from 0 to at most `tokens`: item i of `items` looks at its
// entries from 64 i on, one a lane, and at those a multiple of 64 items further.
// The search reads only some of them, so of others it would not know.  The
// entries come with the search's first ones; `leader`, one workgroup an item,
// flags.
struct RowsSeen {
    int at, base, next;
};

__device__ __forceinline__ RowsSeen load_rows(const KvBatch &B, int64_t at) {
    const int i = (int)min(at, (int64_t)B.seqs);
    return {i, B.cu[i], B.cu[min(i + 1, B.seqs)]};
}

__device__ __forceinline__ bool rows_bad(const KvBatch &B, const RowsSeen &r) {
    return r.at == 0 ? r.base != 0 || r.next < 0 || r.next > B.tokens
                     : r.base < 0 || r.next < r.base || r.next > B.tokens;
}

__device__ __forceinline__ Item search_item(const KvBatch &B, int item, int unit, int extra) {
    const int lane = threadIdx.x & (WAVE - 1);
    int lo = 0, n = B.seqs + 1;
    while (n >= WAVE) {
        const int step = (n + WAVE - 1) / WAVE;
        const int i = lo + lane * step;
        const bool at = lane * step < n && B.cu[i] / unit + extra * i <= item;
        const uint64_t b = __ballot(at);
        const int k = b ? 63 - __builtin_clzll(b) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    // the last step's lanes also hold what comes with the sequence found
    const int i = min(lo + lane, B.seqs);
    const int cu = B.cu[i], len = B.lengths[min(i, B.seqs - 1)];
    const uint64_t b = __ballot(lane < n && cu / unit + extra * i <= item);
    const int k = b ? 63 - __builtin_clzll(b) : 0;
    Item it;
    it.seq = __builtin_amdgcn_readfirstlane(lo + k);
    it.base = __builtin_amdgcn_readlane(cu, k);
    it.length = __builtin_amdgcn_readlane(len, k);
    it.piece = item - (it.base / unit + extra * it.seq);
    it.count = (it.seq < B.seqs ? __builtin_amdgcn_readlane(cu, k + 1) : B.tokens) - it.base;
    // a cu that is no prefix sum of at most `tokens` rows gives no piece
    if (it.base < 0 || it.count < 0 || it.base > B.tokens || it.count > B.tokens - it.base ||
        it.piece < 0)
        it.count = -1;
    return it;
}

__device__ __forceinline__ Item find_item(const KvBatch &B, int item, int64_t items, int unit,
                                          int extra, bool leader, int32_t *status) {
    const int64_t first = (int64_t)item * WAVE + (threadIdx.x & (WAVE - 1));
    const RowsSeen seen = load_rows(B, first);
    const Item it = search_item(B, item, unit, extra);
    if (leader && status != nullptr && threadIdx.x < WAVE) {
        bool bad = rows_bad(B, seen);
        for (int64_t i = first + items * WAVE; i <= B.seqs; i += items * WAVE)
            bad = bad || rows_bad(B, load_rows(B, i));
        if (__ballot(bad) != 0 && threadIdx.x == 0) flag(status, FLAG_CACHE_INDEX);
    }
    return it;
}

// The same launch's items without gaps: item i is the i-th piece there is, and
// what has none comes last.  A lane counts the pieces of up to TILE_SEQS / 64
// sequences, and the wave adds them up.  Items that own nothing end at once, but
// between others they leave shader engines, which get workgroups in turn, with
// less to do: attention of 8 x 4 tokens over 4096 keys, 8 x 8 heads, 32 us, with
// every second item empty 49.
constexpr int TILE_SEQS = 256;  // with the rows past the last one

__device__ __forceinline__ Item find_tile(const KvBatch &B, int item, int unit, int32_t *status) {
    constexpr int K = TILE_SEQS / WAVE;
    const int lane = threadIdx.x & (WAVE - 1);
    const int n = B.seqs + 1, each = (n + WAVE - 1) / WAVE;
    int base[K], count[K], length[K], pieces[K], sum = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int s = lane * each + k;
        base[k] = count[k] = length[k] = pieces[k] = 0;
        if (k < each && s < n) {
            base[k] = B.cu[s];
            length[k] = B.lengths[min(s, B.seqs - 1)];
            const int next = s < B.seqs ? B.cu[s + 1] : B.tokens;
            if (s == 0 ? base[k] != 0 || next < 0 || next > B.tokens
                       : base[k] < 0 || next < base[k] || next > B.tokens) {
                if (item == 0 && threadIdx.x < WAVE) flag(status, FLAG_CACHE_INDEX);
            } else {
                count[k] = next - base[k];
                pieces[k] = (int)((uint32_t)(count[k] + unit - 1) / (uint32_t)unit);
            }
        }
        sum += pieces[k];
    }
    int last = sum;
#pragma unroll
    for (int off = 1; off < WAVE; off <<= 1) {
        const int below = __shfl_up(last, off, WAVE);
        if (lane >= off) last += below;
    }
    const uint64_t b = __ballot(item < last && item >= last - sum);
    Item it = {0, 0, 0, 0, 0};
    if (b == 0) return it;
    const int at = __builtin_ctzll(b);
    it.piece = item - __builtin_amdgcn_readlane(last - sum, at);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int here = __builtin_amdgcn_readlane(pieces[k], at);
        if (it.piece >= 0 && it.piece < here) {
            it.seq = at * each + k;
            it.base = __builtin_amdgcn_readlane(base[k], at);
            it.count = __builtin_amdgcn_readlane(count[k], at);
            it.length = __builtin_amdgcn_readlane(length[k], at);
            break;
        }
        it.piece -= here;
    }
    return it;
}

inline int64_t item_count(int64_t tokens, int64_t seqs, int unit, int extra) {
    return tokens / unit + extra * (seqs + 1);
}

// The page that holds positions [block b of sequence s], or -1 (flagged by
// the caller) when the table has none or names none of the cache's.
__device__ __forceinline__ int find_page(const KvBatch &B, const KvCache &C, int s, int64_t b) {
    if (b < 0 || b >= B.width) return -1;
    const int page = B.table[(int64_t)s * B.table_stride + b];
    return (uint32_t)page < (uint32_t)C.pages ? page : -1;
}

// 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 is NaN.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
    return byte == 0u ? 0x1p-127f : (byte == 255u ? __builtin_nanf("") : u2f(byte << 23));
}

// The page's scale byte: the smallest e >= -127 with 448 2^e >= amax, so
// nothing saturates.  For a normal amax = m 2^(E-127), m in [1, 2), that is
// e = E - 127 - 8 + [m > 1.75], since 448 = 1.75 2^8; a zero page takes byte 0,
// the neutral element of the maximum that joins scales.
__device__ __forceinline__ uint32_t kv_scale_byte(float amax) {
    const uint32_t b = f2u(amax);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e > 0 ? (uint32_t)e : 0u;
}

// Four E4M3 codes of four values, nearest with ties to the even code.  The
// callers keep |q| <= 448, or NaN.
__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

template <bool HI>
__device__ __forceinline__ f32x2_t e4m3_pair(uint32_t codes) {
    return __builtin_amdgcn_cvt_pk_f32_fp8((int)codes, HI);
}

}  // namespace fp4dev

// fp4_attention.hip - attention over the 8-bit key/value cache.
//
//   S_rj = scale q_r . k_j over the visible keys j of row r,
//   out_r = sum_j exp(S_rj - m_r) v_j / sum_j exp(S_rj - m_r),  m_r = max_j S_rj.
//
// One pass over the keys with a running maximum and sum per row, both fp32.
#include <algorithm>

#include "fp4_kernels.h"
#include "fp4_kv.h"

namespace fp4dev {
namespace {

struct AttnArgs {
    const void *q;
    int64_t q_token, q_head;
    void *out;
    float *lse;
    int32_t heads, group, causal, window;
    float scale;
};

__device__ __forceinline__ float load_q(const void *q, int64_t at, bool bf16) {
    return bf16 ? u2f((uint32_t)((const uint16_t *)q)[at] << 16) : ((const float *)q)[at];
}

// One wave per query row.  A step takes 64 keys, one per lane for the scores;
// then a lane has every 64th dimension of the output.
template <bool BF16>
__global__ __launch_bounds__(WAVE) void attention_simple_kernel(KvCache C, KvBatch B, AttnArgs A,
                                                                int32_t *status) {
    __shared__ float qs[256], ps[WAVE];
    __shared__ int64_t vrow[WAVE];
    __shared__ float vsc[WAVE];
    const int lane = threadIdx.x;
    const int64_t t = blockIdx.x;
    const int hq = blockIdx.y, head = hq / A.group;
    const Item it = find_item(B, (int)t, 0, 0);
    const int D = C.dim;
    for (int d = lane; d < D; d += WAVE)
        qs[d] = load_q(A.q, t * A.q_token + hq * A.q_head + d, BF16) * A.scale;
    __syncthreads();
    const bool real = it.count > 0 && it.seq < B.seqs;
    const int64_t len = real ? B.lengths[it.seq] : 0;
    const int64_t pos = len - it.count + (t - it.base);
    const int64_t last = real ? (A.causal ? pos : len - 1) : -1;
    const int64_t first = A.window ? max(pos - A.window + 1, (int64_t)0) : 0;
    float m = -__builtin_inff(), l = 0.0f, o[4] = {0, 0, 0, 0};
    for (int64_t j0 = first; j0 <= last; j0 += WAVE) {
        const int64_t j = j0 + lane;
        const int page = j <= last ? find_page(B, C, it.seq, j >> C.block_shift) : -1;
        if (j <= last && page < 0) flag(status, FLAG_CACHE_INDEX);
        float s = -__builtin_inff();
        int64_t at = 0;
        if (page >= 0) {
            at = page_offset(C, page, head) + (j & (C.block - 1)) * D;
            float dot = 0.0f;
            for (int d = 0; d < D; d += 4) {
                const uint32_t w = *(const uint32_t *)(C.k_codes + at + d);
                const f32x2_t a = e4m3_pair<false>(w), b = e4m3_pair<true>(w);
                dot = __builtin_fmaf(qs[d], a.x, dot);
                dot = __builtin_fmaf(qs[d + 1], a.y, dot);
                dot = __builtin_fmaf(qs[d + 2], b.x, dot);
                dot = __builtin_fmaf(qs[d + 3], b.y, dot);
            }
            s = dot * e8m0_value(C.k_scales[(int64_t)page * C.heads + head]);
            vsc[lane] = e8m0_value(C.v_scales[(int64_t)page * C.heads + head]);
        }
        vrow[lane] = page >= 0 ? at : -1;
        float top = s;
        for (int off = 32; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off, WAVE));
        // a NaN score makes its row NaN: the maximum skips it, the sum does not
        const float next = __builtin_fmaxf(m, top);
        const float ref = next == -__builtin_inff() ? 0.0f : next;
        const float p = __expf(s - ref), keep = __expf(m - ref);
        m = next;
        float sum = p;
        for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, WAVE);
        l = __builtin_fmaf(l, keep, sum);
        ps[lane] = p;
        __syncthreads();
        for (int i = 0; i < 4; ++i) o[i] *= keep;
        for (int k = 0; k < WAVE; ++k) {
            if (vrow[k] < 0) continue;
            const float pk = ps[k] * vsc[k];
            for (int i = 0; i * WAVE < D; ++i) {
                const f32x2_t v = e4m3_pair<false>(C.v_codes[vrow[k] + lane + i * WAVE]);
                o[i] = __builtin_fmaf(pk, v.x, o[i]);
            }
        }
        __syncthreads();
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const int64_t row = t * A.heads + hq;
    for (int i = 0; i * WAVE < D; ++i) {
        const float y = o[i] * inv;
        const int64_t at = row * D + lane + i * WAVE;
        if (BF16)
            ((__bf16 *)A.out)[at] = (__bf16)y;
        else
            ((float *)A.out)[at] = y;
    }
    if (A.lse != nullptr && lane == 0)
        A.lse[row] = l == 0.0f ? -__builtin_inff() : (m == -__builtin_inff() ? 0.0f : m) + __logf(l);
}

}  // namespace

size_t attention_workspace_bytes(const KvCache &C, const KvBatch &B, int heads) {
    (void)C;
    (void)B;
    (void)heads;
    return 0;
}

hipError_t launch_attention(const KvCache &C, const KvBatch &B, const void *q, int64_t q_token,
                            int64_t q_head, bool bf16, int heads, float scale, bool causal,
                            int window, void *out, float *lse, void *workspace, int32_t *status,
                            hipStream_t s) {
    (void)workspace;
    const AttnArgs A{q, q_token, q_head, out, lse, heads, heads / C.heads, causal, window, scale};
    const dim3 grid((uint32_t)B.tokens, (uint32_t)heads);
    if (bf16)
        hipLaunchKernelGGL(attention_simple_kernel<true>, grid, dim3(WAVE), 0, s, C, B, A, status);
    else
        hipLaunchKernelGGL(attention_simple_kernel<false>, grid, dim3(WAVE), 0, s, C, B, A, status);
    return hipGetLastError();
}

}  // namespace fp4dev

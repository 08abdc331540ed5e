// moe_tree_attn.cuh -- attention of the drafted tokens of each sequence (one
// token, a chain, or a tree) over the quantised paged cache.
//
//   o = sum_j softmax_j(scale q . K_j | j seen) V_j
// in one pass over the cache: a running maximum m and sum l of each row,
// o and l scaled by e^(m - m') when the maximum rises.
#pragma once
#include <cuda_bf16.h>

#include "moe_kv.cuh"

namespace moe {

struct TreeArgs {
    KvDims k;
    const uint8_t *pages;
    int n_pages;
    const uint16_t *q;
    long long q_tok, q_head;  // strides, elements
    uint16_t *out;
    long long o_tok, o_head;
    const int32_t *q_start;   // [batch + 1]
    const int32_t *kv_len;    // [batch]
    const int32_t *table;     // [batch, table_stride]
    long long table_stride;
    int table_pages;          // pages a sequence can have
    const unsigned long long *mask;  // [tokens] or NULL: causal
    int batch, tokens, q_heads;
    float scale;
    uint32_t *ctrl;
};

// rows and length of a sequence, checked; n = 0 where they do not hold
__device__ __forceinline__ void tree_sequence(const TreeArgs &a, int b, int &first, int &n, int &len)
{
    first = a.q_start[b];
    n = a.q_start[b + 1] - first;
    len = a.kv_len[b];
    const bool ok = first >= 0 && n >= 0 && n <= MOE_MAX_DRAFT && first + n <= a.tokens && len >= n &&
                    len <= (long long)a.table_pages * a.k.page;
    if (!ok) {
        atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_INDEX);
        n = 0;
    }
}

// One warp a query row (token and head), lanes over the dimensions.
__global__ void __launch_bounds__(128) moe_tree_attn_kernel(const TreeArgs a)
{
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= a.tokens * a.q_heads)
        return;
    const int token = row / a.q_heads, head = row % a.q_heads, kvh = head / (a.q_heads / a.k.heads);
    int first = 0, n = 0, len = 0, b = 0;
    for (; b < a.batch; ++b) {
        tree_sequence(a, b, first, n, len);
        if (token >= first && token < first + n)
            break;
    }
    if (b == a.batch)  // a row of no sequence, or of one whose length does not hold
        n = len = 0;
    const int i = max(0, min(token - first, MOE_MAX_DRAFT - 1)), per = a.k.dim / 32, d0 = lane * per;
    const unsigned long long mask = a.mask ? a.mask[token] : (2ull << i) - 1;
    float q[8], o[8], top = -INFINITY, sum = 0.0f;
    for (int e = 0; e < per; ++e) {
        q[e] = bf16_to_f32(a.q[token * a.q_tok + head * a.q_head + d0 + e]) * a.scale;
        o[e] = 0.0f;
    }
    for (int j = 0; j < len; ++j) {
        const int place = j - (len - n);
        if (place >= 0 && !(mask >> place & 1))
            continue;
        const int page = a.table[b * a.table_stride + j / a.k.page];
        if (page < 0 || page >= a.n_pages) {
            atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_INDEX);
            continue;
        }
        const int in = j % a.k.page, t = in % 16;
        const uint8_t *blk = a.pages + (((size_t)page * a.k.heads + kvh) * (a.k.page / 16) + in / 16) * a.k.block_bytes();
        float v[8], s = 0.0f;
        kv_values8(a.k, blk, false, t, d0 / 8, v);
        for (int e = 0; e < per; ++e)
            s = fmaf(q[e], v[d0 % 8 + e], s);
        for (int m = 16; m; m /= 2)
            s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
        const float up = fmaxf(top, s), keep = expf(top - up), p = expf(s - up);
        top = up;
        sum = sum * keep + p;
        kv_values8(a.k, blk + a.k.half_bytes(), true, t, d0 / 8, v);
        for (int e = 0; e < per; ++e)
            o[e] = fmaf(p, v[d0 % 8 + e], o[e] * keep);
    }
    for (int e = 0; e < per; ++e)
        a.out[token * a.o_tok + head * a.o_head + d0 + e] = __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.0f ? 0.0f : o[e] / sum));
}

}  // namespace moe

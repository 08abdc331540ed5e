// moe_latent_attn.cuh -- latent attention in expanded form, over a prompt's keys
// and values.
//
// A CTA works on one query row of one head: tiles of 32 tokens, a score by a warp
// at a time, one pass with a running maximum and sum, a thread a few dimensions
// of the output.
#pragma once
#include "moe_latent.cuh"

namespace moe {

#define MOE_ROW_THREADS 128
#define MOE_ROW_TILE 32

struct PromptArgs {
    const uint16_t *q, *k, *kr, *v;
    uint16_t *out;
    long long q_tok, q_head, k_tok, k_head, kr_tok, v_tok, v_head, o_tok, o_head;
    const int32_t *q_start, *kv_start;
    int batch, heads, nope, rope, q_tokens, kv_tokens, causal;
    float scale;
    uint32_t *status;
};

// one row: qs [dims] in shared memory; key(j, d), value(j, d), seen(j); out(d, x)
template <typename K, typename V, typename S, typename O>
__device__ __forceinline__ void row_attention(const float *qs, int dims, int vdims, int len, float scale, K key, V value,
                                              S seen, O out)
{
    __shared__ float score[MOE_ROW_TILE];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < len; j0 += MOE_ROW_TILE) {
        __syncthreads();
        for (int j = warp; j < MOE_ROW_TILE; j += MOE_ROW_THREADS / 32) {
            float s = 0.0f;
            const bool live = j0 + j < len && seen(j0 + j);
            if (live)
                for (int d = lane; d < dims; d += 32)
                    s = fmaf(qs[d], key(j0 + j, d), s);
            s = warp_sum(s);
            if (lane == 0)
                score[j] = live ? s * scale : -INFINITY;
        }
        __syncthreads();
        float top = m;
        for (int j = 0; j < MOE_ROW_TILE; ++j)
            top = fmaxf(top, score[j]);
        const float ref = top == -INFINITY ? 0.0f : top, f = m == -INFINITY ? 0.0f : __expf(m - ref);
        l *= f;
        for (int i = 0; i < 4; ++i)
            o[i] *= f;
        m = top;
        for (int j = 0; j < MOE_ROW_TILE && j0 + j < len; ++j) {
            if (!seen(j0 + j))
                continue;
            const float w = __expf(score[j] - ref);
            l += w;
            for (int i = 0, d = tid; d < vdims; d += MOE_ROW_THREADS, ++i)
                o[i] = fmaf(w, value(j0 + j, d), o[i]);
        }
    }
    for (int i = 0, d = tid; d < vdims; d += MOE_ROW_THREADS, ++i)
        out(d, l == 0.0f ? 0.0f : o[i] / l);
}

__global__ void __launch_bounds__(MOE_ROW_THREADS) moe_prompt_row_kernel(const __grid_constant__ PromptArgs a)
{
    __shared__ float qs[192];
    __shared__ int which;
    pdl_wait();
    const int token = blockIdx.x, head = blockIdx.y;
    if (threadIdx.x == 0)
        which = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < a.batch; b += MOE_ROW_THREADS)
        if (a.q_start[b] <= token && token < a.q_start[b + 1])
            which = b;
    __syncthreads();
    const int b = which;
    if (b < 0)
        return;
    const int q0 = a.q_start[b], n = a.q_start[b + 1] - q0, k0 = a.kv_start[b], len = a.kv_start[b + 1] - k0;
    uint16_t *out = a.out + token * a.o_tok + head * a.o_head;
    if (q0 < 0 || q0 > a.q_tokens - n || k0 < 0 || len < 0 || k0 > a.kv_tokens - len) {
        if (threadIdx.x == 0 && a.status)
            atomicOr(a.status, (uint32_t)MOE_WS_INDEX);
        for (int d = threadIdx.x; d < a.nope; d += MOE_ROW_THREADS)
            out[d] = 0;
        return;
    }
    for (int d = threadIdx.x; d < a.nope + a.rope; d += MOE_ROW_THREADS)
        qs[d] = bf16_to_f32(a.q[token * a.q_tok + head * a.q_head + d]);
    const int last = a.causal ? len - n + token - q0 : len - 1;
    row_attention(
        qs, a.nope + a.rope, a.nope, max(0, min(len, last + 1)), a.scale,
        [&](int j, int d) {
            return bf16_to_f32(d < a.nope ? a.k[(k0 + j) * a.k_tok + head * a.k_head + d] : a.kr[(k0 + j) * a.kr_tok + d - a.nope]);
        },
        [&](int j, int d) { return bf16_to_f32(a.v[(k0 + j) * a.v_tok + head * a.v_head + d]); }, [](int) { return true; },
        [&](int d, float x) { out[d] = (uint16_t)pack_bf2(x, x); });
}

}  // namespace moe

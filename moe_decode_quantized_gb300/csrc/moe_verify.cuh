// moe_verify.cuh -- verification of drafted tokens against the target's
// logits with given random numbers.
//
// Sequence b has n rows of logits, row 0 of its last accepted token and row j
// of drafted node j. With p_j = softmax(logits_j / T) and r = p_0, Z = 1 at
// cur = 0, each node j = 1 .. n - 1 whose parent is cur is accepted when
// u_j Z q_j(x_j) < r(x_j) (then cur = j, r = p_j, Z = 1) and otherwise taken
// out of the residual, r = max(r - Z q_j, 0), Z = sum r. The next token is
// argmax r_i / e_i with e_i exponential numbers: a sample of r / Z. Only the
// rows on the accepted path are ever needed.
#pragma once
#include "moe_common.cuh"

namespace moe {

struct VerifyArgs {
    const void *logits;
    int f32;
    long long stride;
    const int32_t *q_start, *tokens, *parents;
    const float *draft;
    long long draft_stride;
    const float *temperature, *uniforms, *noise;
    long long noise_stride;
    int batch, rows, vocab;
    int32_t *n_accepted, *path, *next;
    uint32_t *ctrl;
};

__device__ __forceinline__ float verify_logit(const VerifyArgs &a, long long row, int i)
{
    return a.f32 ? static_cast<const float *>(a.logits)[row * a.stride + i]
                 : bf16_to_f32(static_cast<const uint16_t *>(a.logits)[row * a.stride + i]);
}

#define MOE_VERIFY_THREADS 1024

// value and index of the largest (lowest index of equals) over the CTA
__device__ __forceinline__ void cta_argmax(float &v, int &i, float *sv, int *si)
{
    for (int m = 16; m; m /= 2) {
        const float w = __shfl_xor_sync(0xFFFFFFFFu, v, m);
        const int k = __shfl_xor_sync(0xFFFFFFFFu, i, m);
        if (w > v || (w == v && k < i)) {
            v = w;
            i = k;
        }
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        sv[threadIdx.x / 32] = v;
        si[threadIdx.x / 32] = i;
    }
    __syncthreads();
    v = sv[0];
    i = si[0];
    for (int w = 1; w < MOE_VERIFY_THREADS / 32; ++w)
        if (sv[w] > v || (sv[w] == v && si[w] < i)) {
            v = sv[w];
            i = si[w];
        }
}

__device__ __forceinline__ float cta_sum(float v, float *sv)
{
    for (int m = 16; m; m /= 2)
        v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        sv[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.0f;
    for (int w = 0; w < MOE_VERIFY_THREADS / 32; ++w)
        v += sv[w];
    return v;
}

// One CTA a sequence. r is recomputed from the logits and the rejected
// nodes' draft rows wherever it is needed.
__global__ void __launch_bounds__(MOE_VERIFY_THREADS) moe_verify_kernel(const VerifyArgs a)
{
    __shared__ float sv[32];
    __shared__ int si[32];
    __shared__ int rejected[MOE_MAX_DRAFT];
    __shared__ float zed[MOE_MAX_DRAFT + 1];  // Z before each rejection
    const int b = blockIdx.x, tid = threadIdx.x;
    const int first = a.q_start[b], n = a.q_start[b + 1] - first;
    if (first < 0 || n < 0 || n > MOE_MAX_DRAFT || first + n > a.rows || n == 0) {
        if (tid == 0) {
            if (n != 0)
                atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_INDEX);
            a.n_accepted[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    const float temp = a.temperature ? a.temperature[b] : 1.0f;
    const bool greedy = !(temp > 0.0f) || !a.noise;
    const float c = greedy ? 0.0f : 1.4426950408889634f / temp;
    int cur = 0, count = 0, nrej = 0, next = -1;
    float top = 0.0f, total = 0.0f;
    int best = 0;
    bool fresh = true;

    auto weight = [&](int row, int i) {  // e^((l - top) / T)
        const float l = verify_logit(a, first + row, i), d = l - top;
        if (!(l < INFINITY) || l == -INFINITY)
            return 0.0f;
        return greedy ? (i == best ? 1.0f : 0.0f) : d >= 0.0f ? 1.0f : exp2f(d * c);
    };
    auto residual = [&](int i) {
        float r = weight(cur, i);
        for (int k = 0; k < nrej; ++k) {
            const float q = a.draft ? a.draft[(long long)(first + rejected[k]) * a.draft_stride + i]
                                    : (a.tokens[first + rejected[k]] == i ? 1.0f : 0.0f);
            r = fmaxf(r - zed[k] * q, 0.0f);
        }
        return r;
    };
    for (int j = 1; j <= n; ++j) {
        if (fresh) {  // statistics of row cur
            float v = -INFINITY;
            int at = a.vocab;
            bool odd = false;
            for (int i = tid; i < a.vocab; i += MOE_VERIFY_THREADS) {
                const float l = verify_logit(a, first + cur, i);
                odd |= !(l < INFINITY);
                if (l < INFINITY && l > v) {
                    v = l;
                    at = i;
                }
            }
            if (odd)
                atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_NONFINITE);
            cta_argmax(v, at, sv, si);
            top = v;
            best = at;
            float s = 0.0f;
            for (int i = tid; i < a.vocab; i += MOE_VERIFY_THREADS)
                s += weight(cur, i);
            total = cta_sum(s, sv);
            nrej = 0;
            fresh = false;
            __syncthreads();
            if (tid == 0)
                zed[0] = total;
            __syncthreads();
        }
        if (j == n)
            break;
        const int parent = a.parents ? a.parents[first + j] : j - 1;
        if (parent != cur)
            continue;
        const int x = a.tokens[first + j];
        if (x < 0 || x >= a.vocab) {
            if (tid == 0)
                atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_INDEX);
            continue;
        }
        const float q = a.draft ? a.draft[(long long)(first + j) * a.draft_stride + x] : 1.0f;
        const float u = a.uniforms && !greedy ? a.uniforms[first + j] : 0.5f;
        const float rx = residual(x);
        if (u * zed[nrej] * q < rx) {
            cur = j;
            fresh = true;
            if (tid == 0)
                a.path[first + count] = j;
            ++count;
            continue;
        }
        __syncthreads();
        if (tid == 0)
            rejected[nrej] = j;
        ++nrej;
        __syncthreads();
        float z;
        if (a.draft) {
            float s = 0.0f;
            for (int i = tid; i < a.vocab; i += MOE_VERIFY_THREADS)
                s += residual(i);
            z = cta_sum(s, sv);
        } else {
            z = fmaxf(zed[nrej - 1] - rx, 0.0f);
        }
        __syncthreads();
        if (tid == 0)
            zed[nrej] = z;
        __syncthreads();
    }
    if (total > 0.0f) {
        if (!(zed[nrej] > 0.0f))
            nrej = 0;
        float v = -1.0f;
        int at = a.vocab;
        for (int i = tid; i < a.vocab; i += MOE_VERIFY_THREADS) {
            const float e = greedy ? 1.0f : fmaxf(a.noise[(long long)b * a.noise_stride + i], 1.17549435e-38f);
            const float s = residual(i) / e;
            if (s > v) {
                v = s;
                at = i;
            }
        }
        cta_argmax(v, at, sv, si);
        next = at;
    }
    if (tid == 0) {
        a.n_accepted[b] = count;
        a.next[b] = next;
        for (int k = count; k < n; ++k)
            a.path[first + k] = -1;
    }
}

}  // namespace moe

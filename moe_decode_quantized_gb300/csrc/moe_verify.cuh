// moe_verify.cuh -- verification of drafted tokens against the target's
// logits with given random numbers.
//
// Sequence b has n rows of logits, row 0 of its last accepted token and row j
// of drafted node j. With p_j = softmax(logits_j / T) and r = p_0, Z = 1 at
// cur = 0, each node j = 1 .. n - 1 whose parent is cur is accepted when
// u_j Z q_j(x_j) < r(x_j) (then cur = j, r = p_j, Z = 1) and otherwise taken
// out of the residual, r = max(r - Z q_j, 0), Z = sum r. The next token is
// argmax r_i / e_i with e_i exponential numbers: a sample of r / Z.
//
// A cluster of CTAs takes a sequence, each CTA a slice of the vocabulary. r is
// kept times the row's sum of e^((l - top) / T), which no division by the sum
// then touches. Every pass over a slice ends in one exchange through the
// cluster's shared memory that gives every CTA all slices' results, and each
// makes the same decisions from them. What a row's largest logit and sum are
// comes from one of two places:
//  - a kernel that goes through all rows ahead, over the whole GPU (AHEAD);
//    the walk then has one pass, the race that ends it, and one more for each
//    rejection of a drawn token but the last;
//  - a pass of the walk over each row that the path reaches, one after the
//    other. Only what is needed is read, which for a large tree is a small
//    part, but a path of k nodes is k + 1 passes in turn.
// Bound by the latency of the passes for one sequence (a chain of 3 drafts over
// 32000: 7.2 us), by the reads for many (48 chains of 7 over 131072: 38 us, 157
// MB with the draft rows that the residuals take; 16 trees of 12 to 24 rows over
// 100003 in f32: 18 us, bound by the passes in turn).
#pragma once
#include "moe_common.cuh"

namespace moe {

#define MOE_VERIFY_THREADS 256
#define MOE_VERIFY_MAX_CLUSTER 8
#define MOE_VERIFY_STAT_THREADS 256
#define MOE_VERIFY_MAX_SPLITS 64

struct VerifySlice;

struct VerifyArgs {
    const void *logits;
    long long stride;
    const int32_t *q_start, *tokens, *parents;
    const float *draft;
    long long draft_stride;
    const float *temperature, *uniforms, *noise;
    long long noise_stride;
    int rows, vocab, slice;  // slice: of a CTA, a multiple of 8
    int32_t *n_accepted, *path, *next;
    uint32_t *ctrl;
    int batch, splits, split;  // AHEAD: parts of a row and their size, a multiple of 8
    VerifySlice *stats;  // [rows][splits]
};

// what a slice gives: a row pass its largest logit, where, and the sum of its
// weights against that logit; a race pass its best, where, and the plain sum
struct VerifySlice {
    float best, sum;
    int at;
};

// the larger value, the lower index of equals
__device__ __forceinline__ void keep_larger(float &v, int &i, float w, int k)
{
    if (w > v || (w == v && k < i)) {
        v = w;
        i = k;
    }
}

// a warp's largest value and the lowest of its indexes: two 32-bit
// reductions, the first over the floats' bits in their order (no NaN; -0 as 0)
__device__ __forceinline__ void warp_larger(float &v, int &i)
{
    const uint32_t u = __float_as_uint(v + 0.0f), key = u & 0x80000000u ? ~u : u | 0x80000000u;
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, key);
    i = (int)__reduce_min_sync(0xFFFFFFFFu, key == top ? (uint32_t)i : 0x7FFFFFFFu);
    v = __uint_as_float(top & 0x80000000u ? top & 0x7FFFFFFFu : ~top);
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_nan(float x, float y)
{
    float z;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(x), "f"(y));
    return z;
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the two halves of a barrier that orders no memory: every CTA of the cluster has started
__device__ __forceinline__ void cluster_started_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_started_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster(const void *p, uint32_t rank, uint32_t v)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

// A thread's view of [lo, hi) of rows of vocab values, eight values at a time
// (a step of the CTA is 8 NT): where rows can be read 16 bytes at a time
// (WIDE) eight consecutive ones, else every NT-th. F32: logits' type. FULL:
// the whole step lies below hi; else what does not is `fill`.
template <bool F32, bool WIDE, int NT>
struct VerifyView {
    const VerifyArgs &a;
    int hi;
    static constexpr int STEP = 8 * NT;

    __device__ __forceinline__ int place(int at, int k) const
    {
        return WIDE ? at + (int)threadIdx.x * 8 + k : at + (int)threadIdx.x + k * NT;
    }
    template <bool FULL>
    __device__ __forceinline__ void load(const float *row, int at, float (&v)[8], float fill) const
    {
        if (WIDE && (FULL || place(at, 8) <= hi)) {
            const float4 x = __ldg(reinterpret_cast<const float4 *>(row + place(at, 0)));
            const float4 y = __ldg(reinterpret_cast<const float4 *>(row + place(at, 4)));
            v[0] = x.x;
            v[1] = x.y;
            v[2] = x.z;
            v[3] = x.w;
            v[4] = y.x;
            v[5] = y.y;
            v[6] = y.z;
            v[7] = y.w;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = FULL || place(at, k) < hi ? __ldg(row + place(at, k)) : fill;
        }
    }
    template <bool FULL>
    __device__ __forceinline__ void logits(long long row, int at, float (&v)[8]) const
    {
        if (F32) {
            load<FULL>(static_cast<const float *>(a.logits) + row * a.stride, at, v, -INFINITY);
        } else {
            const uint16_t *p = static_cast<const uint16_t *>(a.logits) + row * a.stride;
            if (WIDE && (FULL || place(at, 8) <= hi)) {
                const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p + place(at, 0)));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = k & 1 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    v[k] = FULL || place(at, k) < hi ? bf16_to_f32(__ldg(p + place(at, k))) : -INFINITY;
            }
        }
    }
    __device__ __forceinline__ float logit(long long row, int i) const
    {
        const long long at = row * a.stride + i;
        return F32 ? static_cast<const float *>(a.logits)[at] : bf16_to_f32(static_cast<const uint16_t *>(a.logits)[at]);
    }
    static __device__ __forceinline__ float clean(float l) { return l < INFINITY ? l : -INFINITY; }

    // takes G groups of eight of a row from chunk position `at` into a thread's
    // largest logit `best` and the sum of the weights against it (greedy: where it is)
    template <int G>
    __device__ __forceinline__ void take(float (&l)[G][8], int at, float c, bool greedy, float &best, float &sum, int &where) const;
};

// log2(e) / T, held inside the range where (l - top) c is 0 for l = top and -inf for l = -inf at any T
__device__ __forceinline__ float verify_scale(const VerifyArgs &a, int b, bool &greedy)
{
    const float temp = a.temperature ? a.temperature[b] : 1.0f;
    greedy = !(temp > 0.0f) || !a.noise;
    return greedy ? 1.0f : fminf(fmaxf(1.4426950408889634f / temp, 1e-37f), 1e37f);
}

// e^((l - top) / T) for a logit l and the reference top >= l (-inf where all are)
__device__ __forceinline__ float verify_weight(float l, float top, float c)
{
    return ex2((l - fmaxf(top, -3.402823466e38f)) * c);
}

template <bool F32, bool WIDE, int NT>
template <int G>
__device__ __forceinline__ void VerifyView<F32, WIDE, NT>::take(float (&l)[G][8], int at, float c, bool greedy, float &best,
                                                                float &sum, int &where) const
{
    float up = -INFINITY;
#pragma unroll
    for (int x = 0; x < G; ++x)
#pragma unroll
        for (int k = 0; k < 8; ++k)
            up = max_nan(up, l[x][k]);
    if (!(up < INFINITY)) {  // NaN and +inf count as -inf
        atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_NONFINITE);
        up = -INFINITY;
#pragma unroll
        for (int x = 0; x < G; ++x)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                l[x][k] = clean(l[x][k]);
                up = fmaxf(up, l[x][k]);
            }
    }
    if (greedy) {
        if (up > best)  // ascending indexes: the first of equals
#pragma unroll
            for (int x = 0; x < G; ++x)
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (l[x][k] > best) {
                        best = l[x][k];
                        where = place(at + x * STEP, k);
                    }
        return;
    }
    up = fmaxf(up, best);
    const float ref = -fmaxf(up, -3.402823466e38f);
    const F2 r2(ref, ref), c2(c, c);
    F2 s2(sum * verify_weight(best, up, c), 0.0f);
    best = up;
#pragma unroll
    for (int x = 0; x < G; ++x)
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            float e0, e1;
            mul2(add2(F2(l[x][k], l[x][k + 1]), r2), c2).get(e0, e1);
            s2 = add2(s2, F2(ex2(e0), ex2(e1)));
        }
    float s0, s1;
    s2.get(s0, s1);
    sum = s0 + s1;
}

// a warp's slices as one: ROW: sums are weights against the best of their lane
__device__ __forceinline__ VerifySlice warp_slice(VerifySlice v, bool row, float c)
{
    VerifySlice w = v;
    warp_larger(w.best, w.at);
    w.sum = warp_sum(row ? v.sum * verify_weight(v.best, w.best, c) : v.sum);
    return w;
}

// All rows ahead: CTA (row, part). Bound by the reads (384 rows of 131072 in
// bf16 are 101 MB: about 20 of the 38 us of such a call).
template <bool F32, bool WIDE>
__global__ void __launch_bounds__(MOE_VERIFY_STAT_THREADS) moe_verify_rows_kernel(const VerifyArgs a)
{
    constexpr int NT = MOE_VERIFY_STAT_THREADS, NW = NT / 32;
    __shared__ VerifySlice warps[NW];
    __shared__ int seq;
    pdl_wait();
    pdl_launch_dependents();
    const int row = blockIdx.x / a.splits, part = blockIdx.x % a.splits;
    const int lo = min(part * a.split, a.vocab), hi = min(lo + a.split, a.vocab);
    using View = VerifyView<F32, WIDE, NT>;
    const View view{a, hi};
    constexpr int G = F32 ? 2 : 4;  // groups of eight loaded at once
    float l[G][8];
    auto load = [&](int at) {
        if (at + G * View::STEP <= hi)
#pragma unroll
            for (int x = 0; x < G; ++x)
                view.template logits<true>(row, at + x * View::STEP, l[x]);
        else
#pragma unroll
            for (int x = 0; x < G; ++x)
                view.template logits<false>(row, at + x * View::STEP, l[x]);
    };
    load(lo);  // while the row's sequence is found
    if (threadIdx.x == 0)
        seq = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < a.batch; b += NT)
        if (a.q_start[b] <= row && row < a.q_start[b + 1])
            seq = b;
    __syncthreads();
    if (seq < 0)
        return;
    bool greedy;
    const float c = verify_scale(a, seq, greedy);
    VerifySlice mine{-INFINITY, 0.0f, a.vocab};
    for (int at = lo; at < hi; at += G * View::STEP) {
        if (at > lo)
            load(at);
        view.take(l, at, c, greedy, mine.best, mine.sum, mine.at);
    }
    const VerifySlice v = warp_slice(mine, !greedy, c);
    if ((threadIdx.x & 31) == 0)
        warps[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        VerifySlice w = warps[threadIdx.x % NW];  // the upper lanes repeat the lower ones'
        if (threadIdx.x >= NW)
            w.sum = 0.0f;
        w = warp_slice(w, !greedy, c);
        if (threadIdx.x == 0)
            a.stats[(size_t)row * a.splits + part] = w;
    }
}

template <bool F32, bool WIDE, bool AHEAD>
__global__ void __launch_bounds__(MOE_VERIFY_THREADS, 3) moe_verify_kernel(const VerifyArgs a)
{
    constexpr int NT = MOE_VERIFY_THREADS, NW = NT / 32;
    __shared__ VerifySlice slices[2][MOE_VERIFY_MAX_CLUSTER];
    __shared__ VerifySlice warps[NW];
    __shared__ VerifySlice rows[AHEAD ? MOE_MAX_DRAFT : 1];
    __shared__ int token[MOE_MAX_DRAFT], parent[MOE_MAX_DRAFT], path[MOE_MAX_DRAFT], rejected[MOE_MAX_DRAFT];
    __shared__ float zeds[MOE_MAX_DRAFT];  // Z (times the row's sum) before each rejection
    __shared__ float uniform[MOE_MAX_DRAFT], draft_x[MOE_MAX_DRAFT], logit_x[MOE_MAX_DRAFT];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cluster_rank(), ranks = cluster_size();
    const int b = blockIdx.x / ranks;
    // Before anything is read or written, the refusal below included: what earlier kernels wrote is promised to be
    // seen only behind it, and a call of refused sequences alone would end beside its rows kernel without it. (With the
    // tokens and drafts read ahead of it, a chain of 3 drafts over 32000 took 6.6 us, now 7.2, 48 chains over 131072
    // 36.3 us, now 38.2.)
    pdl_wait();
    const int first = a.q_start[b], n = a.q_start[b + 1] - first;
    if (first < 0 || n < 1 || n > MOE_MAX_DRAFT || first > a.rows - n) {  // the whole cluster
        if (rank == 0 && tid == 0) {
            if (n != 0)
                atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_INDEX);
            a.n_accepted[b] = 0;
            a.next[b] = -1;
        }
        return;
    }
    cluster_started_arrive();
    bool greedy;
    const float c = verify_scale(a, b, greedy);
    const int lo = min((int)rank * a.slice, a.vocab), hi = min(lo + a.slice, a.vocab);
    const float *noise = a.noise ? a.noise + b * a.noise_stride : nullptr;

    using View = VerifyView<F32, WIDE, NT>;
    const View view{a, hi};
    auto weight = [&](float l, float top) { return verify_weight(l, top, c); };
    // by the last warps, while the first ones bring the rows' results
    if (const int i = tid - (NT - MOE_MAX_DRAFT); i >= 0 && i < n) {
        const int x = a.tokens[first + i], up = a.parents ? a.parents[first + i] : i - 1;
        const bool in = x >= 0 && x < a.vocab;
        if (i > 0 && !in && rank == 0)
            atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_INDEX);
        token[i] = x;
        parent[i] = i > 0 && in && up < i ? up : -1;  // -1: never a candidate
        uniform[i] = a.uniforms && !greedy ? a.uniforms[first + i] : 0.5f;
        if (i > 0 && in && up >= 0 && up < i) {
            draft_x[i] = a.draft ? a.draft[(first + i) * a.draft_stride + x] : 1.0f;
            logit_x[i] = View::clean(view.logit(first + up, x));
        }
    }

    // A CTA's shared memory may be written once the CTA has started: a barrier of the whole cluster before the first
    // exchange (one that returned above did so with its whole cluster, and takes no part).
    cluster_started_wait();
    // All slices' results to all CTAs of the cluster: one barrier, buffers in turn. A buffer is written again two
    // exchanges later, behind the barrier between, at which every CTA arrives after its last read of it.
    int turn = 0;
    auto exchange = [&](VerifySlice v, bool row) -> const VerifySlice * {
        v = warp_slice(v, row, c);
        if (lane == 0)
            warps[warp] = v;
        __syncthreads();
        if (warp == 0) {
            v = warps[lane % NW];  // the upper lanes repeat the lower ones'
            if (lane >= NW)
                v.sum = 0.0f;
            v = warp_slice(v, row, c);
            if (lane < (int)ranks) {
                const VerifySlice *to = &slices[turn][rank];
                st_cluster(&to->best, lane, __float_as_uint(v.best));
                st_cluster(&to->sum, lane, __float_as_uint(v.sum));
                st_cluster(&to->at, lane, (uint32_t)v.at);
            }
        }
        cluster_sync();
        const VerifySlice *got = slices[turn];
        turn ^= 1;
        return got;
    };
    // the rows' results ahead, a warp a row
    if constexpr (AHEAD) {
        for (int r = warp; r < n; r += NW) {
            VerifySlice v{-INFINITY, 0.0f, a.vocab};
            for (int k = lane; k < a.splits; k += 32) {
                const VerifySlice w = a.stats[(size_t)(first + r) * a.splits + k];
                const float up = fmaxf(v.best, w.best);
                v.sum = v.sum * weight(v.best, up) + w.sum * weight(w.best, up);
                keep_larger(v.best, v.at, w.best, w.at);
            }
            v = warp_slice(v, !greedy, c);
            if (lane == 0)
                rows[r] = v;
        }
        __syncthreads();
    }

    int cur = 0, count = 0, nrej = 0, next = -1;
    float top = 0.0f, total = 0.0f, zed = 0.0f;  // zed: Z times the row's sum
    int top_at = 0, best_at = -1;

    // the weight of index i less the rejected drafts, of row cur
    auto less = [&](float w, int i) {
        for (int k = 0; k < nrej; ++k) {
            const int j = rejected[k];
            if (a.draft)
                w = fmaxf(fmaf(-zeds[k], __ldg(a.draft + (first + j) * a.draft_stride + i), w), 0.0f);
            else if (token[j] == i)
                w = 0.0f;
        }
        return w;
    };
    // the sum of the residual of row cur and the race over it
    auto race = [&]() {  // one call: this is the kernel's bulk
        float best = -1.0f, sum = 0.0f;
        int where = a.vocab;
        auto step = [&](auto full, int at) {
            constexpr bool FULL = decltype(full)::value != 0;
            float l[8], e[8];
            view.template logits<FULL>(first + cur, at, l);
            view.template load<FULL>(noise, at, e, 1.0f);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                l[k] = weight(View::clean(l[k]), top);  // past the slice: of -inf, 0
            for (int x = 0; x < nrej; ++x) {
                const int j = rejected[x];
                if (a.draft) {
                    const float z = zeds[x];
                    float q[8];
                    view.template load<FULL>(a.draft + (first + j) * a.draft_stride, at, q, 0.0f);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        l[k] = fmaxf(fmaf(-z, q[k], l[k]), 0.0f);
                } else {
                    const int i = token[j];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        l[k] = view.place(at, k) == i ? 0.0f : l[k];
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum += l[k];
                const float s = l[k] * rcp(fmaxf(e[k], 1.17549435e-38f));
                if (s > best && (FULL || view.place(at, k) < hi)) {  // ascending indexes: the first of equals
                    best = s;
                    where = view.place(at, k);
                }
            }
        };
        int at = lo;
        for (; at + View::STEP <= hi; at += View::STEP)
            step(IntC<1>{}, at);
        if (at < hi)
            step(IntC<0>{}, at);
        const VerifySlice *got = exchange({best, sum, where}, false);
        float s = 0.0f, v = -1.0f;
        best_at = a.vocab;
        for (uint32_t r = 0; r < ranks; ++r) {
            s += got[r].sum;
            keep_larger(v, best_at, got[r].best, got[r].at);
        }
        return s;
    };

    // walk to the next pass over the slices that a decision (or the end) needs
    enum { NONE, SUM, LAST_RESIDUAL, LAST_ROW };
    bool fresh = true;
    for (int j = 1;;) {
        if (fresh) {  // row cur
            if constexpr (AHEAD) {
                top = rows[cur].best;
                top_at = rows[cur].at;
                total = rows[cur].sum;
            } else {
                VerifySlice mine{-INFINITY, 0.0f, a.vocab};
                constexpr int G = F32 ? 1 : 2;
                float l[G][8];
                int at = lo;
                for (; at + G * View::STEP <= hi; at += G * View::STEP) {
#pragma unroll
                    for (int x = 0; x < G; ++x)
                        view.template logits<true>(first + cur, at + x * View::STEP, l[x]);
                    view.take(l, at, c, greedy, mine.best, mine.sum, mine.at);
                }
                for (; at < hi; at += G * View::STEP) {
#pragma unroll
                    for (int x = 0; x < G; ++x)
                        view.template logits<false>(first + cur, at + x * View::STEP, l[x]);
                    view.take(l, at, c, greedy, mine.best, mine.sum, mine.at);
                }
                const VerifySlice *got = exchange(mine, !greedy);
                top = -INFINITY;
                top_at = a.vocab;
                for (uint32_t r = 0; r < ranks; ++r)
                    keep_larger(top, top_at, got[r].best, got[r].at);
                total = 0.0f;
                for (uint32_t r = 0; r < ranks; ++r)
                    total += got[r].sum * weight(got[r].best, top);
            }
            if (greedy)
                total = top > -INFINITY ? 1.0f : 0.0f;
            zed = total;
            nrej = 0;
            best_at = -1;
            fresh = false;
        }
        int pass = NONE;
        while (j < n && total > 0.0f && !fresh && pass == NONE) {
            const int at = j++;
            if (parent[at] != cur)
                continue;
            const int x = token[at];
            const float r = greedy ? (x == top_at ? zed : 0.0f) : less(weight(logit_x[at], top), x);
            if (uniform[at] * zed * draft_x[at] < r) {
                cur = at;
                fresh = true;
                if (tid == 0)
                    path[count] = at;
                ++count;
            } else if (greedy) {  // the residual stays on the row's largest logit, unless the draft was certain of it
                if (a.draft && a.draft[(first + at) * a.draft_stride + top_at] >= 1.0f)
                    zed = 0.0f;
            } else {
                __syncthreads();
                if (tid == 0) {
                    rejected[nrej] = at;
                    zeds[nrej] = zed;
                }
                ++nrej;
                __syncthreads();
                // a chosen token takes its own weight out of the sum; where that leaves little, and for a drawn one, a pass
                if (!a.draft)
                    zed = fmaxf(zed - r, 0.0f);
                if (a.draft || zed < total * 0.015625f)
                    pass = SUM;
            }
        }
        if (fresh)
            continue;
        if (pass == NONE) {  // the walk has ended
            if (greedy || !(total > 0.0f)) {
                next = total > 0.0f ? top_at : -1;
                break;
            }
            if (nrej > 0 && zed > 0.0f) {
                if (a.draft) {  // the last rejection's pass was over this residual
                    next = best_at;
                    break;
                }
                pass = LAST_RESIDUAL;
            } else {
                nrej = 0;
                pass = LAST_ROW;
            }
        }
        zed = race();
        if (pass == LAST_ROW || (pass == LAST_RESIDUAL && zed > 0.0f)) {
            next = best_at;
            break;
        }
    }
    if (rank == 0) {
        __syncthreads();
        if (tid < n)
            a.path[first + tid] = tid < count ? path[tid] : -1;
        if (tid == 0) {
            a.n_accepted[b] = count;
            a.next[b] = next;
        }
    }
}

}  // namespace moe

// moe_tree_tc.cuh -- tree attention for more than 16 query rows a kv head, on
// the 5th-generation tensor cores: the same sums, list of work and partials
// as moe_tree_attn.cuh, in tiles of 128 tokens.
//
// Tokens are the M side, so that any number of rows costs what it is:
//   S^T [128 tokens x N rows] = K [tokens x 128] Q^T,
//   O^T [128 dims x N rows] += V^T [dims x tokens] P^T [tokens x rows],
// both accumulators in tensor memory, a token (a dimension) a lane. V lies in
// shared memory as K does, 128-byte rows of 64 dimensions a token in the
// 128-byte swizzle: read with M contiguous it is V^T; P^T likewise, a token's
// row of 64 weights, read with N contiguous. The maximum of a row runs across
// lanes, so the weights are taken against a reference that only moves when a
// score passes it by 2^8 (one vote a tile; the exact maxima are then found,
// and o and the sums scaled).
//
// One CTA an SM: a warp copies the cache's blocks, four turn codes into f16
// tiles, eight (two column halves of the four lane quarters) do the softmax,
// one thread issues the products. K of tile t + 1 is made while the softmax
// of tile t runs. What bounds it: shared memory, which a tile's codes and f16
// values cross five times (128 tokens of Q8: 35 KB in, out, 64 KB in, out,
// and Q, P in proportion to N), about 1800 cycles a tile for any N <= 64.
#pragma once
#include "moe_tc.cuh"
#include "moe_tree_attn.cuh"

namespace moe {

#define MOE_TTC_TOKENS 128
#define MOE_TTC_SOFT 8   // softmax warps
#define MOE_TTC_CODE 4   // warps that turn codes into f16
// the offset of a row without a reference: every finite score then asks for one
#define MOE_TTC_NONE 3.0e38f
#define MOE_TTC_THREADS ((MOE_TTC_SOFT + MOE_TTC_CODE + 2) * 32)

template <int FMT, int N>
struct TtcShape {
    static constexpr int D = 128;
    static constexpr int RB = FMT == MOE_KV_Q8 ? D : D / 2;
    static constexpr int GR = D / MOE_KV_GROUP;
    static constexpr int HALF = 16 * RB + 16 * GR * (FMT == MOE_KV_Q8 ? 2 : 4);
    static constexpr int BLOCK = 2 * HALF;
    static constexpr int STAGE = 8 * BLOCK;                // a tile's blocks
    static constexpr int PANEL = MOE_TTC_TOKENS * 128;     // 64 columns of 128 tokens
    static constexpr int PP = (N + 63) / 64;               // panels of P
    static constexpr int K_AT = 0, V_AT = 2 * PANEL, P_AT = 4 * PANEL, Q_AT = P_AT + PP * PANEL;
    static constexpr int RAW_AT = Q_AT + 2 * N * 128;
    static constexpr int COLS = N <= 32 ? 128 : N <= 64 ? 256 : 512;  // of tensor memory: S, S, O
    static constexpr int CPT = N / 2;                      // columns of a softmax thread
    // small arrays, after the raw stages: barriers, (multiplier, offset), factors, per-quarter maxima and sums,
    // masks, places of the output rows, stage flags, the scan and the list
    static constexpr int BARS = 256;
    static constexpr int SMALL = BARS + N * (8 + 4 + 4 * 4 + 4 * 4 + 4 + 8 + 8) + 128;
    static constexpr int PART = N * D + 2 * N;             // floats of a partial: [row][dim], references, sums
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i)
        v[i] = __uint_as_float(r[i]);
}

// descriptor of a tile whose M (N) side is contiguous: 128-byte rows of 64
// elements, one row a k, in the 128-byte swizzle; 8 rows are 1024 bytes apart
// (stride offset), the next 64 elements PANEL bytes (leading offset)
__device__ __forceinline__ uint64_t mn_desc(const void *tile)
{
    const uint64_t addr = smem_u32(tile);
    return ((addr >> 4) & 0x3FFFull) | ((uint64_t)(MOE_TTC_TOKENS * 128 / 16) << 16) | ((1024ull >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// the softmax warps' own barrier
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(MOE_TTC_SOFT * 32) : "memory"); }
__device__ __forceinline__ bool soft_any(bool p)
{
    uint32_t r;
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n"
                 " selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)p), "n"(MOE_TTC_SOFT * 32)
                 : "memory");
    return r != 0;
}

__device__ __forceinline__ float warp_max(float v)  // no NaN
{
    const uint32_t u = __float_as_uint(v), key = u & 0x80000000u ? ~u : u | 0x80000000u;
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, key);
    return __uint_as_float(top & 0x80000000u ? top & 0x7FFFFFFFu : ~top);
}

// 16 codes (four words) of a 16-byte piece of Q8 as f16 pairs
__device__ __forceinline__ void q8_sixteen(const uint4 &w, __half2 d, uint32_t (&h)[8])
{
    h[0] = q8_pair(w.x, 0x5140, d);
    h[1] = q8_pair(w.x, 0x5342, d);
    h[2] = q8_pair(w.y, 0x5140, d);
    h[3] = q8_pair(w.y, 0x5342, d);
    h[4] = q8_pair(w.z, 0x5140, d);
    h[5] = q8_pair(w.z, 0x5342, d);
    h[6] = q8_pair(w.w, 0x5140, d);
    h[7] = q8_pair(w.w, 0x5342, d);
}

// 16 codes (two words) of Q4
__device__ __forceinline__ void q4_sixteen(uint32_t w0, uint32_t w1, __half2 d, __half2 m, uint32_t (&h)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = q4_pair((w0 >> (4 * i) & 0x000F000Fu) | 0x64006400u, d, m);
        h[4 + i] = q4_pair((w1 >> (4 * i) & 0x000F000Fu) | 0x64006400u, d, m);
    }
}

// 16 consecutive dimensions (from 16 x) of a token's row of an f16 tile: two
// 16-byte pieces, the `second` one first in half of the lanes (bank conflicts)
__device__ __forceinline__ void put_sixteen(uint8_t *tile, int token, int x, const uint32_t (&h)[8], bool swap)
{
    uint8_t *row = tile + (x >> 2) * (MOE_TTC_TOKENS * 128) + token * 128;
    const int c = (x & 3) * 2;
    const uint4 lo = make_uint4(h[0], h[1], h[2], h[3]), hi = make_uint4(h[4], h[5], h[6], h[7]);
    *reinterpret_cast<uint4 *>(row + (((c + (swap ? 1 : 0)) ^ (token & 7)) << 4)) = swap ? hi : lo;
    *reinterpret_cast<uint4 *>(row + (((c + (swap ? 0 : 1)) ^ (token & 7)) << 4)) = swap ? lo : hi;
}

template <int FMT, int N>
__global__ void __launch_bounds__(MOE_TTC_THREADS, 1) moe_tree_tc_kernel(const __grid_constant__ TreeArgs a, const int stages)
{
    using T = TtcShape<FMT, N>;
    constexpr int D = T::D, CPT = T::CPT;
    extern __shared__ __align__(1024) uint8_t smem_any[];
    uint8_t *smem = smem_any + (-smem_u32(smem_any) & 1023u);  // the swizzle goes by address bits
    uint8_t *sk = smem + T::K_AT, *sv = smem + T::V_AT, *sp = smem + T::P_AT, *sq = smem + T::Q_AT;
    uint8_t *raw = smem + T::RAW_AT, *small = raw + (size_t)stages * T::STAGE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(small);
    uint64_t *raw_full = bars, *raw_free = bars + 4, *k_full = bars + 8, *v_full = bars + 9, *p_full = bars + 10,
             *q_full = bars + 11, *pv_done = bars + 12, *s_full = bars + 13;  // s_full[2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 16);
    uint32_t *gone = tmem_slot + 1;  // [8] blocks of tile t that are not there, at t % 8: kept longer than its stage
    int *last = reinterpret_cast<int *>(gone + 8);
    float2 *mul = reinterpret_cast<float2 *>(small + T::BARS);                // [N] (c, 7 - m)
    float *ref = reinterpret_cast<float *>(mul + N);                          // [N] m
    float *qmax = ref + N, *qsum = qmax + 4 * N;                              // [4][N]
    float *factor = qsum + 4 * N;                                             // [N]
    unsigned long long *masks = reinterpret_cast<unsigned long long *>(factor + N);  // [N]
    long long *rowat = reinterpret_cast<long long *>(masks + N);              // [N]
    long long *scan = rowat + N, *cum = scan + 16;                            // [batch + 1]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t *status = a.ctrl + MOE_CTRL_STATUS;

    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(raw_full + s, 1);
            mbar_init(raw_free + s, MOE_TTC_CODE);
        }
        mbar_init(k_full, MOE_TTC_CODE);
        mbar_init(v_full, MOE_TTC_CODE);
        mbar_init(p_full, MOE_TTC_SOFT);
        mbar_init(q_full, MOE_TTC_SOFT);
        mbar_init(pv_done, 1);
        mbar_init(s_full, 1);
        mbar_init(s_full + 1, 1);
        fence_barrier_init();
    }
    if (warp == 0)
        tmem_alloc(tmem_slot, T::COLS);
    // the list: tiles before each sequence
    {
        constexpr int NT = MOE_TTC_THREADS;
        const int per = (a.batch + NT - 1) / NT;
        long long mine = 0;
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b >= a.batch)
                break;
            int first, n, len, rows;
            tree_sequence(a, b, first, n, len, rows);
            cum[b] = mine;
            mine += (long long)((len + MOE_TTC_TOKENS - 1) / MOE_TTC_TOKENS) *
                    (n > 0 ? tree_blocks<N>(n, a.group) * a.k.heads : 0);
            if (n == 0 && rows > 0 && blockIdx.x == (unsigned)(b % gridDim.x))
                tree_zero<D>(a, first, rows);
        }
        long long incl = mine;
        for (int m = 1; m < 32; m *= 2) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, m);
            if (lane >= m)
                incl += v;
        }
        if (lane == 31)
            scan[warp] = incl;
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        long long before = incl - mine;
        for (int w = 0; w < warp; ++w)
            before += scan[w];
        for (int i = 0; i < per; ++i)
            if (tid * per + i < a.batch)
                cum[tid * per + i] += before;
        if (tid == NT - 1)
            cum[a.batch] = before + mine;
        __syncthreads();
    }
    const uint32_t tmem = *tmem_slot;
    const long long total = cum[a.batch];
    const long long run = max((total + gridDim.x - 1) / (long long)gridDim.x, (long long)a.min_units);
    const long long lo = min(run * blockIdx.x, total), hi = min(lo + run, total);
    const int tiles = (int)(hi - lo);
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_wait(bar, parity, status, a.wait_ns); };
    auto item_at = [&](long long u) { return tree_item<N, MOE_TTC_TOKENS>(a, cum, u); };

    if (warp == MOE_TTC_SOFT + MOE_TTC_CODE) {
        // ---------------- the copies: lane i the i-th block of a tile
        const uint64_t policy = policy_evict_first();
        bool ok = true;
        int t = 0;
        for (; t < tiles && ok; ++t) {
            const TreeItem it = item_at(lo + t);
            const int blk = (int)(lo + t - it.lo) * 8 + lane, per_page = a.k.page / 16;
            const bool there = lane < 8 && blk * 16 < it.len;
            const uint8_t *src = nullptr;
            if (there) {
                const int page = a.table[it.b * a.table_stride + blk / per_page];
                if (page < 0 || page >= a.n_pages)
                    atomicOr(status, (uint32_t)MOE_WS_INDEX);
                else
                    src = a.pages + (((size_t)page * a.k.heads + it.head) * per_page + blk % per_page) * T::BLOCK;
            }
            const uint32_t got = __ballot_sync(0xFFFFFFFFu, src != nullptr);
            const int s = t % stages;
            if (t >= stages)
                ok = __all_sync(0xFFFFFFFFu, wait(raw_free + s, (uint32_t)(t / stages - 1) & 1u));
            if (!ok)
                break;
            if (lane == 0) {
                gone[t & 7] = ~got & 0xFFu;
                mbar_arrive_expect_tx(raw_full + s, __popc(got) * T::BLOCK);
            }
            __syncwarp();
            if (src)
                bulk_g2s(raw + (size_t)s * T::STAGE + lane * T::BLOCK, src, T::BLOCK, raw_full + s, policy);
        }
        for (int k = max(0, t - stages); k < t; ++k)  // nothing in flight when the memory is given back
            wait(raw_full + k % stages, (uint32_t)(k / stages) & 1u);
    } else if (warp == MOE_TTC_SOFT + MOE_TTC_CODE + 1) {
        // ---------------- the products
        if (lane == 0) {
            constexpr uint32_t id_s = mma_idesc(128, N, false), id_o = id_s | (1u << 15) | (1u << 16);
            bool ok = true, open = false;  // open: tile t - 1's second product is still to come
            uint32_t items = 0;
            bool fresh = false;  // that tile is its item's first
            long long end = lo;
            auto second = [&](int t) {
                ok = ok && wait(v_full, (uint32_t)t & 1u) && wait(p_full, (uint32_t)t & 1u);
                if (!ok)
                    return;
                tc_fence_after();
                const uint64_t ad = mn_desc(sv), bd = mn_desc(sp);
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 16 tokens: 2048 bytes
                    mma_f16(tmem + 2 * N, ad + k * 128, bd + k * 128, id_o, !fresh || k > 0);
                mma_commit(pv_done);
            };
            for (int t = 0; t < tiles && ok; ++t) {
                const bool starts = lo + t == end;
                if (starts) {  // the softmax warps finish the last item before they bring the next one's queries
                    if (open)
                        second(t - 1);
                    open = false;
                    const TreeItem it = item_at(lo + t);
                    end = min(hi, it.lo + it.units);
                    ok = ok && wait(q_full, items & 1u);
                    ++items;
                }
                ok = ok && wait(k_full, (uint32_t)t & 1u);
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t ad = sw128_desc(sk), bd = sw128_desc(sq);
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 16 dimensions: 32 bytes, then the next panel
                    mma_f16(tmem + (t & 1) * N, ad + (k / 4) * (T::PANEL / 16) + (k % 4) * 2,
                            bd + (k / 4) * (N * 128 / 16) + (k % 4) * 2, id_s, k > 0);
                mma_commit(s_full + (t & 1));
                if (open)
                    second(t - 1);
                open = true;
                fresh = starts;
            }
            if (open && ok)
                second(tiles - 1);
            if (tiles > 0 && ok)
                wait(pv_done, (uint32_t)(tiles - 1) & 1u);
        }
    } else if (warp >= MOE_TTC_SOFT) {
        // ---------------- codes to f16: warp w the blocks w, w + 4 of a tile
        const int w = warp - MOE_TTC_SOFT, g = lane >> 2, t4 = lane & 3;
        bool ok = true;
        for (int t = 0; t < tiles; ++t) {
            const TreeItem it = item_at(lo + t);
            const int s = t % stages, left = it.len - (int)(lo + t - it.lo) * MOE_TTC_TOKENS;  // tokens from the tile on
            ok = ok && wait(raw_full + s, (uint32_t)(t / stages) & 1u);
            if (t > 0)  // K has been read
                ok = ok && wait(s_full + ((t - 1) & 1), (uint32_t)((t - 1) >> 1) & 1u);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
            const uint32_t out = *reinterpret_cast<volatile uint32_t *>(gone + (t & 7));
            const uint8_t *stage = raw + (size_t)s * T::STAGE;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int blk = w + 4 * x;
                const uint8_t *b = stage + blk * T::BLOCK;
#pragma unroll
                for (int nb = 0; nb < 2; ++nb) {
                    const int tok = nb * 8 + g, at = blk * 16 + tok;
                    uint32_t h[8];
                    if (FMT == MOE_KV_Q8) {
                        const __half2 d = __half2half2(reinterpret_cast<const __half *>(b + 16 * T::RB)[tok * 4 + t4]);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = i ^ (g & 1);
                            const uint4 v = *reinterpret_cast<const uint4 *>(b + (nb * 2 + c) * 512 + lane * 16);
                            q8_sixteen(v, d, h);
                            put_sixteen(sk, at, t4 * 2 + c, h, t4 >= 2);
                        }
                    } else {
                        const uint32_t dm = reinterpret_cast<const uint32_t *>(b + 16 * T::RB)[tok * 4 + t4];
                        const __half2 d = h2(dup_lo(dm)), m = h2(dup_hi(dm));
                        const uint4 v = *reinterpret_cast<const uint4 *>(b + nb * 512 + lane * 16);
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = i ^ (g & 1);
                            q4_sixteen(c ? v.z : v.x, c ? v.w : v.y, d, m, h);
                            put_sixteen(sk, at, t4 * 2 + c, h, t4 >= 2);
                        }
                    }
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(k_full);
            if (t > 0)  // V has been read
                ok = wait(pv_done, (uint32_t)(t - 1) & 1u);
            if (!__all_sync(0xFFFFFFFFu, ok))
                break;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int blk = w + 4 * x;
                const uint8_t *b = stage + blk * T::BLOCK + T::HALF;
                const __half *sc = reinterpret_cast<const __half *>(b + 16 * T::RB);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tok = (r >> 1) * 8 + t4 * 2 + (r & 1), at = blk * 16 + tok;
                    const bool in = at < left && !(out >> blk & 1);  // else the bytes are anything: 0
                    const __half2 d = __half2half2(in ? sc[(g >> 1) * 16 + tok] : __ushort_as_half(0));
                    uint32_t h[8];
                    if (FMT == MOE_KV_Q8) {
                        q8_sixteen(*reinterpret_cast<const uint4 *>(b + r * 512 + lane * 16), d, h);
                    } else {
                        const __half2 m = __half2half2(in ? sc[(T::GR + (g >> 1)) * 16 + tok] : __ushort_as_half(0));
                        const uint2 v = *reinterpret_cast<const uint2 *>(b + (r >> 1) * 512 + lane * 16 + (r & 1) * 8);
                        q4_sixteen(v.x, v.y, d, m, h);
                    }
                    put_sixteen(sv, at, g, h, g & 1);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(v_full);
                mbar_arrive(raw_free + s);
            }
        }
    } else {
        // ---------------- softmax: quarter q's lanes (tokens; dimensions of O), columns from c0
        const int quarter = warp & 3, half = warp >> 2, c0 = half * CPT, row = quarter * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        bool ok = true;
        int t = 0;
        while (t < tiles && ok) {
            const long long u = lo + t;
            const TreeItem it = item_at(u);
            const long long end = min(hi, it.lo + it.units);
            // ---- the item's queries: a row a pair of threads (64 dimensions each)
            for (int r = tid >> 1; r < N; r += MOE_TTC_SOFT * 16) {
                const int rr = it.block * N + r;
                const bool live = rr < it.n * a.group;
                const int i = live ? rr / a.group : 0, h = it.head * a.group + (live ? rr % a.group : 0);
                uint32_t x[32];
                const float c = tree_row<64, 2>(a, live, it.first + i, h, (tid & 1) * 64, x);
                if ((tid & 1) == 0) {
                    mul[r] = make_float2(c, MOE_TTC_NONE);
                    ref[r] = -INFINITY;
                    masks[r] = !live ? 0 : a.mask ? a.mask[it.first + i] : (2ull << i) - 1;
                    rowat[r] = live ? (it.first + i) * a.o_tok + h * a.o_head : -1;
                }
                uint8_t *p = sq + (tid & 1) * (N * 128) + r * 128;
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4 *>(p + ((c ^ (r & 7)) << 4)) =
                        make_uint4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
            }
            fence_proxy_async_smem();
            soft_sync();
            if (lane == 0)
                mbar_arrive(q_full);
            float sum[CPT];
#pragma unroll
            for (int i = 0; i < CPT; ++i)
                sum[i] = 0.0f;
            const int prefix = it.len - it.n, t0 = t;
            for (; lo + t < end; ++t) {
                ok = ok && wait(s_full + (t & 1), (uint32_t)(t >> 1) & 1u);
                if (soft_any(!ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int first = (int)(lo + t - it.lo) * MOE_TTC_TOKENS, j = first + row;  // this lane's token
                const uint32_t out = *reinterpret_cast<volatile uint32_t *>(gone + (t & 7));
                const bool masked = first + MOE_TTC_TOKENS > prefix || out;
                const bool in = j < it.len && !(out >> (row >> 4) & 1);
                auto scores = [&](int c, float (&s)[16]) {
                    tmem_ld16(lanes + (t & 1) * N + c0 + c, s);
                    if (masked)
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (!in || (j >= prefix && !(masks[c0 + c + i] >> (j - prefix) & 1)))
                                s[i] = -INFINITY;
                };
                // does a score pass its reference? (no reference yet: every finite one)
                bool up = t == t0;
                if (!up) {
#pragma unroll
                    for (int c = 0; c < CPT; c += 16) {
                        float s[16];
                        scores(c, s);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 m = mul[c0 + c + i];
                            up |= fmaf(s[i], m.x, m.y) > MOE_TREE_LIFT + MOE_TREE_SLACK;
                        }
                    }
                }
                if (soft_any(up)) {
#pragma unroll
                    for (int c = 0; c < CPT; c += 16) {
                        float s[16];
                        scores(c, s);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float v = warp_max(fmaxf(s[i], -INFINITY) * mul[c0 + c + i].x);
                            if (lane == 0)
                                qmax[quarter * N + c0 + c + i] = v;
                        }
                    }
                    soft_sync();
                    for (int r = tid; r < N; r += MOE_TTC_SOFT * 32) {
                        const float v = fmaxf(fmaxf(qmax[r], qmax[N + r]), fmaxf(qmax[2 * N + r], qmax[3 * N + r]));
                        const float m = ref[r], to = v > m + MOE_TREE_SLACK ? v : m;
                        factor[r] = to == m ? 1.0f : ex2(m - to);
                        ref[r] = to;
                        mul[r].y = to == -INFINITY ? MOE_TTC_NONE : MOE_TREE_LIFT - to;
                    }
                    soft_sync();
#pragma unroll
                    for (int i = 0; i < CPT; ++i)
                        sum[i] *= factor[c0 + i];
                    if (t > t0) {  // O, once the last tile's product is in
                        ok = ok && wait(pv_done, (uint32_t)(t - 1) & 1u);
                        __syncwarp();
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < CPT; c += 16) {
                            float o[16];
                            uint32_t w[16];
                            tmem_ld16(lanes + 2 * N + c0 + c, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = __float_as_uint(o[i] * factor[c0 + c + i]);
                            tmem_st16(lanes + 2 * N + c0 + c, w);
                        }
                        tmem_st_wait();
                    }
                }
                if (t > 0 && ok)  // P has been read
                    ok = wait(pv_done, (uint32_t)(t - 1) & 1u);
                __syncwarp();
#pragma unroll
                for (int c = 0; c < CPT; c += 16) {
                    float s[16];
                    scores(c, s);
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float4 m = *reinterpret_cast<const float4 *>(mul + c0 + c + i);
                        const float e0 = ex2(fmaf(s[i], m.x, m.y)), e1 = ex2(fmaf(s[i + 1], m.z, m.w));
                        sum[c + i] += e0;
                        sum[c + i + 1] += e1;
                        w[i / 2] = pack_h2(e0, e1);
                    }
                    const int col = c0 + c;
                    uint8_t *p = sp + (col >> 6) * T::PANEL + row * 128;
                    const int k = (col & 63) >> 3;
                    *reinterpret_cast<uint4 *>(p + ((k ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(p + (((k + 1) ^ (row & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full);
            }
            if (soft_any(!ok)) {
                ok = false;
                break;
            }
            // ---- the rows' sums over the lanes and quarters
#pragma unroll
            for (int i = 0; i < CPT; ++i) {
                const float v = warp_sum(sum[i]);
                if (lane == 0)
                    qsum[quarter * N + c0 + i] = v;
            }
            soft_sync();
            for (int r = tid; r < N; r += MOE_TTC_SOFT * 32)
                factor[r] = (qsum[r] + qsum[N + r]) + (qsum[2 * N + r] + qsum[3 * N + r]);
            ok = wait(pv_done, (uint32_t)(t - 1) & 1u);
            if (soft_any(!ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const long long item_end = it.lo + it.units;
            const bool whole = u == it.lo && end == item_end;
            float *part = a.part + ((size_t)blockIdx.x * 2 + (u == lo ? 0 : 1)) * T::PART;
#pragma unroll
            for (int c = 0; c < CPT; c += 16) {
                float o[16];
                tmem_ld16(lanes + 2 * N + c0 + c, o);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int r = c0 + c + i;
                    if (!whole)
                        part[r * D + row] = o[i];
                    else if (rowat[r] >= 0)
                        a.out[rowat[r] + row] = __bfloat16_as_ushort(
                            __float2bfloat16_rn(factor[r] == 0.0f ? 0.0f : o[i] / factor[r]));
                }
            }
            tc_fence_before();
            if (!whole) {
                for (int r = tid; r < N; r += MOE_TTC_SOFT * 32) {
                    part[N * D + r] = ref[r];
                    part[N * D + N + r] = factor[r];
                }
                __threadfence();
                soft_sync();
                const int p0 = (int)(it.lo / run), p1 = (int)((item_end - 1) / run);  // the item's runs
                if (tid == 0) {
                    const bool end_of_it = atom_add_acq_rel_gpu(a.count + p0, 1) == (unsigned)(p1 - p0);
                    if (end_of_it)
                        st_relaxed_gpu(a.count + p0, 0);
                    *last = end_of_it;
                }
                soft_sync();
                if (*reinterpret_cast<volatile int *>(last)) {  // join the parts in the order of the runs
                    __threadfence();
                    auto slot = [&](int cta) { return a.part + ((size_t)cta * 2 + (it.lo <= cta * run ? 0 : 1)) * T::PART; };
                    for (int r = c0; r < c0 + CPT; ++r) {
                        if (rowat[r] < 0)
                            continue;
                        float m = -INFINITY, l = 0.0f, o = 0.0f;
                        for (int cta = p0; cta <= p1; ++cta)
                            m = fmaxf(m, __ldcg(slot(cta) + N * D + r));
                        for (int cta = p0; cta <= p1; ++cta) {
                            const float *src = slot(cta);
                            const float v = __ldcg(src + N * D + r), f = v == -INFINITY ? 1.0f : ex2(v - m);
                            l = fmaf(__ldcg(src + N * D + N + r), f, l);
                            o = fmaf(__ldcg(src + r * D + row), f, o);
                        }
                        a.out[rowat[r] + row] = __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.0f ? 0.0f : o / l));
                    }
                }
            }
            soft_sync();  // factor, rowat and the queries' arrays are free
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        tmem_dealloc(tmem, T::COLS);
}

}  // namespace moe

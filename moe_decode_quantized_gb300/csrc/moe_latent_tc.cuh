// moe_latent_tc.cuh -- latent attention in absorbed form on the 5th-generation
// tensor cores: for the rows (query token, head) of a sequence
//   S = Q C^T + QR KR^T,   O += P C,   P = 2^(c (S - m)),
// over the sequence's shared rows [C | KR] of the paged cache, in one pass, with
// a running reference m and sum of weights for each row.
//
// O of 128 rows and 512 dimensions would fill a CTA's tensor memory, so a pair of
// CTAs (cta_group::2) shares a block of 128 rows: each has 64 of them, all tokens
// and all dimensions of the result in tensor memory, and half of what both
// multiply with. Tiles of 64 tokens: for S each CTA brings its 32 tokens' rows
// whole; for O it needs all 64 tokens but only its half of the dimensions, which
// it has of its own tokens already, and the other tokens' are brought, from the
// L2, to where its own tokens' other half has stood once S is there. A tile so
// takes no more shared memory than its rows, and every row comes from memory
// once. In a row of tensor memory (lane), lanes 0 to 63 are the pair's 64 rows
// with the first half of S's tokens (O's dimensions), lanes 64 to 127 the same
// rows with the second.
//
// Items, runs and partials are those of moe_tree_attn.cuh, a run a pair.
//
// Bound by products and by bytes nearly alike at 128 heads (242 FLOP a byte), by
// bytes below that, by two launches' latency for one short sequence. One token of
// 64 sequences over 4000 to 24000 tokens, latent vectors of 512: 128 heads 191 us
// (139 at the copy rate, 117 at the products'), 16 heads 177 (5.1 TB/s: the tiles take as long, rows or not); 16
// trees of 8 rows, 32 heads, over up to 16000: 77; one sequence of 511: 14.0. A
// tile of 128 rows takes some 1900 clocks, of which its products need 1160: there
// is one buffer of P, so that a tile's softmax stores only when the product before
// has read it, and that tile's product begins only then. The same chain bounds
// latent vectors of 256 and 128 (64 heads 121 us, 76 at the copy rate; 32 heads
// 112, 46), whatever their bytes. Of tensor memory's 512 columns O takes L / 2 and the two S
// 64. Tiles of 64 tokens leave room for four stages at 512, which is what the
// copies' latency needs; 8 softmax warps gained nothing over 4.
#pragma once
#include "moe_latent.cuh"
#include "moe_tc.cuh"
#include "moe_tree_attn.cuh"

namespace moe {

#define MOE_LTC_TOKENS 64
#define MOE_LTC_ROWS 128   // of a pair
#define MOE_LTC_COST 8     // of an item, beside its tiles (16 trees over 1000 to 16000 tokens: 80 us with 5, 78 with 8, 80 with 12;
                           // 200 sequences of 1 to 2000, 64 heads: 95, 90 and 92)
#define MOE_LTC_SOFT 4     // softmax warps
#define MOE_LTC_THREADS ((MOE_LTC_SOFT + 5) * 32)
#define MOE_LTC_MAX_STAGES 8
#define MOE_LTC_CHUNK 4096  // 64 dimensions of 32 tokens
#define MOE_LTC_SLACK 8.0f  // m moves when an exponent passes it by this

struct LatentArgs {
    TreeArgs t;  // k.heads 1, k.dim the latent vector's, group the heads; q the query's latent part
    const uint16_t *qr;
    long long qr_tok, qr_head;
    int rope, qr_wide;
    int big;  // boxes of 32 tokens and of all chunks; else of 16 tokens and one
    unsigned long long per_page;  // 2^36 / (page / 16), rounded up: x / (page / 16) = x per_page >> 36 below 2^27
    CUtensorMap keys, values, ropes;  // the cache's rows [64, slots, chunks]; the same; their turning part [rope, slots]
};

template <int L>
struct LtcShape {
    static constexpr int CHUNKS = L / 64;        // of the latent vector; one more is the turning part
    static constexpr int HALF = L / 128;         // chunks of the dimensions that a CTA's part of O has
    static constexpr int STAGE = (CHUNKS + 1) * MOE_LTC_CHUNK;
    static constexpr int Q_CHUNK = 8192;         // 64 dimensions of 64 rows
    static constexpr int P_AT = (CHUNKS + 1) * Q_CHUNK;
    static constexpr int P_BYTES = 8192;         // 64 tokens of 64 rows
    static constexpr int RING_AT = P_AT + P_BYTES;
    static constexpr int N = L < 256 ? L : 256;  // dimensions of one product
    static constexpr int O_COLS = L / 2;
    // barriers; maxima [2][2][64]; gone [16]; the scan, then the list
    static constexpr int SMALL = 384 + 4 * 64 * 4 + 64 + 32 * 8;
};

// ---- pairs of CTAs

__device__ __forceinline__ uint32_t cta_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void pair_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// an arrival at the barrier of the pair's first CTA (what it tells of is read by the tensor core alone, and has passed
// fence.proxy.async or has come by an asynchronous copy)
__device__ __forceinline__ void arrive_first(uint64_t *bar)
{
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
                 " mbarrier.arrive.shared::cluster.b64 _, [a];\n}\n" ::"r"(smem_u32(bar))
                 : "memory");
}

// the address of the barrier at `bar` in CTA `of` of the pair
__device__ __forceinline__ uint32_t pair_bar(uint64_t *bar, uint32_t of)
{
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(bar)), "r"(of));
    return at;
}

// tma_load_3d (2d) into this CTA, counted by a barrier of either of the pair
__device__ __forceinline__ void pair_load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void pair_load_2d(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

// D[tmem] (+)= A[smem] . B[smem]: M rows over the pair, each CTA's shared memory holding half of A's rows and half of
// B's columns at the same places. By a whole warp, one lane of which issues it: with the operands the same in every
// lane they are kept in uniform registers (36 products of 64 tokens and two commits: 970 clocks; by a lane that works
// alone, whose operands are moved there each time, 1680)
__device__ __forceinline__ void mma2_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xFFFFFFFF;\n"
        " @e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// the barrier in both CTAs completes (one arrival) once the products that this warp issued before have
__device__ __forceinline__ void mma2_commit(uint64_t *bar)
{
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xFFFFFFFF;\n"
                 " @e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
                     smem_u32(bar)),
                 "h"((uint16_t)3)
                 : "memory");
}

__device__ __forceinline__ void tmem2_alloc(uint32_t *dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem2_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// descriptor of a tile whose N side is contiguous: rows (one a k) of 64 elements, 8 rows 1024 bytes apart, the next 64
// elements `next` bytes
__device__ __forceinline__ uint64_t mn128_desc(const void *tile, uint32_t next)
{
    const uint64_t addr = smem_u32(tile);
    return ((addr >> 4) & 0x3FFFull) | ((uint64_t)(next >> 4) << 16) | ((1024ull >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// The word at p once it is the tile's, which its upper 28 bits say. (Read before the wait for the tile's S, it mostly is. That
// wait does not order it: in a pair's second CTA the barrier passes by way of the first. A wait for a barrier of the word's
// own instead: latent vectors of 256 126 us for 121, of 128 115.4 for 112.7.)
static __device__ __noinline__ uint32_t latent_gone(const uint32_t *p, uint32_t tile, uint32_t *status, unsigned long long wait_ns)
{
    const uint64_t t0 = globaltimer();
    uint32_t v;
    do
        v = *reinterpret_cast<const volatile uint32_t *>(p);
    while ((v ^ tile) >> 4 && globaltimer() - t0 <= wait_ns);
    if ((v ^ tile) >> 4)
        atomicOr(status, (uint32_t)MOE_WS_TIMEOUT);
    return v;
}

// NaN in the dimensions d .. d + n - 1 of a row's results in which a drafted token (of those after the sequence b's first
// `prefix`) that the row sees (mask) holds a value that is not finite: in part, pieces of four `step` apart, or in out
// (rarely needed: out of line)
static __device__ __noinline__ void latent_odd(const LatentArgs &a, int b, int prefix, unsigned long long mask, int d, int n,
                                               float *part, int step, uint16_t *out)
{
    const TreeArgs &t = a.t;
    for (; mask; mask &= mask - 1) {
        const int token = prefix + __ffsll((long long)mask) - 1, page = t.table[b * t.table_stride + token / t.k.page];
        if (page < 0 || page >= t.n_pages)
            continue;
        const uint16_t *row = reinterpret_cast<const uint16_t *>(t.pages) +
                              ((long long)page * t.k.page + token % t.k.page) * (t.k.dim + a.rope) + d;
        for (int i = 0; i < n; ++i) {
            if ((row[i] & 0x7F80u) != 0x7F80u)
                continue;
            if (part)
                part[(size_t)(i / 4) * step + i % 4] = NAN;
            else
                out[i] = 0x7FFF;
        }
    }
}

template <int L>
__global__ void __launch_bounds__(MOE_LTC_THREADS, 1) moe_latent_tc_kernel(const __grid_constant__ LatentArgs a, const int stages)
{
    using T = LtcShape<L>;
    constexpr int ROWS = MOE_LTC_ROWS, TOKENS = MOE_LTC_TOKENS;
    constexpr uint32_t O_COL = 64;  // of tensor memory: S (two of 32 columns), O
    extern __shared__ __align__(1024) uint8_t smem_any[];
    uint8_t *sq = smem_any, *sp = smem_any + T::P_AT, *ring = smem_any + T::RING_AT, *small = ring + (size_t)stages * T::STAGE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(small);
    uint64_t *full = bars, *empty = bars + 8, *v_full = bars + 16, *s_full = bars + 24;  // [stages]
    uint64_t *p_full = bars + 32, *pv_done = bars + 34, *v_here = bars + 36;             // [2]
    uint64_t *q_full = bars + 38, *o_free = bars + 40, *drained = bars + 41;             // q_full [2], by items; drained [4]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 45);
    float *top_of = reinterpret_cast<float *>(small + 384);  // [2][2][64]
    uint32_t *gone = reinterpret_cast<uint32_t *>(top_of + 256);  // [16] at t % 16: t, and tile t's 16-token groups that are not there
    long long *scan = reinterpret_cast<long long *>(gone + 16), *cum = scan + 32;  // cum [batch + 1]
    int *count = reinterpret_cast<int *>(scan + 20), *items = reinterpret_cast<int *>(cum + a.t.batch + 1);  // items [batch + 1]
    const TreeArgs &t = a.t;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = cta_rank();
    const unsigned pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    uint32_t *status = t.ctrl + MOE_CTRL_STATUS;

    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
            mbar_init(v_full + s, 1);
            mbar_init(s_full + s, 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(p_full + x, 2 * MOE_LTC_SOFT);
            mbar_init(pv_done + x, 1);
            mbar_init(v_here + x, 1);
            mbar_init(q_full + x, 2 * MOE_LTC_SOFT);
        }
        mbar_init(o_free, 2 * MOE_LTC_SOFT);
        for (int i = 0; i < 4; ++i)
            mbar_init(drained + i, 1);
        fence_barrier_init();
    }
    if (tid < 16)
        gone[tid] = ~0u;
    pdl_wait();  // before tensor memory is taken: the last kernel may still need it
    if (warp == 0)
        tmem2_alloc(tmem_slot, 512);
    long long lo, hi, run;
    tc_fence_before();
    tree_list<L, ROWS, TOKENS, MOE_LTC_COST, MOE_LTC_THREADS>(t, cum, items, scan, count, lo, hi, run, pair, pairs);
    pair_sync();  // the barriers of both CTAs stand
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = (int)(hi - lo);
    pdl_launch_dependents();
    if (tiles == 0 && tid == 0 && rank == 0)
        t.cuts[pair].runs = 0;
    // (a poll that does not hold the warp first: 15 clocks where the phase is complete, one that may 69; and the clock,
    // which takes longer than most waits, last)
    auto wait = [&](uint64_t *bar, int phase) {
        return mbar_try_wait(bar, (uint32_t)phase & 1u) || tree_poll(bar, (uint32_t)phase & 1u) ||
               tree_wait_on(bar, (uint32_t)phase & 1u, status, t.wait_ns);
    };
    auto drain = [&](uint64_t *bar, int phase) { tree_wait_on(bar, (uint32_t)phase & 1u, status, max(t.wait_ns, MOE_TREE_DRAIN_NS)); };
    auto to_item = [&](int u, TreeItem &it) {
        if (u == 0)
            it = tree_item<ROWS, TOKENS>(t, cum, lo);
        else
            tree_next<ROWS, TOKENS>(t, cum, it);
    };
    auto item_end = [&](const TreeItem &it) { return (int)(min(hi, it.lo + it.units) - lo); };
    // lane i < 4: where the i-th 16 tokens of tile u are, in two steps, so that the table's entry can come under a wait: the
    // entry (block -1: past the length), then the slot; where there is none, one past the pool, which reads as zeros
    const int no_slot = t.n_pages * t.k.page, page_blocks = t.k.page / 16;
    struct Place {
        int page, block;
    };
    auto look = [&](const TreeItem &it, int u) {
        const int blk = (int)(lo + u - it.lo) * (TOKENS / 16) + (lane & 3);
        const int at = (int)((unsigned long long)(unsigned)blk * a.per_page >> 36);
        const bool in = blk * 16 < it.len;
        return Place{in ? t.table[it.b * t.table_stride + at] : -1, in ? blk - at * page_blocks : -1};
    };
    auto find = [&](const Place &p, bool tell) {
        if (p.page >= 0 && p.page < t.n_pages)
            return p.page * t.k.page + p.block * 16;
        if (tell && lane < 4 && p.block >= 0)
            atomicOr(status, (uint32_t)MOE_WS_INDEX);
        return no_slot;
    };
    // copies of chunks `first` on (`n` of them) of the tokens' half h of a tile to `to`, counted by `bar` (pair_bar)
    auto copy = [&](const CUtensorMap *map, uint8_t *to, int first, int n, int slots, int h, uint32_t bar) {
        const int s0 = __shfl_sync(0xFFFFFFFFu, slots, 2 * h), s1 = __shfl_sync(0xFFFFFFFFu, slots, 2 * h + 1);
        if (a.big) {
            if (lane == 0)
                pair_load_3d(to, map, 0, s0, first, bar);
        } else {
            for (int i = lane; i < 2 * n; i += 32)
                pair_load_3d(to + (i >> 1) * MOE_LTC_CHUNK + (i & 1) * 2048, map, 0, i & 1 ? s1 : s0, first + (i >> 1), bar);
        }
    };
    // a tile whose tokens not all rows see, or not all of which are there
    auto special = [&](const TreeItem &it, int u) { return (int)(lo + u - it.lo) * TOKENS + TOKENS > it.len - it.n; };

    if (warp == MOE_LTC_SOFT) {
        // ---------------- this CTA's half of each tile's tokens, whole rows
        bool ok = true;
        int u = 0, end = 0, s = 0, phase = 0;
        TreeItem it{};
        Place next{};
        auto look_on = [&](int v) {
            if (v < tiles) {
                if (v == end) {
                    to_item(v, it);
                    end = item_end(it);
                }
                next = look(it, v);
            }
        };
        look_on(0);
        for (; u < tiles; ++u) {
            const Place now = next;
            look_on(u + 1);
            const int slots = find(now, rank == 0);
            const uint32_t out = __ballot_sync(0xFFFFFFFFu, slots == no_slot) & 15u;
            if (u >= stages)
                ok = __all_sync(0xFFFFFFFFu, wait(empty + s, phase - 1));
            if (!ok)
                break;
            uint8_t *to = ring + (size_t)s * T::STAGE;
            if (lane == 0) {
                *reinterpret_cast<volatile uint32_t *>(gone + (u & 15)) = (uint32_t)u << 4 | out;
                if (rank == 0)  // both CTAs' copies (the other's may come before this)
                    mbar_arrive_expect_tx(full + s, 2 * T::STAGE);
            }
            __syncwarp();
            const uint32_t bar = pair_bar(full + s, 0);
            copy(&a.keys, to, 0, T::CHUNKS, slots, rank, bar);
            const int s0 = __shfl_sync(0xFFFFFFFFu, slots, 2 * rank), s1 = __shfl_sync(0xFFFFFFFFu, slots, 2 * rank + 1);
            if (lane == 0)
                pair_load_2d(to + T::CHUNKS * MOE_LTC_CHUNK, &a.ropes, 0, s0, bar);
            if (lane == 1 && !a.big)
                pair_load_2d(to + T::CHUNKS * MOE_LTC_CHUNK + 2048, &a.ropes, 0, s1, bar);
            if (++s == stages) {
                s = 0;
                ++phase;
            }
        }
        for (int k = max(0, u - stages); k < u; ++k)  // nothing in flight, nothing to arrive when the CTA ends
            drain(ok ? empty + k % stages : rank == 0 ? full + k % stages : drained + 3, ok || rank == 0 ? k / stages : 0);
    } else if (warp == MOE_LTC_SOFT + 4) {
        // ---------------- the other tokens' values, once the tile's S is there
        bool ok = true;
        int u = 0, end = 0, s = 0, phase = 0;
        const int other = 1 - (int)rank;
        uint32_t sent = 0;  // of v_here: phases begun, by x, a bit each for some and for their parity
        TreeItem it{};
        for (; u < tiles; ++u) {
            if (u == end) {
                to_item(u, it);
                end = item_end(it);
            }
            const Place p = look(it, u);
            ok = __all_sync(0xFFFFFFFFu, wait(s_full + s, phase));
            if (!ok)
                break;
            const int slots = find(p, false);
            // counted by the first CTA's barrier, but in a tile that the softmax warps look through by their own CTA's
            const bool own = special(it, u);
            if (lane == 0 && (rank == 0 || own))
                mbar_arrive_expect_tx(rank == 0 ? v_full + s : v_here + (u & 1), (own ? 1 : 2) * T::HALF * MOE_LTC_CHUNK);
            if (own && rank == 1)
                sent = (sent | 1u << (u & 1)) ^ 4u << (u & 1);
            __syncwarp();
            copy(&a.values, ring + (size_t)s * T::STAGE + other * T::HALF * MOE_LTC_CHUNK, (int)rank * T::HALF, T::HALF, slots,
                 other, own && rank == 1 ? pair_bar(v_here + (u & 1), 1) : pair_bar(v_full + s, 0));
            if (++s == stages) {
                s = 0;
                ++phase;
            }
        }
        for (int k = max(0, u - stages); k < u; ++k) {
            if (rank == 0)
                drain(v_full + k % stages, k / stages);
            else if (!ok)
                drain(drained + 3, 0);
        }
        for (int x = 0; x < 2; ++x)
            if (sent >> x & 1)
                drain(v_here + x, (int)(sent >> (2 + x) & 1) - 1);
    } else if (warp >= MOE_LTC_SOFT && rank == 0) {
        // ---------------- the products: two warps those of S, a tile each in turn, another those of O, so that one's
        // waits pass under the others' products
        const int role = warp - MOE_LTC_SOFT - 1;
        const bool scores = role != 2;
        constexpr uint32_t id_s = mma_idesc(ROWS, TOKENS, true), id_o = mma_idesc(ROWS, T::N, true) | (1u << 16);
        const uint64_t qd = sw128_desc(sq), pd = sw128_desc(sp), rd = sw128_desc(ring), vd = mn128_desc(ring, MOE_LTC_CHUNK);
        const uint32_t tm = __reduce_max_sync(0xFFFFFFFFu, tmem);  // (what the loops need is the same in all lanes)
        const int n = __reduce_max_sync(0xFFFFFFFFu, tiles);
        bool ok = true;
        int end = 0, item = -1, s = 0, phase = 0;
        TreeItem it{};
        auto all = [&](bool v) { return __all_sync(0xFFFFFFFFu, v) != 0; };
        for (int u = 0; u < n; ++u) {
            const int x = u & 1;
            const bool first = all(u == end);
            if (first) {
                to_item(u, it);
                end = item_end(it);
                ++item;
                ok = ok && (scores ? all(wait(q_full + (item & 1), item >> 1)) : item == 0 || all(wait(o_free, item - 1)));
            }
            if (scores && x == (role != 0)) {
                // S of tile u, in the place of the last but one, which has been read (and first that wait: then the tile
                // before has had its turn, and no phase of `full` is passed over)
                ok = ok && (u < 2 || all(wait(p_full + x, (u >> 1) - 1))) && all(wait(full + s, phase));
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t k = rd + (uint32_t)(s * T::STAGE) / 16;
#pragma unroll
                for (int d = 0; d <= T::CHUNKS; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma2_f16(tm + x * 32, qd + (d * T::Q_CHUNK + i * 32) / 16, k + (d * MOE_LTC_CHUNK + i * 32) / 16, id_s,
                                 d + i > 0);
                mma2_commit(s_full + s);  // (by stages, so that the values' copies may lag)
            } else if (!scores) {  // O += P V
                ok = ok && all(wait(v_full + s, phase)) && all(wait(p_full + x, u >> 1));
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t v = vd + (uint32_t)(s * T::STAGE) / 16, p = pd;
#pragma unroll
                for (int d = 0; d < L / T::N; ++d)
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 16 tokens: 32 bytes of P, 2048 of V
                        mma2_f16(tm + O_COL + d * (T::N / 2), p + k * 2,
                                 v + (((k >> 1) * T::HALF + d * (T::N / 128)) * MOE_LTC_CHUNK + (k & 1) * 2048) / 16, id_o,
                                 !first || k > 0);
                mma2_commit(empty + s);
                mma2_commit(pv_done + x);
            }
            if (++s == stages) {
                s = 0;
                ++phase;
            }
        }
        if (n > 0) {  // what has been issued ends before tensor and shared memory are given back
            mma2_commit(drained + role);
            drain(drained + role, 0);
        }
    } else if (warp < MOE_LTC_SOFT) {
        // ---------------- softmax: row `row` of this CTA's, tokens (dimensions of O) of half `half`. No loop is left
        // early: the warps of a pair meet at barriers.
        const int row = tid & 63, half = tid >> 6, mine = (int)rank * 64 + row;
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        auto meet = [&]() { asm volatile("barrier.cta.sync %0, 64;" ::"r"(1 + (warp & 1)) : "memory"); };
        const float c = t.join_c, turn = t.scale == 0.0f ? 0.0f : t.scale < 0.0f ? -1.0f : 1.0f;
        bool ok = true;
        int item = 0, s = 0, phase = 0;  // s, phase: the tile's stage and its phase
        uint32_t seen = 0;  // by x, a bit each: parity of the tiles looked through
        // an item's queries, once the last item's S have been made (this warp has seen the last): asked for, and there
        auto ask = [&](const TreeItem &i) {
            const int first = i.block * ROWS + (int)rank * 64, here = min(64, i.n * t.group - first);
            for (int r = warp; r < here; r += MOE_LTC_SOFT) {
                const int token = i.first + (first + r) / t.group, head = (first + r) % t.group;
                const uint16_t *q = t.q + token * t.q_tok + head * t.q_head, *qr = a.qr + token * a.qr_tok + head * a.qr_head;
                uint8_t *to = sq + r * 128;
#pragma unroll
                for (int i = lane; i < T::CHUNKS * 8 + 8; i += 32) {
                    const bool turning = i >= T::CHUNKS * 8;
                    const int k = turning ? i - T::CHUNKS * 8 : i;
                    uint4 *at = reinterpret_cast<uint4 *>(to + (i >> 3) * T::Q_CHUNK + (((i & 7) ^ (r & 7)) << 4));
                    if (turning && k >= a.rope / 8)
                        *at = make_uint4(0, 0, 0, 0);
                    else if (turning ? a.qr_wide : t.q_wide)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(at)),
                                     "l"((turning ? qr : q) + k * 8)
                                     : "memory");
                    else
                        *at = latent_get((turning ? qr : q) + k * 8, false);
                }
            }
        };
        auto there = [&](int i) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                arrive_first(q_full + (i & 1));
        };
        TreeItem it{}, following{};
        if (tiles > 0) {
            to_item(0, it);
            ask(it);
            there(0);
        }
        for (int u = 0; u < tiles; ++item, it = following) {
            const int end = item_end(it), at = it.block * ROWS + mine, rows = it.n * t.group;
            const bool live = at < rows;
            const int node = live ? at / t.group : 0;
            // the drafted tokens that it sees
            const unsigned long long mask = !live ? 0 : (t.mask ? t.mask[it.first + node] : (2ull << node) - 1) &
                                                         (it.n < 64 ? (1ull << it.n) - 1 : ~0ull);
            const int prefix = it.len - it.n;
            float m = -INFINITY, l = 0.0f;
            bool fresh = true, odd = false;  // odd: a token that it sees in a masked tile has a score of -inf
            for (; u < end; ++u) {
                const int x = u & 1;
                uint32_t out = *reinterpret_cast<volatile uint32_t *>(gone + (u & 15));
                ok = ok && wait(s_full + s, phase);
                __syncwarp();
                tc_fence_after();
                const int first = (int)(lo + u - it.lo) * TOKENS;
                float v[32];
                tmem_ld32(lanes + x * 32, v);
                if (turn != 1.0f)
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        v[i] *= turn;
                if (ok && (out ^ (uint32_t)u << 4) >> 4) {
                    out = latent_gone(gone + (u & 15), (uint32_t)u << 4, status, t.wait_ns);
                    ok = (out ^ (uint32_t)u << 4) >> 4 == 0;
                }
                out &= 15u;
                const bool masked = first + TOKENS > prefix || out;
                if (masked) {
                    const int off = prefix - (first + half * 32);
                    uint32_t vis = off >= 32  ? ~0u
                                   : off >= 0 ? ((1u << off) - 1) | (uint32_t)(mask << off)
                                   : off > -64 ? (uint32_t)(mask >> -off)
                                               : 0u;
                    vis &= (out >> (2 * half) & 1 ? 0u : 0xFFFFu) | (out >> (2 * half + 1) & 1 ? 0u : 0xFFFF0000u);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        odd |= vis >> i & 1 && v[i] == -INFINITY;
                        v[i] = vis >> i & 1 ? v[i] : -INFINITY;
                    }
                }
                float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                    top4[i >> 1 & 3] = max3(top4[i >> 1 & 3], v[i], v[i + 1]);
                float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                float *tops = top_of + x * 128;
                tops[half * 64 + row] = top;
                meet();
                top = fmaxf(top, tops[(half ^ 1) * 64 + row]);
                const bool moves = live && (top - m) * c > MOE_LTC_SLACK;  // (rows that are none hold anything)
                if (__any_sync(0xFFFFFFFFu, moves)) {
                    const float f = moves ? ex2((m - top) * c) : 1.0f;
                    m = moves ? top : m;
                    l *= f;
                    if (!fresh) {
                        ok = ok && wait(pv_done + (x ^ 1), (u - 1) >> 1);  // O of the last tile is there
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int k = 0; k < T::O_COLS; k += 16) {
                            float o[16];
                            uint32_t w[16];
                            tmem_ld16(lanes + O_COL + k, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = __float_as_uint(o[i] * f);
                            tmem_st16(lanes + O_COL + k, w);
                        }
                        tmem_st_wait();
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : -m;
                const F2 ref2(ref, ref), c2(c, c);
                uint32_t w[16];
                F2 sum(0.0f, 0.0f), sum1(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float e0, e1;
                    mul2(add2(F2(v[i], v[i + 1]), ref2), c2).get(e0, e1);
                    // (bf16, by 2^-8 at most: the tensor core takes P only in the type of the values beside it)
                    const uint32_t p = pack_bf2(ex2(e0), ex2(e1));
                    w[i / 2] = p;
                    F2 &to = i & 2 ? sum1 : sum;
                    to = add2(to, F2(bf16_lo(p), bf16_hi(p)));  // as rounded
                }
                sum = add2(sum, sum1);
                float l0, l1;
                sum.get(l0, l1);
                l += l0 + l1;
                fresh = false;
                if (u > 0)  // P of the last tile has been read
                    ok = ok && wait(pv_done + (x ^ 1), (u - 1) >> 1);
                uint8_t *p = sp + row * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4 *>(p + (((half * 4 + i) ^ (row & 7)) << 4)) =
                        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                if (special(it, u)) {
                    ok = ok && (rank == 0 ? wait(v_full + s, phase) : wait(v_here + x, (int)(seen >> x & 1)));
                    seen ^= 1u << x;
                    // Values past the length are anything, and those of drafted tokens need not be numbers, which must not
                    // reach rows that do not see them: zeros in their place. A row that sees one of them scores it NaN or
                    // +inf, which makes the row NaN, or -inf, which is seen to at the item's end.
                    uint8_t *values = ring + (size_t)s * T::STAGE;
                    for (int i = tid; i < 64 * T::HALF * 8; i += MOE_LTC_SOFT * 32) {
                        const int token = i / (T::HALF * 8), piece = i % (T::HALF * 8);
                        if (first + token < prefix)
                            continue;
                        uint4 *q = reinterpret_cast<uint4 *>(values + ((token >> 5) * T::HALF + piece / 8) * MOE_LTC_CHUNK +
                                                             (token & 31) * 128 + (piece & 7) * 16);
                        uint4 y = make_uint4(0, 0, 0, 0);
                        if (first + token < it.len) {
                            y = *q;
                            y = make_uint4(finite_bf2(y.x), finite_bf2(y.y), finite_bf2(y.z), finite_bf2(y.w));
                        }
                        *q = y;
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    arrive_first(p_full + x);
                if (++s == stages) {
                    s = 0;
                    ++phase;
                }
            }
            // ---- the item's end. The next one's queries first, so that its S are made under it
            following = it;
            if (u < tiles) {
                to_item(u, following);
                ask(following);
            }
            float *sums = top_of + (end & 1) * 128;  // (the maxima that the last tile has not used)
            sums[half * 64 + row] = odd ? -l : l;  // (sums are not negative)
            ok = ok && wait(pv_done + ((end - 1) & 1), (end - 1) >> 1);
            if (u < tiles)
                there(item + 1);
            meet();
            __syncwarp();
            const float theirs = sums[(half ^ 1) * 64 + row];
            odd |= __float_as_int(theirs) < 0;
            l += fabsf(theirs);
            tc_fence_after();
            const bool whole = it.lo >= lo && it.lo + it.units <= hi;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            float *part = t.part + ((size_t)pair * 2 + (it.lo <= lo ? 0 : 1)) * ROWS * (L + 2);
            uint16_t *to = t.out + (it.first + node) * t.o_tok + (live ? at % t.group : 0) * t.o_head + half * (L / 2);
#pragma unroll 1
            for (int k = 0; k < T::O_COLS; k += 32) {
                float o[32];
                tmem_ld32(lanes + O_COL + k, o);
                if (live && !whole) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        reinterpret_cast<float4 *>(part)[(half * (L / 2) + k + i) / 4 * ROWS + mine] =
                            make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else if (live) {
#pragma unroll
                    for (int i = 0; i < 32; i += 8)
                        latent_put(to + k + i,
                                   make_uint4(pack_bf2(o[i] * inv, o[i + 1] * inv), pack_bf2(o[i + 2] * inv, o[i + 3] * inv),
                                              pack_bf2(o[i + 4] * inv, o[i + 5] * inv), pack_bf2(o[i + 6] * inv, o[i + 7] * inv)),
                                   t.o_wide);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                arrive_first(o_free);
            if (live && odd)  // a weight of 0 times a value that is not finite
                latent_odd(a, it.b, prefix, mask, half * (L / 2), L / 2,
                           whole ? nullptr : part + ((size_t)half * (L / 8) * ROWS + mine) * 4, 4 * ROWS, to);
            if (live && !whole && half == 0) {
                part[ROWS * L + mine] = m;  // (not as an exponent: m c may pass f32 where differences times c need not)
                part[ROWS * L + ROWS + mine] = l;
            }
            if (end == tiles && tid == 0 && rank == 0)
                tree_cut<ROWS, MOE_LTC_COST>(t, it, items, lo, run, pair);
            meet();  // the sums have been read
        }
    }
    tc_fence_before();
    __syncthreads();
    pair_sync();
    if (warp == 0)
        tmem2_dealloc(tmem, 512);
    pair_sync();
}

// Joins the partials of cut items of few parts, in order: a thread a row and 16 dimensions (a sector of the output), the
// rows of a warp side by side in the partials; CTA (run, 32 dimensions). moe_tree_join_kernel, whose threads share an
// item's parts, takes those of many.
#define MOE_LTC_JOIN_THREADS 256
template <int L>
__global__ void __launch_bounds__(MOE_LTC_JOIN_THREADS) moe_latent_join_kernel(const __grid_constant__ TreeArgs a)
{
    constexpr int ROWS = MOE_LTC_ROWS, U = 4;  // parts in flight
    const int r = threadIdx.x % ROWS, d = (blockIdx.y * (MOE_LTC_JOIN_THREADS / ROWS) + threadIdx.x / ROWS) * 16;
    constexpr size_t SIZE = (size_t)ROWS * (L + 2);
    pdl_wait();
    const TreeCut c = a.cuts[blockIdx.x];
    const int rr = c.block * ROWS + r;
    if (c.runs == 0 || rr >= c.n * a.group)
        return;
    // part i: of the first run the second slot, unless the item begins with the run
    const float *base = a.part + (size_t)blockIdx.x * 2 * SIZE;
    auto part = [&](int i) { return base + (i == 0 && !c.whole_run ? SIZE : 2 * i * SIZE); };
    float m = -INFINITY;
    for (int i0 = 0; i0 <= c.runs; i0 += 8) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = i0 + i <= c.runs ? part(i0 + i)[ROWS * L + r] : -INFINITY;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            m = fmaxf(m, v[i]);
    }
    float4 o[4];
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = 0; i0 <= c.runs; i0 += U) {
        float4 v[U][4];
        float f[U], w[U];
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i <= c.runs) {
                const float *p = part(i0 + i);
                f[i] = p[ROWS * L + r];
                w[i] = p[ROWS * L + ROWS + r];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    v[i][k] = reinterpret_cast<const float4 *>(p)[(d / 4 + k) * ROWS + r];
            }
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (i0 + i <= c.runs) {
                const float x = f[i] == -INFINITY ? 1.0f : ex2((f[i] - m) * a.join_c);  // a NaN sum stays
                l += w[i] * x;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    o[k].x = fmaf(v[i][k].x, x, o[k].x);
                    o[k].y = fmaf(v[i][k].y, x, o[k].y);
                    o[k].z = fmaf(v[i][k].z, x, o[k].z);
                    o[k].w = fmaf(v[i][k].w, x, o[k].w);
                }
            }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *to = a.out + (c.first + rr / a.group) * a.o_tok + rr % a.group * a.o_head + d;
#pragma unroll
    for (int k = 0; k < 4; k += 2)
        latent_put(to + 4 * k,
                   make_uint4(pack_bf2(o[k].x * inv, o[k].y * inv), pack_bf2(o[k].z * inv, o[k].w * inv),
                              pack_bf2(o[k + 1].x * inv, o[k + 1].y * inv), pack_bf2(o[k + 1].z * inv, o[k + 1].w * inv)),
                   a.o_wide);
}

}  // namespace moe

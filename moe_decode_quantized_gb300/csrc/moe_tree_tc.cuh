// moe_tree_tc.cuh -- tree attention for more than 32 query rows a kv head, on
// the 5th-generation tensor cores: the same sums, list of work and partials
// as moe_tree_attn.cuh, in tiles of 128 tokens and up to 128 rows an M tile.
//
//   S [128 rows x 128 tokens] = Q [rows x 128] K^T,
//   O [128 rows x 128 dims] += P [rows x tokens] V,
// S, P and O in tensor memory, a row a lane, so that a row's maximum and sum
// are one thread's. P takes the place of its S, as f16, and is the second
// product's A operand from there; K and V lie in shared memory as 128-byte
// rows of 64 dimensions in the 128-byte swizzle (V read with the dimensions
// contiguous). Two groups of four softmax warps, each with an S and an O:
//  - a row block of more than 128 rows: a group an M tile, every token tile
//    for both, so that one's softmax runs under the other's products;
//  - up to 128 rows: the groups take the token tiles in turn, each keeping its
//    own maximum, sum and O, and are joined at the item's end.
// A reference m moves only when a score passes it by 2^8 (O is then scaled).
//
// One CTA an SM: a warp copies the cache's blocks, eight bring the queries and
// turn codes into f16 tiles (K of tile t + 1 while tile t's softmax runs, then
// V of tile t once the second product of tile t - 1 is done), one thread
// issues the products.
//
// 61 rows of 8 heads over 100003 tokens take 123 us, 810 TFLOP/s of products
// (41 % of the measured peak), 16 chains of 16 rows of 4 heads over 4000 tokens
// 68 us. A tile of two M tiles takes some 4500 clocks: the
// products 3300, in order and waiting once a tile for the K that takes the last
// one's place, beside a softmax of some 2000 clocks an M tile. Tiles of one M
// tile take 3000 to 3300, bound by the turning of codes, which no more rows
// share. A second place for K, at the price of halves of raw stages, was measured
// at 131 and 133 us where one place took 123 and left out.
#pragma once
#include "moe_tc.cuh"
#include "moe_tree_attn.cuh"

namespace moe {

#define MOE_TTC_TOKENS 128
#define MOE_TTC_ROWS 256  // of a row block: two M tiles
#define MOE_TTC_COST 2    // of an item, beside its tiles (moe_tree_attn.cuh)
#define MOE_TTC_SOFT 8    // softmax warps
#define MOE_TTC_CODE 8    // warps that turn codes into f16
#define MOE_TTC_THREADS ((MOE_TTC_SOFT + MOE_TTC_CODE + 2) * 32)

template <int FMT>
struct TtcShape {
    static constexpr int D = 128;
    static constexpr int RB = FMT == MOE_KV_Q8 ? D : D / 2;
    static constexpr int GR = D / MOE_KV_GROUP;
    static constexpr int HALF = 16 * RB + 16 * GR * (FMT == MOE_KV_Q8 ? 2 : 4);
    static constexpr int BLOCK = 2 * HALF;
    static constexpr int STAGE = 8 * BLOCK;                // a tile's blocks
    static constexpr int PANEL = MOE_TTC_TOKENS * 128;     // 64 dimensions of 128 tokens (rows)
    static constexpr int K_AT = 0, V_AT = 2 * PANEL, Q_AT = 4 * PANEL;  // Q: [M tile][2 panels]
    static constexpr int RAW_AT = Q_AT + 4 * PANEL;
    // after the raw stages: barriers, rows' multipliers, the groups' references and sums, the scan and the list
    static constexpr int SMALL = 256 + 4 * 4 * 256 + 4 * 128 * 8 + 32 * 8;
};

// descriptor of a tile whose M (N) side is contiguous: 128-byte rows of 64
// elements, one row a k, in the 128-byte swizzle; 8 rows are 1024 bytes apart
// (stride offset), the next 64 elements PANEL bytes (leading offset)
__device__ __forceinline__ uint64_t mn_desc(const void *tile)
{
    const uint64_t addr = smem_u32(tile);
    return ((addr >> 4) & 0x3FFFull) | ((uint64_t)(MOE_TTC_TOKENS * 128 / 16) << 16) | ((1024ull >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

// a place in a ring and its phase, without a division
struct TtcRing {
    int slot = 0, phase = 0;
    __device__ __forceinline__ void next(int n)
    {
        if (++slot == n) {
            slot = 0;
            ++phase;
        }
    }
};

// the softmax warps' own barrier
__device__ __forceinline__ void soft_sync() { asm volatile("barrier.cta.sync 1, %0;" ::"n"(MOE_TTC_SOFT * 32) : "memory"); }

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

// stores 16 consecutive dimensions of a token: pieces of 16 bytes at off and off ^ 16
__device__ __forceinline__ void put_sixteen(uint8_t *tile, uint32_t off, const uint32_t (&h)[8])
{
    *reinterpret_cast<uint4 *>(tile + off) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(tile + (off ^ 16u)) = make_uint4(h[4], h[5], h[6], h[7]);
}

template <int FMT>
__global__ void __launch_bounds__(MOE_TTC_THREADS, 1) moe_tree_tc_kernel(const __grid_constant__ TreeArgs a, const int stages)
{
    using T = TtcShape<FMT>;
    constexpr int D = T::D, ROWS = MOE_TTC_ROWS;
    constexpr uint32_t S_COL = 0, O_COL = 256;  // of tensor memory: S (and P) of the two groups, O of the two
    extern __shared__ __align__(1024) uint8_t smem_any[];
    uint8_t *smem = smem_any + (-smem_u32(smem_any) & 1023u);  // the swizzle goes by address bits
    uint8_t *sk = smem + T::K_AT, *sv = smem + T::V_AT, *sq = smem + T::Q_AT;
    uint8_t *raw = smem + T::RAW_AT, *small = raw + (size_t)stages * T::STAGE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(small);
    uint64_t *raw_full = bars, *raw_free = bars + 4, *q_full = bars + 8;  // [4] each; q_full of item i at i % 4
    uint64_t *k_full = bars + 12, *v_full = bars + 13, *k_done = bars + 14, *v_done = bars + 15, *o_done = bars + 16,
             *o_free = bars + 17, *s_full = bars + 18, *p_full = bars + 20;  // s_full, p_full [2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 22);
    uint64_t *drained = bars + 28;  // after a wait that ran out
    uint32_t *gone = tmem_slot + 1;  // [8] blocks of tile t that are not there, at t % 8: kept longer than its stage
    float *mul = reinterpret_cast<float *>(small + 256);  // [4][256] multipliers of the rows of item i, at i % 4
    float2 *stat = reinterpret_cast<float2 *>(mul + 1024);  // [2][2][128] (reference, sum) of item i, at i % 2, by group
    long long *scan = reinterpret_cast<long long *>(stat + 512), *cum = scan + 32;  // cum [batch + 1]
    int *count = reinterpret_cast<int *>(scan + 20), *items = reinterpret_cast<int *>(cum + a.batch + 1);  // items [batch + 1]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t *status = a.ctrl + MOE_CTRL_STATUS;

    if (tid == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(raw_full + s, 1);
            mbar_init(raw_free + s, MOE_TTC_CODE);
        }
        mbar_init(k_full, MOE_TTC_CODE);
        mbar_init(v_full, MOE_TTC_CODE);
        mbar_init(k_done, 1);
        mbar_init(v_done, 1);
        for (int i = 0; i < 4; ++i)
            mbar_init(q_full + i, MOE_TTC_CODE);
        mbar_init(drained, 1);
        mbar_init(o_done, 1);
        mbar_init(o_free, MOE_TTC_SOFT);
        for (int x = 0; x < 2; ++x) {
            mbar_init(s_full + x, 1);
            mbar_init(p_full + x, MOE_TTC_SOFT / 2);
        }
        fence_barrier_init();
    }
    pdl_wait();  // before tensor memory is taken: the last kernel may still need it
    if (warp == 0)
        tmem_alloc(tmem_slot, 512);
    long long lo, hi, run;
    tc_fence_before();
    tree_list<D, ROWS, MOE_TTC_TOKENS, MOE_TTC_COST, MOE_TTC_THREADS>(a, cum, items, scan, count, lo, hi, run);
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int tiles = (int)(hi - lo);
    pdl_launch_dependents();
    if (tiles == 0 && tid == 0)
        a.cuts[blockIdx.x].runs = 0;
    auto wait = [&](uint64_t *bar, int phase) {
        return tree_wait(bar, (uint32_t)phase & 1u, status, a.wait_ns);
    };
    // to the item that begins at tile t of this run (t = 0: the one it is in)
    auto to_item = [&](int t, TreeItem &it) {
        if (t == 0)
            it = tree_item<ROWS, MOE_TTC_TOKENS>(a, cum, lo);
        else
            tree_next<ROWS, MOE_TTC_TOKENS>(a, cum, it);
    };
    // the item's tiles of this run end before tile:
    auto item_end = [&](const TreeItem &it) { return (int)(min(hi, it.lo + it.units) - lo); };
    auto wide = [&](const TreeItem &it) { return it.n * a.group - it.block * ROWS > 128; };  // a group an M tile

    if (warp == MOE_TTC_SOFT + MOE_TTC_CODE) {
        // ---------------- the copies: lane i the i-th block of a tile
        const uint64_t policy = policy_evict_first();
        bool ok = true;
        int t = 0, end = 0;
        TreeItem it{};
        TtcRing ring;
        for (; t < tiles; ++t, ring.next(stages)) {
            if (t == end) {
                to_item(t, it);
                end = item_end(it);
            }
            const int blk = (int)(lo + t - it.lo) * 8 + lane, per_page = a.k.page / 16;
            const uint8_t *src = nullptr;
            if (lane < 8 && blk * 16 < it.len) {
                const int page = a.table[it.b * a.table_stride + blk / per_page];
                if (page < 0 || page >= a.n_pages)
                    atomicOr(status, (uint32_t)MOE_WS_INDEX);
                else
                    src = a.pages + (((size_t)page * a.k.heads + it.head) * per_page + blk % per_page) * T::BLOCK;
            }
            const uint32_t got = __ballot_sync(0xFFFFFFFFu, src != nullptr);
            const int s = ring.slot;
            if (t >= stages)
                ok = __all_sync(0xFFFFFFFFu, wait(raw_free + s, ring.phase - 1));
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
            tree_wait_on(raw_full + k % stages, (uint32_t)(k / stages) & 1u, status, max(a.wait_ns, MOE_TREE_DRAIN_NS));
    } else if (warp == MOE_TTC_SOFT + MOE_TTC_CODE + 1) {
        // ---------------- the products
        if (lane == 0) {
            constexpr uint32_t id_s = mma_idesc(128, 128, false), id_o = id_s | (1u << 16);
            const uint64_t kd = sw128_desc(sk), vd = mn_desc(sv);
            bool ok = true;
            // by group, a bit each: parity of the products S begun; whether O of the last is still to come; whether
            // that is the group's first of its item; whether the item has had one
            uint32_t jobs = 0, open = 0, fresh = 0, begun = 0;
            int open_tile = -1, end = 0, item = -1, of[2];  // of: the item of a group's last S
            bool two = false, closing = false;              // closing: the open tile is its item's last
            TreeItem it{};
            auto first = [&](int x, int m) {  // S of group x from M tile m
                const uint64_t qd = sw128_desc(sq + m * 2 * T::PANEL);
#pragma unroll
                for (int k = 0; k < 8; ++k) {  // 16 dimensions: 32 bytes, then the next panel
                    const int off = (k >> 2) * (T::PANEL / 16) + (k & 3) * 2;
                    mma_f16(tmem + S_COL + x * 128, qd + off, kd + off, id_s, k > 0);
                }
                mma_commit(s_full + x);
                jobs ^= 1u << x;
                open |= 1u << x;
                fresh = (fresh & ~(1u << x)) | (~begun & 1u << x);
                begun |= 1u << x;
                (x ? of[1] : of[0]) = item;
            };
            auto second = [&](int x) {  // O of group x += P V of the open tile
                if (!(open >> x & 1) || !ok)
                    return;
                const bool begins = fresh >> x & 1;
                const int i = x ? of[1] : of[0];
                ok = wait(v_full, open_tile) && wait(p_full + x, (int)(jobs >> x & 1) - 1) &&
                     (!begins || i == 0 || wait(o_free, i - 1));  // the last item's O has been read
                if (!ok)
                    return;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 8; ++k)  // 16 tokens: 8 columns of P, 2048 bytes of V
                    mma_f16_ts(tmem + O_COL + x * 128, tmem + S_COL + x * 128 + k * 8, vd + k * 128, id_o, !begins || k > 0);
                open &= ~(1u << x);
            };
            auto close = [&]() {  // after the last second product of the open tile
                mma_commit(v_done);
                if (closing)
                    mma_commit(o_done);
                closing = false;
                open_tile = -1;
            };
            for (int t = 0; t < tiles && ok; ++t) {
                if (t == end) {
                    const bool was = two;
                    to_item(t, it);
                    end = item_end(it);
                    two = wide(it);
                    closing = t > 0;
                    if (t > 0 && (was || two)) {  // both groups are needed (were in use)
                        second(0);
                        second(1);
                        close();
                    }
                    ++item;
                    begun = 0;
                    ok = ok && wait(q_full + (item & 3), item >> 2);
                }
                // two M tiles: O of the last tile frees the S that the next product writes; else the groups' S are
                // taken in turn, and O of the last tile comes after S of this one
                if (two) {
                    for (int x = 0; x < 2; ++x) {
                        second(x);
                        if (x == 1 && open_tile >= 0)
                            close();
                        ok = ok && wait(k_full, t);
                        if (!ok)
                            break;
                        tc_fence_after();
                        first(x, x);
                    }
                    mma_commit(k_done);
                } else {
                    ok = ok && wait(k_full, t);
                    if (!ok)
                        break;
                    tc_fence_after();
                    first(t & 1, 0);
                    mma_commit(k_done);
                    if (open_tile >= 0) {
                        second(t & 1 ^ 1);
                        close();
                    }
                }
                open_tile = t;
            }
            second(0);
            second(1);
            if (tiles > 0 && ok) {
                closing = true;
                close();
                ok = wait(o_done, item);
            }
            if (!ok) {  // products may be in flight: they end before tensor and shared memory are given back
                mma_commit(drained);
                tree_wait_on(drained, 0, status, max(a.wait_ns, MOE_TREE_DRAIN_NS));
            }
        }
    } else if (warp >= MOE_TTC_SOFT) {
        // ---------------- codes to f16: warp w the block w of a tile. The lanes of eight that a store serves at once
        // take pieces (tokens) that the swizzle puts in different banks.
        const int w = warp - MOE_TTC_SOFT, g = lane >> 2, t4 = lane & 3, turn = t4 >> 1;
        // K, first piece: 16 dimensions from 32 t4 + 16 turn of token g; the other piece is 32 bytes off (xor)
        const uint32_t k_off = (uint32_t)(turn * T::PANEL + (w * 16 + g) * 128 + ((((t4 & 1) * 4 + turn * 2) ^ g) << 4));
        // V, 16 dimensions from 16 g of token 2 t4 + (g & 1), and of 2 t4 + 1 - (g & 1)
        const int odd = g & 1;
        const uint32_t v_row = (uint32_t)((g >> 2) * T::PANEL + (w * 16 + 2 * t4) * 128);
        const uint32_t v_off[2] = {v_row + odd * 128 + ((((g & 3) * 2) ^ (2 * t4) ^ odd) << 4),
                                   v_row + (1 - odd) * 128 + ((((g & 3) * 2) ^ (2 * t4) ^ (1 - odd)) << 4)};
        constexpr int KP = FMT == MOE_KV_Q8 ? 4 : 2;  // 16-byte pieces of a block's K (V) codes a lane
        bool ok = true;
        TtcRing k_ring, v_ring;
        int end = 0, item = -1, left = 0;  // left: tokens of the item from this warp's block of the last K tile on
        TreeItem it{};
        auto keys = [&](int t) {  // K of tile t, and before an item's first the queries
            const bool begins = t == end;
            if (begins) {
                to_item(t, it);
                end = item_end(it);
                ++item;
            }
            left = it.len - (int)(lo + t - it.lo) * MOE_TTC_TOKENS - w * 16;
            const int s = k_ring.slot;
            if (t > 0)  // K and Q have been read
                ok = ok && wait(k_done, t - 1);
            if (begins) {
                const int rows = it.n * a.group - it.block * ROWS;
                for (int r = (tid >> 1) & 127; r < (rows > 128 ? ROWS : 128); r += 128) {  // a row a pair of threads
                    const bool live = r < rows;
                    const int rr = it.block * ROWS + (live ? r : 0);
                    uint32_t q[32];
                    const float c = tree_row<64, 2>(a, live, it.first + rr / a.group, it.head * a.group + rr % a.group,
                                                    (tid & 1) * 64, q);
                    if ((tid & 1) == 0)
                        mul[(item & 3) * 256 + r] = c;
                    uint8_t *p = sq + ((r >> 7) * 2 + (tid & 1)) * T::PANEL + (r & 127) * 128;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        *reinterpret_cast<uint4 *>(p + ((k ^ (r & 7)) << 4)) =
                            make_uint4(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_full + (item & 3));
            }
            ok = ok && wait(raw_full + s, k_ring.phase);
            k_ring.next(stages);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok)
                return;
            const uint8_t *b = raw + (size_t)s * T::STAGE + w * T::BLOCK;
            uint4 v[KP];
            uint32_t sc[2], mn[2];
#pragma unroll
            for (int i = 0; i < KP; ++i)
                v[i] = *reinterpret_cast<const uint4 *>(b + (FMT == MOE_KV_Q8 ? i ^ turn : i) * 512 + lane * 16);
#pragma unroll
            for (int nb = 0; nb < 2; ++nb) {
                const int at = (nb * 8 + g) * 4 + t4;
                if (FMT == MOE_KV_Q8) {
                    sc[nb] = h2(__half2half2(reinterpret_cast<const __half *>(b + 16 * T::RB)[at]));
                } else {
                    const uint32_t dm = reinterpret_cast<const uint32_t *>(b + 16 * T::RB)[at];
                    sc[nb] = dup_lo(dm);
                    mn[nb] = dup_hi(dm);
                }
            }
#pragma unroll
            for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t h[8];
                    if (FMT == MOE_KV_Q8) {
                        q8_sixteen(v[(nb * 2 + i) % KP], h2(sc[nb]), h);
                    } else {
                        const uint4 u = v[nb];
                        const bool hi2 = (i ^ turn) != 0;
                        q4_sixteen(hi2 ? u.z : u.x, hi2 ? u.w : u.y, h2(sc[nb]), h2(mn[nb]), h);
                    }
                    put_sixteen(sk, (k_off ^ (uint32_t)(i * 32)) + nb * 1024, h);
                }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(k_full);
        };
        auto values = [&](int t, int left) {  // V of tile t
            const int s = v_ring.slot;
            v_ring.next(stages);
            const bool there = !(*reinterpret_cast<volatile uint32_t *>(gone + (t & 7)) >> w & 1);
            const uint8_t *b = raw + (size_t)s * T::STAGE + w * T::BLOCK + T::HALF;
            const __half *p = reinterpret_cast<const __half *>(b + 16 * T::RB) + (g >> 1) * 16;
            uint4 v[KP];
            uint32_t sc[4], mn[4];
#pragma unroll
            for (int i = 0; i < KP; ++i)
                v[i] = *reinterpret_cast<const uint4 *>(b + (FMT == MOE_KV_Q8 ? i ^ odd : i) * 512 + lane * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tok = (i >> 1) * 8 + 2 * t4 + ((i & 1) ^ odd);
                const bool in = there && tok < left;  // else the bytes are anything: values of 0
                sc[i] = in ? h2(__half2half2(p[tok])) : 0u;
                if (FMT == MOE_KV_Q4)
                    mn[i] = in ? h2(__half2half2(p[T::GR * 16 + tok])) : 0u;
            }
            // A token that no row sees may never have been written: whatever its bytes, its values are numbers (they are
            // multiplied by weights of 0). Bounds past what the cache's writer makes: 472.5 (Q8); a minimum of +-60000
            // and a scale of (60000 - minimum) / 15, rounded up (Q4).
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __half2 most = h2(0x5FFF5FFFu);  // 511.75
                if (FMT == MOE_KV_Q4) {
                    const __half2 m = __hmax2(__hmin2(h2(mn[i]), h2(0x7B557B55u)), h2(0xFB55FB55u));  // +-60064
                    mn[i] = h2(m);
                    most = __hfma2(m, __float2half2_rn(-1.0f / 15), __float2half2_rn(4364.0f));
                }
                sc[i] = h2(__hmax2(__hmin2(h2(sc[i]), most), h2(0u)));
            }
            __syncwarp();
            if (lane == 0)  // the stage is in registers
                mbar_arrive(raw_free + s);
            if (t > 0)
                ok = ok && wait(v_done, t - 1);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok)
                return;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[8];
                if (FMT == MOE_KV_Q8) {
                    q8_sixteen(v[i % KP], h2(sc[i]), h);
                } else {
                    const uint4 u = v[i >> 1];
                    const bool hi2 = ((i & 1) ^ odd) != 0;
                    q4_sixteen(hi2 ? u.z : u.x, hi2 ? u.w : u.y, h2(sc[i]), h2(mn[i]), h);
                }
                put_sixteen(sv, v_off[i & 1] + (i >> 1) * 1024, h);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(v_full);
        };
        // K of tile t and V of tile t - 1. With two M tiles V first: the second products come before the first ones
        // of the next tile; else K first: S of the next tile is wanted while the softmax of the last two goes on.
        bool two = false;
        for (int t = 0, here = 0; t <= tiles && ok; ++t) {
            const int last = here;
            const bool values_first = two;
#pragma unroll 1
            for (int step = 0; step < 2; ++step)
                if ((step == 0) == values_first) {
                    if (t > 0 && ok)
                        values(t - 1, last);
                } else if (t < tiles && ok) {
                    keys(t);
                    here = left;
                    two = wide(it);
                }
        }
    } else {
        // ---------------- softmax: group x, row `row` of its M tile. Loops over columns stay loops: the four roles
        // share the instruction cache.
        const int x = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_at = lanes + S_COL + x * 128, o_at = lanes + O_COL + x * 128;
        bool ok = true;
        int jobs = 0, item = 0;
        TreeItem it{};
        for (int t = 0; t < tiles; ++item) {
            // every warp goes through every item's barrier, a failed wait or not
            to_item(t, it);
            const int end = item_end(it), rows = it.n * a.group - it.block * ROWS;
            const bool two = wide(it);
            const int local = two ? x * 128 + row : row, at = it.block * ROWS + local;  // this thread's row
            const bool live = local < rows;
            const int node = live ? at / a.group : 0;
            // the drafted tokens that it sees
            const unsigned long long mask = !live ? 0 : (a.mask ? a.mask[it.first + node] : (2ull << node) - 1) &
                                                         (it.n < 64 ? (1ull << it.n) - 1 : ~0ull);
            const int prefix = it.len - it.n;
            ok = ok && wait(q_full + (item & 3), item >> 2);
            const float c = mul[(item & 3) * 256 + local];
            float m = -INFINITY, l = 0.0f;  // m: the reference as a score, so that exponents are multiples of differences
            bool fresh = true;
            for (int u = t + (two ? 0 : (t ^ x) & 1); u < end; u += two ? 1 : 2) {
                ok = ok && wait(s_full + x, jobs++);
                if (!__all_sync(0xFFFFFFFFu, ok)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int first = (int)(lo + u - it.lo) * MOE_TTC_TOKENS;
                const uint32_t out = *reinterpret_cast<volatile uint32_t *>(gone + (u & 7));
                const bool masked = first + MOE_TTC_TOKENS > prefix || out;
                if (masked)  // the scores of tokens that are not seen to -inf, so that the passes below stay short
#pragma unroll 1
                    for (int k = 0; k < 128; k += 16) {  // bit i: token first + k + i is seen
                        const int off = prefix - (first + k);
                        uint32_t vis = off >= 16   ? 0xFFFFu
                                       : off >= 0  ? ((1u << off) - 1) | (uint32_t)(mask << off)
                                       : off > -64 ? (uint32_t)(mask >> -off)
                                                   : 0u;
                        vis = out >> (k / 16) & 1 ? 0u : vis;
                        float v[16];
                        uint32_t w[16];
                        tmem_ld16(s_at + k, v);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = vis >> i & 1 ? __float_as_uint(v[i]) : 0xFF800000u;
                        tmem_st16(s_at + k, w);
                        tmem_st_wait();
                    }
                // a load takes as long as the work on some 40 columns: two of 32 at a time
                float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                for (int k = 0; k < 128; k += 64) {
                    uint32_t s[2][32];
                    tmem_ld32_begin(s_at + k, s[0]);
                    tmem_ld32_begin(s_at + k + 32, s[1]);
                    tmem_ld32_end(s[0]);
                    tmem_ld32_end(s[1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            top4[i >> 1 & 3] = max3(top4[i >> 1 & 3], __uint_as_float(s[h][i]), __uint_as_float(s[h][i + 1]));
                }
                const float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
                const bool moves = (top - m) * c > MOE_TREE_SLACK;
                if (__any_sync(0xFFFFFFFFu, moves)) {
                    const float f = moves ? ex2((m - top) * c) : 1.0f;
                    m = moves ? top : m;
                    l *= f;
                    if (!fresh)  // S is there, so the last tile's O is too
#pragma unroll 1
                        for (int k = 0; k < 128; k += 16) {
                            float o[16];
                            uint32_t w[16];
                            tmem_ld16(o_at + k, o);
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                w[i] = __float_as_uint(o[i] * f);
                            tmem_st16(o_at + k, w);
                        }
                }
                const float ref = m == -INFINITY ? 0.0f : -m;
                const F2 ref2(ref, ref), c2(c, c), lift2(MOE_TREE_LIFT, MOE_TREE_LIFT);
                F2 sum(0.0f, 0.0f), sum1(0.0f, 0.0f);
#pragma unroll 1
                for (int k = 0; k < 128; k += 64) {
                    uint32_t s[2][32];
                    tmem_ld32_begin(s_at + k, s[0]);
                    tmem_ld32_begin(s_at + k + 32, s[1]);
                    tmem_ld32_end(s[0]);
                    tmem_ld32_end(s[1]);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 32; i += 2) {
                            float e0, e1;
                            fma2(add2(F2(__uint_as_float(s[h][i]), __uint_as_float(s[h][i + 1])), ref2), c2, lift2).get(e0, e1);
                            e0 = ex2(e0);
                            e1 = ex2(e1);
                            F2 &to = i & 2 ? sum1 : sum;
                            to = add2(to, F2(e0, e1));
                            w[i / 2] = pack_h2(e0, e1);
                        }
                        tmem_st16(s_at + k / 2 + 16 * h, w);  // P over the columns that have been read
                    }
                }
                sum = add2(sum, sum1);
                float s0, s1;
                sum.get(s0, s1);
                l += s0 + s1;
                fresh = false;
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_full + x);
            }
            // ---- the item's end. Two M tiles: each group its rows. Else both have the same rows (a lane of tensor
            // memory is the same row in either's O), and each writes half of the dimensions of their sum
            float f0 = 1.0f, f1 = 0.0f;  // factors of this group's O and of the other's
            if (!two) {
                float2 *mine = stat + ((item & 1) * 2) * 128 + row;
                mine[x * 128] = make_float2(m, l);
                soft_sync();
                const float2 other = mine[(x ^ 1) * 128];
                const float up = fmaxf(m, other.x);
                f0 = m == -INFINITY ? 1.0f : ex2((m - up) * c);  // sums of NaN stay
                f1 = other.x == -INFINITY ? 1.0f : ex2((other.x - up) * c);
                l = l * f0 + other.y * f1;
                m = up;
            }
            ok = ok && wait(o_done, item);
            __syncwarp();
            tc_fence_after();
            const bool whole = lo + t == it.lo && lo + end == it.lo + it.units;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            float *part = a.part + ((size_t)blockIdx.x * 2 + (t == 0 ? 0 : 1)) * ROWS * (D + 2);
            uint16_t *to = a.out + (it.first + node) * a.o_tok + (it.head * a.group + (live ? at % a.group : 0)) * a.o_head;
            const bool own = !fresh, others = !two && (end - t > 1 || fresh);  // of one tile only one group has an O
            const int k0 = two ? 0 : x * 64, k1 = two ? 128 : k0 + 64;
#pragma unroll 1
            for (int k = k0; k < k1; k += 16) {
                float o[16];
                if (own) {
                    tmem_ld16(o_at + k, o);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] *= f0;
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = 0.0f;
                }
                if (others) {
                    float v[16];
                    tmem_ld16(lanes + O_COL + (x ^ 1) * 128 + k, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = fmaf(v[i], f1, o[i]);
                }
                if (live && !whole) {
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        reinterpret_cast<float4 *>(part)[(k + i) / 4 * ROWS + local] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                } else if (live) {
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(o[i] * inv, o[i + 1] * inv);
                        w[i / 2] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    if (a.o_wide) {
                        *reinterpret_cast<uint4 *>(to + k) = make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4 *>(to + k + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            to[k + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(o_free);
            if (live && !whole && (two || x == 0)) {
                part[ROWS * D + local] = m * c;  // as an exponent of 2
                part[ROWS * D + ROWS + local] = l;
            }
            if (end == tiles && tid == 0)
                tree_cut<ROWS, MOE_TTC_COST>(a, it, items, lo, run);
            t = end;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        tmem_dealloc(tmem, 512);
}

}  // namespace moe

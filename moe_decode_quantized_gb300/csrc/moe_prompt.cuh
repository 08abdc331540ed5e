// moe_prompt.cuh -- latent attention in expanded form, for prompts, on the
// 5th-generation tensor cores: a CTA takes 256 query rows of one head of a
// sequence, in two M tiles of 128 (of few, 128 rows, one tile), over tiles of 128
// tokens,
//   S = [Q | QR] [K | KR]^T,   O += P V,   P = 2^(c (S - m)),
// in one pass with a running reference m and sum of weights a row.
//
// S, P and O are in tensor memory, a row a lane, so that a row's maximum and sum
// are one thread's; P (bf16) takes its S's place and is the second product's A
// operand from there. One M tile's softmax passes under the other's products.
// Keys and values come by TMA through a ring of eight 16 KB places: K (and the
// part that all heads share) in chunks of 64 dimensions of 128 tokens, V in
// chunks of 64 tokens of all dimensions, read with the dimensions contiguous.
//
// Tokens that not all rows see (of the causal edge, past the sequence's end) may
// hold anything: their scores are taken out, their values that are not finite
// are zeros in the product, and are added at the end to the rows that see them.
//
// Where blocks are few, a cluster of CTAs shares one's tokens; their O, references
// and sums meet in shared memory, each CTA adding up some dimensions, in order.
//
// Bound by products at 128 + 64 dimensions, and by the chain of an M tile's scores,
// their softmax and the product with its weights at 64 + 64 (8192 tokens of 32
// heads, causal: 491 us, 1.40 PFLOP/s, 74 % of the rate that was measured for large
// products; and 430 to 455 us where products are 219). One warp issues all
// products, in the order in which their operands come to be: by two, one an M
// tile, 718 us, and 609 with turns between them. Heads vary fastest over the grid,
// so that the CTAs that run together have rows of one length: with row blocks
// fastest 564 us, where this took 531.
#pragma once
#include "moe_latent.cuh"
#include "moe_tc.cuh"
#include "moe_tree_attn.cuh"
#include "moe_verify.cuh"

namespace moe {

#define MOE_PROMPT_ROWS 256
#define MOE_PROMPT_TOKENS 128
#define MOE_PROMPT_SOFT 8   // softmax warps
#define MOE_PROMPT_THREADS ((MOE_PROMPT_SOFT + 2) * 32)
#define MOE_PROMPT_PLACE 16384
#define MOE_PROMPT_PLACES 8
#define MOE_PROMPT_SPLIT 8     // CTAs that share a block's tokens at most
#define MOE_PROMPT_SLACK 8.0f  // m moves when an exponent passes it by this

struct PromptArgs {
    const uint16_t *q, *v;
    uint16_t *out;
    long long q_tok, q_head, v_tok, v_head, o_tok, o_head;
    const int32_t *q_start, *kv_start;
    int batch, rope, q_tokens, kv_tokens, causal, q_wide, o_wide;
    int one_k, one_v;  // heads share their keys (values)
    int block;         // query rows of a CTA: MOE_PROMPT_ROWS, or half
    int split;         // CTAs (a cluster) that share a block's tokens
    float scale;
    uint32_t *status;
    unsigned long long wait_ns;
    CUtensorMap queries, keys, ropes, values;  // [D + rope, heads, rows], [D, heads, tokens], [rope, tokens], [D, heads, tokens]
};

__device__ uint32_t prompt_unasked;  // the status of calls that ask for none

// tcgen05.mma by a whole warp, one lane of which issues it (see moe_latent_tc.cuh's). Descriptors as the low word, where
// the address is, and the high one, which stays.
__device__ __forceinline__ void mma1_f16(uint32_t tmem_d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 a, b;\n mov.b64 a, {%1, %3};\n mov.b64 b, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
        " elect.sync _|e, 0xFFFFFFFF;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n}\n" ::"r"(tmem_d),
        "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

__device__ __forceinline__ void mma1_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint32_t b_lo, uint32_t hi, uint32_t idesc, bool accumulate)
{
    asm volatile(
        "{\n .reg .pred p, e;\n .reg .b64 b;\n mov.b64 b, {%2, %3};\n setp.ne.b32 p, %5, 0;\n"
        " elect.sync _|e, 0xFFFFFFFF;\n @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n}\n" ::"r"(tmem_d),
        "r"(tmem_a), "r"(b_lo), "r"(hi), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

__device__ __forceinline__ void mma1_commit(uint64_t *bar)
{
    asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xFFFFFFFF;\n"
                 " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
                 : "memory");
}

// block `at` of the call's row blocks, those of the sequences that hold, in order; q1 <= q0: there is no such block
struct PromptBlock {
    int q0, q1, row, k0, t, n;  // query rows [q0, q1) of the call, the first's place in the sequence; tokens [k0, k0 + t)
};

// whether a sequence's own starts hold
__device__ __forceinline__ bool prompt_held(const PromptArgs &a, int b)
{
    const int q0 = a.q_start[b], q1 = a.q_start[b + 1], k0 = a.kv_start[b], k1 = a.kv_start[b + 1];
    return q0 >= 0 && q1 >= q0 && q1 <= a.q_tokens && k0 >= 0 && k1 >= k0 && k1 <= a.kv_tokens;
}

// Where not all starts hold (rarely: out of line). By the whole CTA: of the sequences whose own starts hold, those that
// begin before an earlier one do not hold either, so that no row is two sequences'; the sequences that hold as bits [32];
// and zeros in the rows of the others that none of these has, those of this CTA's share.
template <int D>
static __device__ __noinline__ void prompt_sort_out(const PromptArgs &a, uint32_t *held, int head, bool clears)
{
    const int tid = threadIdx.x, lane = tid & 31;
    for (int b = tid; b < 1024; b += MOE_PROMPT_THREADS) {  // (whole warps)
        bool ok = b < a.batch && prompt_held(a, b);
        for (int i = 0; i < b && ok; ++i)
            ok = a.q_start[i] <= a.q_start[b];
        const uint32_t bits = __ballot_sync(0xFFFFFFFFu, ok);
        if (lane == 0)
            held[b >> 5] = bits;
    }
    __syncthreads();
    constexpr int WARPS = MOE_PROMPT_THREADS / 32;
    for (int r = blockIdx.y * WARPS + (tid >> 5); clears && r < a.q_tokens; r += gridDim.y * WARPS) {
        bool other = false, own = false;
        for (int b = lane; b < a.batch; b += 32)
            if (a.q_start[b] <= r && r < a.q_start[b + 1])
                (held[b >> 5] >> (b & 31) & 1 ? own : other) = true;
        if (__any_sync(0xFFFFFFFFu, other) && !__any_sync(0xFFFFFFFFu, own))
            for (int d = lane; d < D; d += 32)
                a.out[(long long)r * a.o_tok + head * a.o_head + d] = 0;
    }
}

// whole CTA: found [3], scan [33] and held [32] in shared memory; clears: whether it takes part in prompt_sort_out's zeros
template <int D>
__device__ __forceinline__ PromptBlock prompt_block(const PromptArgs &a, int at, int *scan, int *found, uint32_t *held,
                                                    uint32_t *status, int head, bool clears)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = MOE_PROMPT_THREADS;
    if (tid == 0)
        found[0] = -1;
    const int per = (a.batch + nt - 1) / nt;
    int mine = 0;
    bool odd = false;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= a.batch)
            break;
        if (prompt_held(a, b))
            mine += (a.q_start[b + 1] - a.q_start[b] + a.block - 1) / a.block;
        else
            odd = true;
    }
    const bool all = !__syncthreads_or(odd);  // (then the starts do not fall)
    auto holds = [&](int b) { return all || (held[b >> 5] >> (b & 31) & 1); };
    if (!all) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0)
            atomicOr(status, (uint32_t)MOE_WS_INDEX);
        prompt_sort_out<D>(a, held, head, clears);
        mine = 0;
        for (int b = tid * per; b < min(tid * per + per, a.batch); ++b)
            mine += holds(b) ? (a.q_start[b + 1] - a.q_start[b] + a.block - 1) / a.block : 0;
    }
    int incl = mine;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, m);
        incl += lane >= m ? u : 0;
    }
    if (lane == 31)
        scan[warp] = incl;
    __syncthreads();
    int before = incl - mine;
    for (int w = 0; w < warp; ++w)
        before += scan[w];
    if (at >= before && at < before + mine)
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b >= a.batch)
                break;
            const int q0 = a.q_start[b], q1 = a.q_start[b + 1], blocks = holds(b) ? (q1 - q0 + a.block - 1) / a.block : 0;
            if (at < before + blocks) {
                found[0] = b;
                found[1] = q0 + (at - before) * a.block;
                found[2] = q1;
                break;
            }
            before += blocks;
        }
    __syncthreads();
    PromptBlock r{};
    const int b = found[0];
    if (b < 0)
        return r;
    r.k0 = a.kv_start[b];
    r.t = a.kv_start[b + 1] - r.k0;
    r.n = found[2] - a.q_start[b];
    r.q0 = found[1];
    r.q1 = min(found[1] + a.block, found[2]);
    r.row = r.q0 - a.q_start[b];
    return r;
}

// 32 bytes, a sector, at once
__device__ __forceinline__ void put8(uint16_t *p, const uint32_t (&w)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// adds the values that are not finite, of the noted tokens that a row sees (the first `most`), to 16 dimensions from k on
// (rarely needed: out of line)
static __device__ __noinline__ void prompt_add(const PromptArgs &a, float (&o)[16], const uint32_t *bad, int edge, int most, int k0,
                                               int head, int k)
{
    for (int w = 0; w < 12; ++w)
        for (uint32_t set = *reinterpret_cast<const volatile uint32_t *>(bad + w); set; set &= set - 1) {
            const int token = (edge + w / 4) * MOE_PROMPT_TOKENS + (w & 3) * 32 + __ffs(set) - 1;
            if (token >= most)
                continue;
            const uint16_t *v = a.v + (long long)(k0 + token) * a.v_tok + head * a.v_head + k;
            for (int i = 0; i < 16; ++i)
                if ((v[i] & 0x7F80u) == 0x7F80u)
                    o[i] += bf16_to_f32(v[i]);
        }
}

// 16 dimensions of an output row
__device__ __forceinline__ void prompt_put(uint16_t *to, const float (&o)[16], float by, int o_wide)
{
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 16; i += 2)
        w[i / 2] = pack_bf2(o[i] * by, o[i + 1] * by);
    if (o_wide == 2) {
        put8(to, w);
    } else {
        latent_put(to, make_uint4(w[0], w[1], w[2], w[3]), o_wide);
        latent_put(to + 8, make_uint4(w[4], w[5], w[6], w[7]), o_wide);
    }
}

// a part's share of a sum: what is not finite stays, whatever its weight
__device__ __forceinline__ float prompt_part(float o, float by)
{
    return by > 0.0f || fabsf(o) <= 3.402823466e38f ? o * by : o;
}

// shared memory of CTA `of` of the cluster, at the place of p
__device__ __forceinline__ float4 peer_get4(const void *p, int of)
{
    float4 v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %4, %5;\n ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(smem_u32(p)), "r"(of)
                 : "memory");
    return v;
}

__device__ __forceinline__ float2 peer_get2(const void *p, int of)
{
    float2 v;
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %2, %3;\n ld.shared::cluster.v2.f32 {%0, %1}, [a];\n}\n"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(smem_u32(p)), "r"(of)
                 : "memory");
    return v;
}

template <int D>
__global__ void __launch_bounds__(MOE_PROMPT_THREADS, 1) moe_prompt_kernel(const __grid_constant__ PromptArgs a)
{
    constexpr int KC = D / 64 + 1;   // places of a tile's K
    constexpr int VC = D / 64;       // and of its V: VT tokens each
    constexpr int VT = MOE_PROMPT_TOKENS / VC;
    constexpr uint32_t S_COL = 0, O_COL = 256;  // of tensor memory: S (and P) of the M tiles, O of the two
    constexpr int TOKENS = MOE_PROMPT_TOKENS, PLACE = MOE_PROMPT_PLACE, Q_TILE = KC * PLACE;
    extern __shared__ __align__(1024) uint8_t smem_prompt[];
    uint8_t *sq = smem_prompt, *ring = smem_prompt + 2 * Q_TILE, *small = ring + MOE_PROMPT_PLACES * PLACE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(small);
    uint64_t *k_full = bars, *v_full = bars + 2, *k_free = bars + 4, *v_free = bars + 6;  // [2], by tiles
    uint64_t *s_full = bars + 8, *p_full = bars + 10, *o_full = bars + 12;                // [2], by M tile
    uint64_t *v_edge = bars + 14, *v_clean = bars + 17;  // [3] values of the tiles that are looked through: there, and fit
    uint64_t *q_full = bars + 20, *drained = bars + 21;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 22);
    uint32_t *bad = tmem_slot + 1;  // [3][4] tokens of the tiles that are looked through with values that are not finite
    int *scan = reinterpret_cast<int *>(bad + 12), *found = scan + 33;
    uint32_t *held = reinterpret_cast<uint32_t *>(found + 3);  // [32]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, split = a.split;
    const int head = blockIdx.x / split, part = blockIdx.x - head * split;  // (split CTAs are a cluster)
    uint32_t *status = a.status ? a.status : &prompt_unasked;

    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(k_full + x, 1);
            mbar_init(v_full + x, 1);
            mbar_init(k_free + x, 1);
            mbar_init(v_free + x, 1);
            mbar_init(s_full + x, 1);
            mbar_init(p_full + x, MOE_PROMPT_SOFT / 2);
            mbar_init(o_full + x, 1);
        }
        for (int i = 0; i < 3; ++i)
            mbar_init(v_edge + i, 1);
        mbar_init(q_full, a.q_wide ? 1 : MOE_PROMPT_SOFT);
        mbar_init(drained, 1);
        fence_barrier_init();
    }
    if (tid < 12)
        bad[tid] = 0;
    pdl_wait();  // before tensor memory is taken: the last kernel may still need it
    // (the last blocks first: a sequence's later rows see more)
    PromptBlock b = prompt_block<D>(a, gridDim.y - 1 - blockIdx.y, scan, found, held, status, head, part == 0);
    if (b.q1 <= b.q0)
        return;
    const int rows = b.q1 - b.q0;
    // tokens that row i of the block sees, of this CTA's part of them
    int from = 0, len = b.t;
    auto sees = [&](int i) { return max(0, min(len, (a.causal ? min(b.t, b.t - b.n + b.row + i + 1) : b.t) - from)); };
    if (split > 1) {
        const int all = (sees(rows - 1) + TOKENS - 1) / TOKENS, end = all * (part + 1) / split;
        const int begin = all * part / split * TOKENS;
        len = max(0, min(b.t, end * TOKENS) - begin);
        from = begin;
    }
    b.k0 += from;
    // tiles of each M tile, and the first that not all rows see whole
    const int tiles0 = (sees(min(rows, 128) - 1) + TOKENS - 1) / TOKENS, tiles1 = rows > 128 ? (sees(rows - 1) + TOKENS - 1) / TOKENS : 0;
    const int tiles = max(tiles0, tiles1), edge = sees(0) / TOKENS;
    if (tid == 0) {
        for (int i = 0; i < 3; ++i)  // the warps of the M tiles that the tile is for
            mbar_init(v_clean + i, max(1, (edge + i < tiles0 ? MOE_PROMPT_SOFT / 2 : 0) + (edge + i < tiles1 ? MOE_PROMPT_SOFT / 2 : 0)));
        fence_barrier_init();
    }
    if (warp == 0)
        tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_launch_dependents();
    // (a poll that does not hold the warp first: 15 clocks where the phase is complete, one that may 69; and the clock,
    // which takes longer than most waits, last)
    auto wait = [&](uint64_t *bar, int phase) {
        return mbar_try_wait(bar, (uint32_t)phase & 1u) || tree_poll(bar, (uint32_t)phase & 1u) ||
               tree_wait_on(bar, (uint32_t)phase & 1u, status, a.wait_ns);
    };
    auto drain = [&](uint64_t *bar, int phase) { tree_wait_on(bar, (uint32_t)phase & 1u, status, max(a.wait_ns, MOE_TREE_DRAIN_NS)); };
    auto get_o = [&](float (&o)[16], uint32_t at, int n) {
        if (n > 0) {
            tmem_ld16(at, o);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                o[i] = 0.0f;
        }
    };
    auto place = [&](int i) { return ring + (i & (MOE_PROMPT_PLACES - 1)) * PLACE; };

    float m_end = -INFINITY, l_end = 0.0f;
    if (warp < MOE_PROMPT_SOFT && tiles > 0 && !a.q_wide) {
        // ---------------- queries that TMA does not take
        constexpr int PIECES = D / 8 + 8;
        for (int i = tid; i < rows * PIECES; i += MOE_PROMPT_SOFT * 32) {
            const int r = i / PIECES, k = i % PIECES;
            *reinterpret_cast<uint4 *>(sq + (r >> 7) * Q_TILE + (k >> 3) * PLACE + (r & 127) * 128 + (((k & 7) ^ (r & 7)) << 4)) =
                k < D / 8 + a.rope / 8 ? latent_get(a.q + (long long)(b.q0 + r) * a.q_tok + head * a.q_head + k * 8, false)
                                       : make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0)
            mbar_arrive(q_full);
    }

    if (warp == MOE_PROMPT_SOFT) {
        // ---------------- the copies: K of tile u once V of tile u - 2 is done with, V of it once K of tile u - 1 is
        if (lane == 0) {
            bool ok = true;
            int u = 0, half = 0;  // half: K of tile u has been asked for
            if (a.q_wide && tiles > 0) {
                const int m = rows > 128 ? 2 : 1;
                mbar_arrive_expect_tx(q_full, m * Q_TILE);
                for (int i = 0; i < m * KC; ++i)
                    tma_load_3d(sq + i * PLACE, &a.queries, i % KC * 64, head, b.q0 + i / KC * 128, q_full);
            }
            for (; u < tiles; ++u) {
                const int x = u & 1, at = u * (KC + VC), token = b.k0 + u * TOKENS;
                half = 0;
                ok = u < 2 || wait(v_free + x, (u >> 1) - 1);
                if (!ok)
                    break;
                mbar_arrive_expect_tx(k_full + x, KC * PLACE);
#pragma unroll
                for (int d = 0; d < D / 64; ++d)
                    tma_load_3d(place(at + d), &a.keys, d * 64, a.one_k ? 0 : head, token, k_full + x);
                tma_load_2d(place(at + D / 64), &a.ropes, 0, token, k_full + x);
                half = 1;
                ok = u < 1 || wait(k_free + (x ^ 1), (u - 1) >> 1);
                if (!ok)
                    break;
                uint64_t *v_bar = u < edge ? v_full + x : v_edge + (u - edge);
                mbar_arrive_expect_tx(v_bar, VC * PLACE);
#pragma unroll
                for (int i = 0; i < VC; ++i)
#pragma unroll
                    for (int d = 0; d < D / 64; ++d)
                        tma_load_3d(place(at + KC + i) + d * VT * 128, &a.values, d * 64, a.one_v ? 0 : head, token + i * VT, v_bar);
            }
            // nothing in flight when the CTA ends
            if (a.q_wide && tiles > 0)
                drain(q_full, 0);
            for (int k = max(0, u - 2); k < u; ++k) {
                drain(k_full + (k & 1), k >> 1);
                drain(k < edge ? v_full + (k & 1) : v_edge + (k - edge), k < edge ? k >> 1 : 0);
            }
            if (!ok && half)
                drain(k_full + (u & 1), u >> 1);
        }
    } else if (warp == MOE_PROMPT_SOFT + 1) {
        // ---------------- the products, in order: for each M tile in turn, O with the last tile's P, then S of this one in
        // P's place, so that one's products pass under the other's softmax
        constexpr uint32_t id_s = mma_idesc(128, TOKENS, true), id_o = mma_idesc(128, D, true) | (1u << 16);
        const uint32_t tm = __reduce_max_sync(0xFFFFFFFFu, tmem);  // (what the loops need is the same in all lanes)
        const int n = __reduce_max_sync(0xFFFFFFFFu, tiles), n0 = __reduce_max_sync(0xFFFFFFFFu, tiles0),
                  n1 = __reduce_max_sync(0xFFFFFFFFu, tiles1), e = __reduce_max_sync(0xFFFFFFFFu, edge);
        const uint64_t desc = sw128_desc(ring);
        const uint32_t hi = (uint32_t)(desc >> 32), kd = (uint32_t)desc, qd = (uint32_t)sw128_desc(sq);
        // V: rows (one a token) of 64 dimensions, 8 rows 1024 bytes apart, the next 64 dimensions VT rows
        const uint32_t vd = kd & ~(0x3FFFu << 16) | (uint32_t)(VT * 128 / 16) << 16;
        auto all = [&](bool v) { return __all_sync(0xFFFFFFFFu, v) != 0; };
        auto off = [&](int i) { return (uint32_t)((i & (MOE_PROMPT_PLACES - 1)) * PLACE) / 16; };
        bool ok = n == 0 || all(wait(q_full, 0));
        for (int u = 0; u <= n && ok && n > 0; ++u) {
            const int x = u & 1;
            ok = u == 0 || all(u - 1 < e ? wait(v_full + (x ^ 1), (u - 1) >> 1) : wait(v_clean + (u - 1 - e), 0));
            bool keys = false;
#pragma unroll 1
            for (int g = 0; g < 2 && ok; ++g) {
                const int last = g ? n1 : n0;
                int at = u * (KC + VC);
                asm volatile("" : "+r"(at));  // (addresses are made as the products go: ahead of them all, they hold them up)
                if (u > 0 && u <= last) {
                    ok = all(wait(p_full + g, u - 1));
                    if (!ok)
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int k = 0; k < 8; ++k)  // 16 tokens: 8 columns of P, 2048 bytes of V
                        mma1_f16_ts(tm + O_COL + g * 128, tm + S_COL + g * 128 + k * 8,
                                    vd + off(at - VC + k * 16 / VT) + (uint32_t)(k * 16 % VT * 128) / 16, hi, id_o,
                                    u > 1 || k > 0);
                    if (u == last)
                        mma1_commit(o_full + g);
                    if (g || u > n1)  // the last M tile's: before S's products, so that the copies wait no longer
                        mma1_commit(v_free + (x ^ 1));
                }
                if (u < last) {
                    if (!keys) {
                        ok = all(wait(k_full + x, u >> 1));
                        if (!ok)
                            break;
                        tc_fence_after();
                        keys = true;
                    }
#pragma unroll
                    for (int d = 0; d < KC; ++d)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma1_f16(tm + S_COL + g * 128, qd + (uint32_t)(g * Q_TILE + d * PLACE + k * 32) / 16,
                                     kd + off(at + d) + k * 2, hi, id_s, d + k > 0);
                    mma1_commit(s_full + g);
                }
            }
            if (u < n)
                mma1_commit(k_free + x);
        }
        if (n > 0) {  // what has been issued ends before tensor and shared memory are given back
            mma1_commit(drained);
            drain(drained, 0);
        }
    } else {
        // ---------------- softmax: M tile g, row `row` of it
        const int g = warp >> 2, row = (warp & 3) * 32 + lane, mine = g * 128 + row, n = g ? tiles1 : tiles0;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t s_at = lanes + S_COL + g * 128, o_at = lanes + O_COL + g * 128;
        const bool live = mine < rows;
        const int most = live ? sees(mine) : 0;
        const float scaled = fminf(fabsf(a.scale) * 1.4426950408889634f, 3.0e38f);
        const bool flat = scaled == 0.0f;  // all scores alike
        const float c = flat ? 1.0f : scaled, turn = flat ? 0.0f : a.scale < 0.0f ? -1.0f : 1.0f;
        float m = -INFINITY, l = 0.0f;
        bool ok = true;
        for (int u = 0; u < n; ++u) {
            if (u >= edge) {
                // values of a tile that not all rows see: those past the end zeros, those that are not finite zeros and
                // noted; each M tile that the tile is for looks through its part
                ok = ok && wait(v_edge + (u - edge), 0);
                __syncwarp();
                const int at = u * (KC + VC) + KC, other = g ? tiles0 : tiles1, step = u < other ? 256 : 128;
#pragma unroll 2
                for (int i = u < other ? tid : tid & 127; i < TOKENS * D / 8; i += step) {
                    const int token = i / (D / 8), piece = i % (D / 8);
                    uint4 *p = reinterpret_cast<uint4 *>(place(at + token / VT) + (piece >> 3) * VT * 128 + token % VT * 128 + (piece & 7) * 16);
                    const uint4 v = *p, w = u * TOKENS + token >= len ? make_uint4(0, 0, 0, 0)
                                                                      : make_uint4(finite_bf2(v.x), finite_bf2(v.y), finite_bf2(v.z), finite_bf2(v.w));
                    if (v.x != w.x || v.y != w.y || v.z != w.z || v.w != w.w) {
                        *p = w;
                        if (u * TOKENS + token < len)
                            atomicOr(bad + (u - edge) * 4 + (token >> 5), 1u << (token & 31));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(v_clean + (u - edge));
            }
            ok = ok && wait(s_full + g, u);
            __syncwarp();
            tc_fence_after();
            if (u >= edge || turn != 1.0f) {  // the scores of tokens that are not seen to -inf, so that the passes below stay short
                const int vis = most - u * TOKENS;
#pragma unroll 1
                for (int k = 0; k < TOKENS; k += 16) {
                    float v[16];
                    uint32_t w[16];
                    tmem_ld16(s_at + k, v);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        w[i] = k + i < vis ? __float_as_uint(v[i] * turn) : 0xFF800000u;
                    tmem_st16(s_at + k, w);
                    tmem_st_wait();
                }
            }
            float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
            for (int k = 0; k < TOKENS; k += 64) {
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
            const bool moves = live && (top - m) * c > MOE_PROMPT_SLACK;  // (rows that are none hold anything)
            if (__any_sync(0xFFFFFFFFu, moves)) {
                const float f = moves ? ex2((m - top) * c) : 1.0f;
                m = moves ? top : m;
                l *= f;
                if (u > 0)  // S is there, so the last tile's O is too
#pragma unroll 1
                    for (int k = 0; k < D; k += 16) {
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
            const F2 ref2(ref, ref), c2(c, c);
            F2 sum(0.0f, 0.0f), sum1(0.0f, 0.0f);
#pragma unroll 1
            for (int k = 0; k < TOKENS; k += 64) {
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
                        mul2(add2(F2(__uint_as_float(s[h][i]), __uint_as_float(s[h][i + 1])), ref2), c2).get(e0, e1);
                        // (bf16, by 2^-8 at most: the tensor core takes P only in the type of the values beside it)
                        const uint32_t p = pack_bf2(ex2(e0), ex2(e1));
                        F2 &to = i & 2 ? sum1 : sum;
                        to = add2(to, F2(bf16_lo(p), bf16_hi(p)));  // as rounded
                        w[i / 2] = p;
                    }
                    tmem_st16(s_at + k / 2 + 16 * h, w);  // P over the columns that have been read
                }
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(p_full + g);
            sum = add2(sum, sum1);
            float l0, l1;
            sum.get(l0, l1);
            l += l0 + l1;
        }
        // ---- the end
        if (n > 0)
            ok = ok && wait(o_full + g, 0);
        __syncwarp();
        tc_fence_after();
        m_end = m;
        l_end = l;
        if (split == 1) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint16_t *to = a.out + (long long)(b.q0 + mine) * a.o_tok + head * a.o_head;
            uint32_t any = 0;  // values that are not finite
            for (int w = 0; w < 12; ++w)
                any |= *reinterpret_cast<volatile uint32_t *>(bad + w);
#pragma unroll 1
            for (int k = 0; k < D && mine - lane < rows; k += 16) {
                float o[16];
                get_o(o, o_at + k, n);
                if (any)
                    prompt_add(a, o, bad, edge, most, b.k0, head, k);
                if (live)
                    prompt_put(to + k, o, inv, a.o_wide);
            }
        }
    }
    if (split > 1) {
        // ---------------- the parts of a block joined: each CTA's O, references and sums into its shared memory, where
        // products and copies have ended; then each CTA some dimensions of all rows, the parts in order
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        float4 *kept = reinterpret_cast<float4 *>(smem_prompt);  // [D / 4][256]
        float2 *ends = reinterpret_cast<float2 *>(smem_prompt + 256 * D * 4);
        const int row = tid & 255;
        const bool live = warp < MOE_PROMPT_SOFT && row < rows;
        if (warp < MOE_PROMPT_SOFT && row - lane < rows) {
            const int g = warp >> 2, n = g ? tiles1 : tiles0, most = live ? sees(row) : 0;
            const uint32_t o_at = tmem + ((uint32_t)((warp & 3) * 32) << 16) + O_COL + g * 128;
            uint32_t any = 0;
            for (int w = 0; w < 12; ++w)
                any |= *reinterpret_cast<volatile uint32_t *>(bad + w);
#pragma unroll 1
            for (int k = 0; k < D; k += 16) {
                float o[16];
                get_o(o, o_at + k, n);
                if (any)
                    prompt_add(a, o, bad, edge, most, b.k0, head, k);
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    kept[(k + i) / 4 * 256 + row] = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
            ends[row] = make_float2(m_end, l_end);
        }
        __syncwarp();
        cluster_sync();
        if (live) {
            const float scaled = fminf(fabsf(a.scale) * 1.4426950408889634f, 3.0e38f), c = scaled == 0.0f ? 1.0f : scaled;
            float m = -INFINITY, l = 0.0f, by[MOE_PROMPT_SPLIT];
#pragma unroll
            for (int i = 0; i < MOE_PROMPT_SPLIT; ++i)
                if (i < split)
                    m = fmaxf(m, peer_get2(ends + row, i).x);
#pragma unroll
            for (int i = 0; i < MOE_PROMPT_SPLIT; ++i)
                if (i < split) {
                    const float2 e = peer_get2(ends + row, i);
                    by[i] = e.x == -INFINITY ? 1.0f : ex2((e.x - m) * c);  // a NaN sum stays
                    l += e.y * by[i];
                }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint16_t *to = a.out + (long long)(b.q0 + row) * a.o_tok + head * a.o_head;
#pragma unroll 1
            for (int k = D / split * part; k < D / split * (part + 1); k += 16) {
                float o[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    o[i] = 0.0f;
#pragma unroll
                for (int x = 0; x < MOE_PROMPT_SPLIT; ++x)
                    if (x < split)
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            const float4 v = peer_get4(kept + (k + i) / 4 * 256 + row, x);
                            o[i] += prompt_part(v.x, by[x]);
                            o[i + 1] += prompt_part(v.y, by[x]);
                            o[i + 2] += prompt_part(v.z, by[x]);
                            o[i + 3] += prompt_part(v.w, by[x]);
                        }
                prompt_put(to + k, o, inv, a.o_wide);
            }
        }
        __syncwarp();
        cluster_sync();  // (no CTA's shared memory goes while it is read)
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        tmem_dealloc(tmem, 512);
}

}  // namespace moe

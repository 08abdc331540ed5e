// moe_tree_attn.cuh -- attention of the drafted tokens of each sequence (one
// token, a chain, or a tree) over the quantised paged cache.
//
//   o = sum_j softmax_j(scale q . K_j | j seen) V_j
// in one pass over the cache: a running reference m of each row's scores, the
// sum l of its weights and o, both scaled by 2^(m - m') when m moves.
//
// The rows of one kv head are its query rows times the heads of its group,
// row r = token r / G, head r % G; 16 MT of them (a row block) are worked on
// together. An item is (sequence, kv head, row block), a unit of it one block
// of 16 tokens of the cache. The units of all items form one list that is cut
// into runs of equal cost, one a CTA, so ragged lengths cost nothing; a run that cuts
// an item leaves a partial (o, m, l) in the workspace, and a second kernel,
// launched behind the first so that it starts the moment that one ends, joins
// the partials of each cut item in a fixed order.
//
// A warp takes every fourth unit of its CTA's run through a ring of its own
// (one bulk copy a unit), and everything stays in registers: codes to f16 B
// fragments (the cache's byte order is the fragments'), S = Q K^T by 16x8x16
// products, the weights as the A fragments of o += P V. 16 rows cost 32 such
// products a unit of 128 dimensions, and 598 TFLOP/s of them were measured:
// bound by the copies while the rows are few (64 sequences of 4000 to 24000
// tokens, one row of 4 heads: 264 us, 97 % of the copy rate), by the turning of
// codes and the products from some 16 rows on (64 of 12000, 32 rows: 386 us, 65
// %) and, in 4 bits, from the first (the former case 339 us, 45 % of the rate), by
// latency for short contexts (one sequence of 511 tokens: 11.7 us).
#pragma once
#include "moe_kv.cuh"

namespace moe {

#define MOE_TREE_WARPS 4
#define MOE_TREE_THREADS (MOE_TREE_WARPS * 32)
#define MOE_TREE_MAX_LEN 0x7FFFFF00   // tokens of a sequence: whole tiles past them end below 2^31
#define MOE_TREE_DRAIN_NS 1000000ull  // a wait for what is in flight after another wait ran out: at least this long
#define MOE_TREE_COST 24  // of an item, beside its units
// the weights are 2^(s - m + 7): m moves when a score passes it by 8, so a
// weight stays below 2^15, and f16 holds weights of 2^-31 of the largest
#define MOE_TREE_SLACK 8.0f
#define MOE_TREE_LIFT 7.0f

// an item that more than one run works on: its query rows, and the runs after
// the one it starts in (0: there is no such item)
struct TreeCut {
    int first, n, head, block, runs, whole_run;  // whole_run: it begins where its first run does
};

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
    int max_len;              // tokens that a sequence can have
    const unsigned long long *mask;  // [tokens] or NULL: causal
    int batch, tokens, group;
    float scale;
    int q_wide, o_wide;       // rows of q (out) can be read (written) 16 bytes at a time
    int min_units;            // fewest units of a run
    uint32_t *ctrl;
    TreeCut *cuts;     // [grid] the item that starts in the run and leaves it
    float *part;              // [grid][2] partials: [head size / 4][rows][4], then the rows' references, then sums
    float join_c;             // what turns differences of the references into exponents of 2
    unsigned long long wait_ns;
};

// geometry of an instance: FMT, head size, 16-row tiles
template <int FMT, int D, int MT>
struct TreeShape {
    static constexpr int RB = FMT == MOE_KV_Q8 ? D : D / 2;
    static constexpr int GR = D / MOE_KV_GROUP;
    static constexpr int SCALES = 16 * GR * (FMT == MOE_KV_Q8 ? 2 : 4);
    static constexpr int HALF = 16 * RB + SCALES;
    static constexpr int BLOCK = 2 * HALF;
    static constexpr int KS = D / 16;       // steps of the contraction over the dimensions
    static constexpr int NB = D / 8;        // column blocks of the output
    static constexpr int WK = RB / 16;      // words of a lane's quarter of a K row
    static constexpr int WV = RB / 32;      // words of a lane's eighth of a V row
    static constexpr int ROWS = 16 * MT;
    static constexpr int OREGS = MT * NB * 4;
    // CTAs an SM, by registers (heads of 64 with two and four tiles spill 44 and 28 bytes a thread within them)
    static constexpr int CTAS = OREGS <= 32 ? 4 : OREGS <= 64 ? 3 : 2;
    static constexpr bool QREG = OREGS + MT * KS * 4 <= 96;  // query fragments kept in registers
    static constexpr int PART = ROWS * D + 2 * ROWS;         // floats of a partial
    static constexpr int BARS = 8 * 8 * MOE_TREE_WARPS;      // room for 8 stages' barriers
    static constexpr int HEAD = BARS + 8 * ROWS + 12 * ROWS * MOE_TREE_WARPS + 64;
    static constexpr int QBYTES = MT * KS * 512;
    static constexpr int MERGE = 2 * OREGS * 128;
    static constexpr int FIXED = (HEAD + QBYTES + MERGE + 127) / 128 * 128;  // then the ring, then the list
};

// D (+)= A B: 16x8x16, f16 operands, f32 sums
__device__ __forceinline__ void mma16816(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
__device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }
__device__ __forceinline__ uint32_t pack_h2(float a, float b) { return h2(__floats2half2_rn(a, b)); }
__device__ __forceinline__ uint32_t dup_lo(uint32_t v) { return __byte_perm(v, v, 0x1010); }
__device__ __forceinline__ uint32_t dup_hi(uint32_t v) { return __byte_perm(v, v, 0x3232); }

// mbar_wait for waits that are short and many: each poll lets the hardware
// hold the warp until the phase completes (10 us at most), so that waiting
// warps leave the issue slots to those that work; the clock that bounds the
// wait is read only after the first poll that fails; what follows the first
// poll is out of line.
__device__ __forceinline__ bool tree_poll(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(10000u)
        : "memory");
    return ok != 0;
}

static __device__ __noinline__ bool tree_wait_on(uint64_t *bar, uint32_t parity, uint32_t *status, unsigned long long wait_ns)
{
    const uint64_t t0 = globaltimer();
    do {
        if (tree_poll(bar, parity))
            return true;
    } while (globaltimer() - t0 <= wait_ns);
    atomicOr(status, (uint32_t)MOE_WS_TIMEOUT);
    return false;
}

__device__ __forceinline__ bool tree_wait(uint64_t *bar, uint32_t parity, uint32_t *status, unsigned long long wait_ns)
{
    return tree_poll(bar, parity) || tree_wait_on(bar, parity, status, wait_ns);
}

// two code bytes (bytes i and j of w) as f16: 0x6400 | u is 1024 + u, less
// 1024 + 128 the code, exactly; times the scale, rounded once
__device__ __forceinline__ uint32_t q8_pair(uint32_t w, uint32_t sel, __half2 d)
{
    const __half2 u = h2(__byte_perm(w, 0x64646464u, sel));
    return h2(__hmul2(__hsub2(u, h2(0x64806480u)), d));
}

// two 4-bit codes at bits 0 and 16 of w (already 0x6400 | code) as code d + m
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, __half2 d, __half2 m)
{
    return h2(__hfma2(__hsub2(h2(w), h2(0x64006400u)), d, m));
}

// rows and length of a sequence, checked; n = 0 where they do not hold (rows:
// the query rows that are then written as zeros)
__device__ __forceinline__ void tree_sequence(const TreeArgs &a, int b, int &first, int &n, int &len, int &rows)
{
    first = a.q_start[b];
    n = a.q_start[b + 1] - first;
    len = a.kv_len[b];
    const bool held = first >= 0 && n >= 0 && n <= MOE_MAX_DRAFT && first <= a.tokens - n;
    rows = held ? n : 0;
    if (!held || len < n || len > a.max_len) {
        if (!held || n > 0)
            atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_INDEX);
        n = 0;
    }
}

// (out of line: it is rarely needed, and the kernels' roles share the instruction cache)
static __device__ __noinline__ long long tree_div_long(long long x, long long y) { return x / y; }

// x / y (x >= 0, y > 0), by a 32-bit division where both fit
__device__ __forceinline__ long long tree_div(long long x, long long y)
{
    if ((unsigned long long)(x | y) >> 32 == 0)
        return (uint32_t)x / (uint32_t)y;
    return tree_div_long(x, y);
}

// the largest of three (a NaN counts for nothing)
__device__ __forceinline__ float max3(float x, float y, float z)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// zeros for the query rows of a sequence that does not hold
template <int D>
__device__ __forceinline__ void tree_zero(const TreeArgs &a, int first, int rows)
{
    const int heads = a.k.heads * a.group;
    for (int r = 0; r < rows * heads; ++r) {
        uint16_t *p = a.out + (first + r / heads) * a.o_tok + r % heads * a.o_head;
        for (int d = 0; d < D; ++d)
            p[d] = 0;
    }
}

// The list is cut by cost: an item costs its units and COST more (its queries
// are brought, its warps joined), so that no CTA gets many short items (8
// sequences of 8000, one without a context, up to 20 rows a head: 68 us without,
// 43, 37, 37, 37 with a cost of 8, 16, 24, 32; 64 sequences of 1 to 300 tokens 48
// and 21 us; 64 of 4000 to 24000 270 without, 264 with 24, 266 with 32; the
// tensor-core kernel's tiles of 128 tokens, 64 trees of up to 16 rows over 1 to
// 2000: 110 us without, 97 with 2, 98 with 6). cum [batch + 1] and items [batch + 1] are the units and the items before each
// sequence; a place in the list of costs is turned into a unit by tree_place.

// one item: the units [lo, lo + units) of the list
struct TreeItem {
    int b, head, block, first, n, len, units;
    long long lo;
};

template <int ROWS>
__device__ __forceinline__ int tree_blocks(int n, int group) { return (n * group + ROWS - 1) / ROWS; }

// the item that holds unit u: cum [batch + 1] is the list's units before each sequence
// of TOKENS tokens
template <int ROWS, int TOKENS>
__device__ __forceinline__ TreeItem tree_item(const TreeArgs &a, const long long *cum, long long u)
{
    int x = 0, y = a.batch;  // cum[x] <= u < cum[y]
    while (y - x > 1) {
        const int z = (x + y) / 2;
        if (cum[z] <= u)
            x = z;
        else
            y = z;
    }
    TreeItem it;
    it.b = x;
    it.first = a.q_start[x];
    it.n = a.q_start[x + 1] - it.first;
    it.len = a.kv_len[x];
    it.units = (it.len + TOKENS - 1) / TOKENS;
    const int at = (int)tree_div(u - cum[x], it.units), blocks = tree_blocks<ROWS>(it.n, a.group);
    it.head = at / blocks;
    it.block = at % blocks;
    it.lo = cum[x] + (long long)at * it.units;
    return it;
}

// the first unit at or after place w of the list of costs (an item's units come before the rest of its cost)
template <int ROWS, int TOKENS, int COST>
__device__ __forceinline__ long long tree_place(const TreeArgs &a, const long long *cum, const int *items, long long w)
{
    int x = 0, y = a.batch;
    while (y - x > 1) {
        const int z = (x + y) / 2;
        if (cum[z] + (long long)COST * items[z] <= w)
            x = z;
        else
            y = z;
    }
    const int here = items[x + 1] - items[x];
    if (here == 0)
        return cum[x];
    const int units = (a.kv_len[x] + TOKENS - 1) / TOKENS;
    const long long off = w - cum[x] - (long long)COST * items[x], at = min(tree_div(off, units + COST), (long long)here - 1);
    return cum[x] + at * units + min(off - at * (units + COST), (long long)units);
}

// Fills cum and items (scan, count: a word a warp) and gives this CTA's (worker's) units
// [lo, hi) and the cost of a run; zeros for rows of sequences that do not hold
template <int D, int ROWS, int TOKENS, int COST, int NT>
__device__ __forceinline__ void tree_list(const TreeArgs &a, long long *cum, int *items, long long *scan, int *count,
                                          long long &lo, long long &hi, long long &run, unsigned worker = blockIdx.x,
                                          unsigned workers = gridDim.x)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = (a.batch + NT - 1) / NT;
    long long mine = 0;
    int own = 0;
    for (int i = 0; i < per; ++i) {
        const int b = tid * per + i;
        if (b >= a.batch)
            break;
        int first, n, len, rows;
        tree_sequence(a, b, first, n, len, rows);
        cum[b] = mine;
        items[b] = own;
        const int here = n > 0 ? tree_blocks<ROWS>(n, a.group) * a.k.heads : 0;
        mine += (long long)((len + TOKENS - 1) / TOKENS) * here;
        own += here;
        if (n == 0 && rows > 0 && worker == (unsigned)b % workers)
            tree_zero<D>(a, first, rows);
    }
    long long incl = mine;
    int got = own;
    for (int m = 1; m < 32; m *= 2) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, incl, m);
        const int u = __shfl_up_sync(0xFFFFFFFFu, got, m);
        if (lane >= m) {
            incl += v;
            got += u;
        }
    }
    if (lane == 31) {
        scan[warp] = incl;
        count[warp] = got;
    }
    __syncthreads();
    long long before = incl - mine;
    int ahead = got - own;
    for (int w = 0; w < warp; ++w) {
        before += scan[w];
        ahead += count[w];
    }
    for (int i = 0; i < per; ++i)
        if (tid * per + i < a.batch) {
            cum[tid * per + i] += before;
            items[tid * per + i] += ahead;
        }
    if (tid == NT - 1) {
        cum[a.batch] = before + mine;
        items[a.batch] = ahead + own;
    }
    __syncthreads();
    const long long total = cum[a.batch] + (long long)COST * items[a.batch];
    run = max(tree_div(total + workers - 1, workers), (long long)a.min_units);
    const long long w = run * worker + (lane & 1 ? run : 0);  // even lanes the begin, odd ones the end
    const long long place = w < total ? tree_place<ROWS, TOKENS, COST>(a, cum, items, w) : cum[a.batch];
    lo = __shfl_sync(0xFFFFFFFFu, place, 0);
    hi = __shfl_sync(0xFFFFFFFFu, place, 1);
}

// the item after `it` in the list (there is one)
template <int ROWS, int TOKENS>
__device__ __forceinline__ void tree_next(const TreeArgs &a, const long long *cum, TreeItem &it)
{
    it.lo += it.units;
    if (++it.block < tree_blocks<ROWS>(it.n, a.group))
        return;
    it.block = 0;
    if (++it.head < a.k.heads)
        return;
    it.head = 0;
    do
        ++it.b;
    while (it.b + 1 < a.batch && cum[it.b + 1] == it.lo);  // sequences without units
    it.first = a.q_start[it.b];
    it.n = a.q_start[it.b + 1] - it.first;
    it.len = a.kv_len[it.b];
    it.units = (it.len + TOKENS - 1) / TOKENS;
}

// COUNT values (from dimension d0) of a query row that LANES neighbouring
// lanes hold between them, as f16 pairs: the row times the power of two that
// brings its largest magnitude into [2^13, 2^14) (and the scale's sign). f16
// then holds bf16's values exactly down to 2^-17, 2^-30 of the largest; smaller
// ones lose bits to its subnormal numbers, 2^-25 at most. Returns what turns the row's scores into
// exponents of 2. A row with a NaN or an infinity becomes a row of NaN; a row
// that is not live (and every row for scale 0) one of zeros.
template <int COUNT, int LANES>
__device__ __forceinline__ float tree_row(const TreeArgs &a, bool live, int token, int head, int d0, uint32_t (&x)[COUNT / 2])
{
    const uint16_t *p = a.q + token * a.q_tok + head * a.q_head + d0;
    float top = 0.0f;
    bool odd = false;
#pragma unroll
    for (int e = 0; e < COUNT / 2; e += 4) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live && a.q_wide) {
            v = *reinterpret_cast<const uint4 *>(p + 2 * e);
        } else if (live) {
            v.x = p[2 * e] | (uint32_t)p[2 * e + 1] << 16;
            v.y = p[2 * e + 2] | (uint32_t)p[2 * e + 3] << 16;
            v.z = p[2 * e + 4] | (uint32_t)p[2 * e + 5] << 16;
            v.w = p[2 * e + 6] | (uint32_t)p[2 * e + 7] << 16;
        }
        x[e] = v.x;
        x[e + 1] = v.y;
        x[e + 2] = v.z;
        x[e + 3] = v.w;
#pragma unroll
        for (int i = e; i < e + 4; ++i) {
            const float f0 = fabsf(bf16_lo(x[i])), f1 = fabsf(bf16_hi(x[i]));
            odd |= !(f0 < INFINITY) || !(f1 < INFINITY);
            top = fmaxf(top, fmaxf(f0, f1));
        }
    }
#pragma unroll
    for (int m = 1; m < LANES; m *= 2) {
        top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
        odd |= __shfl_xor_sync(0xFFFFFFFFu, (int)odd, m) != 0;
    }
    // 2^e with top 2^e in [2^13, 2^14): two factors, as e can pass f32's exponents
    const int e = top > 0.0f && !odd ? 13 - ilogbf(top) : 0;
    const float up0 = exp2f((float)(e / 2)), up1 = exp2f((float)(e - e / 2));
    const float sign = a.scale < 0.0f ? -1.0f : a.scale > 0.0f ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 0; i < COUNT / 2; ++i) {
        const float f0 = bf16_lo(x[i]) * up0 * up1 * sign, f1 = bf16_hi(x[i]) * up0 * up1 * sign;
        x[i] = odd ? 0x7E007E00u : pack_h2(f0, f1);
    }
    // Not below 2^-126: there the exponents of all scores (below 2^38) vanish as they should, and -inf, of a token that
    // is not seen, is not multiplied by 0. Not above 2^88: the exponents stay finite, and scores that differ, by 2^-48
    // at least (a product of two of f16's smallest numbers), still do by 2^40.
    return sign == 0.0f ? 1.0f
                        : fminf(fmaxf(fabsf(a.scale) * 1.4426950408889634f / up0 / up1, 1.17549435e-38f), 3.0948501e26f);
}

// writes a row block: o[mt][j] of this lane divided by the rows' sums
template <int D, int MT>
__device__ __forceinline__ void tree_store(const TreeArgs &a, const TreeItem &it, float (&o)[MT][D / 8][4],
                                           const float (&l)[MT][2], int lane)
{
    constexpr int Q = D / 4;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int r = it.block * 16 * MT + mt * 16 + s * 8 + lane / 4;
            if (r >= it.n * a.group)
                continue;
            uint16_t *p = a.out + (it.first + r / a.group) * a.o_tok + (it.head * a.group + r % a.group) * a.o_head +
                          (lane & 3) * Q;
            const float inv = l[mt][s] == 0.0f ? 0.0f : 1.0f / l[mt][s];
#pragma unroll
            for (int x = 0; x < Q; x += 8) {  // column 2 tid of block j is dimension 2 tid D / 8 + j
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = x + 2 * i, c = s * 2 + e / (D / 8), j = e % (D / 8);
                    const __nv_bfloat162 v = __floats2bfloat162_rn(o[mt][j][c] * inv, o[mt][j + 1][c] * inv);
                    w[i] = *reinterpret_cast<const uint32_t *>(&v);
                }
                if (a.o_wide) {
                    *reinterpret_cast<uint4 *>(p + x) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        p[x + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
                }
            }
        }
}

// the run's last item, if it starts in the run and goes on after it
template <int ROWS, int COST>
__device__ __forceinline__ void tree_cut(const TreeArgs &a, const TreeItem &it, const int *items, long long lo, long long run,
                                         unsigned worker = blockIdx.x)
{
    const int ordinal = items[it.b] + it.head * tree_blocks<ROWS>(it.n, a.group) + it.block;
    const long long w = it.lo + (long long)COST * ordinal;  // where it begins in the list of costs
    const long long p0 = tree_div(w, run), p1 = tree_div(w + it.units - 1, run);
    a.cuts[worker] = {it.first, it.n, it.head, it.block, p0 == worker ? (int)(p1 - p0) : 0, it.lo == lo};
}

#define MOE_TREE_JOIN_ROWS 16
#define MOE_TREE_JOIN_PARTS 128  // whose weights are held at once

// Joins the partials of cut items: CTA (runs, 16 rows of the row block, CS
// pieces of four dimensions), LOADS loads of 16 bytes in flight a thread. Where
// an item has fewer (row, piece)s than the CTA threads, groups of threads take
// its parts in turn and are added in order. Bound by latency: a round of loads
// for the weights, then one for each LOADS parts of a group. Two instances are
// used: small ones, whose CTAs take all dimensions, where the items are many and
// of few parts (a run's end each), and large ones for few items of many parts.
template <int D, int NT, int CS, int LOADS>
__global__ void __launch_bounds__(NT) moe_tree_join_kernel(const __grid_constant__ TreeArgs a, const int rows, const int runs)
{
    constexpr int R = MOE_TREE_JOIN_ROWS, P = MOE_TREE_JOIN_PARTS, J = P / 32;
    constexpr int PER = CS * R > NT ? CS * R / NT : 1, U = LOADS / PER;  // (row, piece)s of a thread; parts at once
    __shared__ float weight[P][R], top[R], sum[R];
    __shared__ float4 group_sum[NT];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = blockIdx.y * R, first_piece = blockIdx.z * CS;
    const size_t size = (size_t)rows * (D + 2);
    pdl_wait();
    for (int begin = blockIdx.x; begin < runs; begin += 32 * gridDim.x) {
        const int look = begin + lane * gridDim.x;  // every warp looks at the same 32 runs
        uint32_t found = gridDim.x >= runs ? 1u : __ballot_sync(0xFFFFFFFFu, look < runs && a.cuts[min(look, runs - 1)].runs != 0);
        for (; found; found &= found - 1) {
            const int at = begin + (__ffs(found) - 1) * gridDim.x;
            const TreeCut c = a.cuts[at];
            const int live = min(R, c.n * a.group - c.block * rows - r0);
            if (c.runs == 0 || live <= 0)
                continue;
            // part i: of the first run the second slot, unless the item begins with the run
            const float *base = a.part + (size_t)at * 2 * size;
            auto part = [&](int i) { return base + (i == 0 && !c.whole_run ? size : 2 * i * size); };
            __syncthreads();  // the last item's numbers have been read
            for (int r = warp; r < live; r += NT / 32) {
                float v[J], s[J], m = -INFINITY, l = 0.0f;
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const bool there = lane + 32 * j <= c.runs;
                    v[j] = there ? part(lane + 32 * j)[rows * D + r0 + r] : -INFINITY;
                    s[j] = there ? part(lane + 32 * j)[rows * (D + 1) + r0 + r] : 0.0f;
                }
#pragma unroll
                for (int j = 0; j < J; ++j)
                    m = fmaxf(m, v[j]);
                for (int i = lane + P; i <= c.runs; i += 32)
                    m = fmaxf(m, part(i)[rows * D + r0 + r]);
#pragma unroll
                for (int x = 16; x; x /= 2)
                    m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
                auto factor = [&](float v) { return v == -INFINITY ? 1.0f : ex2((v - m) * a.join_c); };  // a NaN sum stays
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float f = factor(v[j]);
                    l += s[j] * f;
                    weight[lane + 32 * j][r] = f;
                }
                for (int i = lane + P; i <= c.runs; i += 32)
                    l += part(i)[rows * (D + 1) + r0 + r] * factor(part(i)[rows * D + r0 + r]);
                l = warp_sum(l);
                if (lane == 0) {
                    top[r] = m;
                    sum[r] = l;
                }
            }
            __syncthreads();
            float4 o[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k)
                o[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const int pairs = live * CS, groups = max(1, NT / pairs), group = groups > 1 ? tid / pairs : 0;
            const int x0 = tid - group * pairs;  // pairs x0, x0 + NT, ..: row x % live, piece first_piece + x / live
            int row[PER], place[PER];
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                const int x = group < groups && x0 + k * NT < pairs ? x0 + k * NT : -1;
                row[k] = x < 0 ? -1 : x % live;
                place[k] = x < 0 ? 0 : (first_piece + x / live) * rows + r0 + row[k];
            }
            for (int p0 = 0; p0 <= c.runs; p0 += P) {
                const int n = min(P, c.runs + 1 - p0);
                if (p0 > 0) {  // the next weights
                    __syncthreads();
                    for (int x = tid; x < n * R; x += NT)
                        if (x % R < live) {
                            const float v = part(p0 + x / R)[rows * D + r0 + x % R];
                            weight[x / R][x % R] = v == -INFINITY ? 1.0f : ex2((v - top[x % R]) * a.join_c);
                        }
                    __syncthreads();
                }
                for (int i0 = group; i0 < n && row[0] >= 0; i0 += groups * U) {
                    float4 v[U][PER];
#pragma unroll
                    for (int i = 0; i < U; ++i)
#pragma unroll
                        for (int k = 0; k < PER; ++k) {
                            const int p = i0 + i * groups;
                            v[i][k] = p < n && row[k] >= 0 ? reinterpret_cast<const float4 *>(part(p0 + p))[place[k]]
                                                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
#pragma unroll
                    for (int i = 0; i < U; ++i)
#pragma unroll
                        for (int k = 0; k < PER; ++k) {
                            const int p = i0 + i * groups;
                            const float f = p < n && row[k] >= 0 ? weight[p][row[k]] : 0.0f;
                            o[k].x = fmaf(v[i][k].x, f, o[k].x);
                            o[k].y = fmaf(v[i][k].y, f, o[k].y);
                            o[k].z = fmaf(v[i][k].z, f, o[k].z);
                            o[k].w = fmaf(v[i][k].w, f, o[k].w);
                        }
                }
            }
            if (groups > 1) {
                group_sum[tid] = o[0];
                __syncthreads();
                for (int g = 1; g < groups && group == 0; ++g) {  // (group 0: x0 < pairs)
                    const float4 v = group_sum[g * pairs + x0];
                    o[0].x += v.x;
                    o[0].y += v.y;
                    o[0].z += v.z;
                    o[0].w += v.w;
                }
            }
#pragma unroll
            for (int k = 0; k < PER; ++k) {
                if (group > 0 || row[k] < 0)
                    continue;
                const int rr = c.block * rows + r0 + row[k];
                const float inv = sum[row[k]] == 0.0f ? 0.0f : 1.0f / sum[row[k]];
                uint16_t *to = a.out + (c.first + rr / a.group) * a.o_tok + (c.head * a.group + rr % a.group) * a.o_head +
                               (first_piece + (x0 + k * NT) / live) * 4;
                const __nv_bfloat162 lo = __floats2bfloat162_rn(o[k].x * inv, o[k].y * inv);
                const __nv_bfloat162 hi = __floats2bfloat162_rn(o[k].z * inv, o[k].w * inv);
                const uint32_t w0 = *reinterpret_cast<const uint32_t *>(&lo), w1 = *reinterpret_cast<const uint32_t *>(&hi);
                if (a.o_wide) {
                    *reinterpret_cast<uint2 *>(to) = make_uint2(w0, w1);
                } else {
                    to[0] = (uint16_t)w0;
                    to[1] = (uint16_t)(w0 >> 16);
                    to[2] = (uint16_t)w1;
                    to[3] = (uint16_t)(w1 >> 16);
                }
            }
        }
    }
}

template <int FMT, int D, int MT>
__global__ void __launch_bounds__(MOE_TREE_THREADS, TreeShape<FMT, D, MT>::CTAS) moe_tree_attn_kernel(const __grid_constant__ TreeArgs a, const int stages)
{
    using T = TreeShape<FMT, D, MT>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem);                           // [warps][8]
    unsigned long long *masks = reinterpret_cast<unsigned long long *>(smem + T::BARS);  // [rows]
    float *cmul = reinterpret_cast<float *>(smem + T::BARS + 8 * T::ROWS);         // [rows]
    float *wm = cmul + T::ROWS, *wl = wm + MOE_TREE_WARPS * T::ROWS;               // [warps][rows]
    long long *scan = reinterpret_cast<long long *>(smem + T::HEAD - 48);          // [warps]
    uint4 *qf = reinterpret_cast<uint4 *>(smem + T::HEAD);                         // [mt][ks][lane]
    float4 *merge = reinterpret_cast<float4 *>(smem + T::HEAD + T::QBYTES);        // [2][regs / 4][lane]
    long long *cum = reinterpret_cast<long long *>(smem + T::FIXED + (size_t)MOE_TREE_WARPS * stages * T::BLOCK);  // [batch + 1]
    int *items = reinterpret_cast<int *>(cum + a.batch + 1);                       // [batch + 1]
    int *count = reinterpret_cast<int *>(scan + MOE_TREE_WARPS);                   // [warps]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    uint8_t *ring = smem + T::FIXED + (size_t)warp * stages * T::BLOCK;
    uint64_t *bar = bars + warp * 8;
    if (lane == 0) {
        for (int s = 0; s < stages; ++s)
            mbar_init(bar + s, 1);
        fence_barrier_init();
    }
    long long lo, hi, run;
    pdl_wait();
    tree_list<D, T::ROWS, MOE_KV_BLOCK, MOE_TREE_COST, MOE_TREE_THREADS>(a, cum, items, scan, count, lo, hi, run);
    pdl_launch_dependents();
    if (lo >= hi) {
        if (tid == 0)
            a.cuts[blockIdx.x].runs = 0;
        return;
    }
    const int mine = (int)((hi - lo - warp + MOE_TREE_WARPS - 1) / MOE_TREE_WARPS);  // this warp's units
    const uint64_t policy = policy_evict_first();
    bool ok = true;

    // the copies' side: lane i holds the place of this warp's unit batch + i
    int asked = 0, batch = 0;
    const uint8_t *place = nullptr;
    uint32_t bad = 0, bad_before = 0;  // units of this batch (the one before) whose page lay outside
    auto look = [&](int at) {
        batch = at;
        bool out = false;
        place = a.pages;
        if (at + lane < mine) {
            const long long u = lo + warp + (long long)(at + lane) * MOE_TREE_WARPS;
            const TreeItem it = tree_item<T::ROWS, MOE_KV_BLOCK>(a, cum, u);
            const int blk = (int)(u - it.lo), per_page = a.k.page / 16;
            const int page = a.table[it.b * a.table_stride + blk / per_page];
            out = page < 0 || page >= a.n_pages;
            if (out)
                atomicOr(a.ctrl + MOE_CTRL_STATUS, (uint32_t)MOE_WS_INDEX);
            else
                place = a.pages + (((size_t)page * a.k.heads + it.head) * per_page + blk % per_page) * T::BLOCK;
        }
        bad_before = bad;
        bad = __ballot_sync(0xFFFFFFFFu, out);
    };
    auto ask = [&](int s) {  // the copy of the next unit, into stage s
        if (asked - batch == 32)
            look(asked);
        const uint8_t *src = reinterpret_cast<const uint8_t *>(
            __shfl_sync(0xFFFFFFFFu, reinterpret_cast<unsigned long long>(place), asked - batch));
        if (lane == 0) {
            mbar_arrive_expect_tx(bar + s, T::BLOCK);
            bulk_g2s(ring + s * T::BLOCK, src, T::BLOCK, bar + s, policy);
        }
        ++asked;
    };
    if (mine > 0)
        look(0);
    for (int s = 0; s < stages && asked < mine; ++s)
        ask(s);

    int done = 0, stage = 0;
    uint32_t phase = 0;
    for (long long u = lo; u < hi;) {
        const TreeItem it = tree_item<T::ROWS, MOE_KV_BLOCK>(a, cum, u);
        const long long end = min(hi, it.lo + it.units);
        // query fragments: k step ks of lane (g, t4) is dimensions t4 D / 4 + 4 ks .. + 3 of rows g and g + 8; here
        // eight threads have a row between them
#pragma unroll 1
        for (int mt = 0; mt < MT; ++mt) {
            const int at = mt * 16 + (tid >> 3), part = tid & 7, r = it.block * T::ROWS + at;
            const bool live = r < it.n * a.group;
            const int i = live ? r / a.group : 0;
            uint32_t x[D / 16];
            const float mul = tree_row<D / 8, 8>(a, live, it.first + i, it.head * a.group + (live ? r - i * a.group : 0),
                                                 part * (D / 8), x);
            if (part == 0) {
                cmul[at] = mul;
                masks[at] = !live ? 0 : a.mask ? a.mask[it.first + i] : (2ull << i) - 1;
            }
            uint32_t *to = reinterpret_cast<uint32_t *>(
                qf + (mt * T::KS + (part & 1) * (D / 32)) * 32 + (at & 7) * 4 + (part >> 1)) + (at >> 3 & 1);
#pragma unroll
            for (int e = 0; e < D / 16; ++e)
                to[(e >> 1) * 128 + (e & 1) * 2] = x[e];
        }
        __syncthreads();
        uint4 qr[T::QREG ? MT : 1][T::QREG ? T::KS : 1];
        if constexpr (T::QREG)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int ks = 0; ks < T::KS; ++ks)
                    qr[mt][ks] = qf[(mt * T::KS + ks) * 32 + lane];
        // z: minus the row's reference, as a score: where the scores' sums begin. So an exponent is the multiple of a
        // difference, as exact as the scores however large they are. The bits 0: there is no reference yet.
        float c[MT][2], z[MT][2], l[MT][2], o[MT][T::NB][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                c[mt][s] = cmul[mt * 16 + s * 8 + g];
                z[mt][s] = 0.0f;
                l[mt][s] = 0.0f;
            }
#pragma unroll
            for (int j = 0; j < T::NB; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[mt][j][i] = 0.0f;
        }
        const int prefix = it.len - it.n;
        // this warp's units below `last` belong to the item; the first token of unit `done`
        const int last = min(mine, (int)((end - lo - warp + MOE_TREE_WARPS - 1) / MOE_TREE_WARPS));
        int first = (int)(lo + warp + (long long)done * MOE_TREE_WARPS - it.lo) * 16;
        for (; done < last; ++done, first += 16 * MOE_TREE_WARPS) {
            if (ok)
                ok = __all_sync(0xFFFFFFFFu, mbar_wait(bar + stage, phase, a.ctrl + MOE_CTRL_STATUS, a.wait_ns));
            const uint8_t *blk = ring + stage * T::BLOCK;
            const bool gone = (done >= batch ? bad >> (done - batch) : bad_before >> (done - batch + 32)) & 1;
            const bool masked = gone || first + 16 > prefix;

            // ---- scores: columns 2 t4, 2 t4 + 1 of two blocks of eight tokens
            float s[MT][2][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[mt][nb][i] = z[mt][i / 2];
            {
                uint32_t kw[2 * T::WK];
#pragma unroll
                for (int i = 0; i < 2 * T::WK; i += 4)
                    *reinterpret_cast<uint4 *>(kw + i) = *reinterpret_cast<const uint4 *>(blk + i * 128 + lane * 16);
                constexpr int GL = D == 256 ? 2 : 1;  // groups of a lane's quarter
                __half2 kd[2][GL], km[2][GL];
#pragma unroll
                for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                    for (int x = 0; x < GL; ++x) {
                        const int at2 = (nb * 8 + g) * T::GR + (D == 64 ? t4 / 2 : t4 * GL + x);
                        if (FMT == MOE_KV_Q8) {
                            kd[nb][x] = __half2half2(reinterpret_cast<const __half *>(blk + 16 * T::RB)[at2]);
                        } else {
                            const uint32_t w = reinterpret_cast<const uint32_t *>(blk + 16 * T::RB)[at2];
                            kd[nb][x] = h2(dup_lo(w));
                            km[nb][x] = h2(dup_hi(w));
                        }
                    }
#pragma unroll
                for (int ks = 0; ks < T::KS; ++ks) {
                    const int x = GL == 1 ? 0 : ks / (T::KS / 2);
                    uint32_t b[2][2];
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb) {
                        if (FMT == MOE_KV_Q8) {
                            const uint32_t w = kw[nb * T::WK + ks];
                            b[nb][0] = q8_pair(w, 0x5140, kd[nb][x]);
                            b[nb][1] = q8_pair(w, 0x5342, kd[nb][x]);
                        } else {
                            const uint32_t w = kw[nb * T::WK + ks / 2] >> (8 * (ks & 1));
                            b[nb][0] = q4_pair((w & 0x000F000Fu) | 0x64006400u, kd[nb][x], km[nb][x]);
                            b[nb][1] = q4_pair((w >> 4 & 0x000F000Fu) | 0x64006400u, kd[nb][x], km[nb][x]);
                        }
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint4 q = T::QREG ? qr[T::QREG ? mt : 0][T::QREG ? ks : 0] : qf[(mt * T::KS + ks) * 32 + lane];
                        mma16816(s[mt][0], q, b[0][0], b[0][1]);
                        mma16816(s[mt][1], q, b[1][0], b[1][1]);
                    }
                }
            }
            if (masked) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int j = first + (i / 4) * 8 + t4 * 2 + (i & 1), row = mt * 16 + (i & 2) * 4 + g;
                        const bool sees = !gone && j < it.len && (j < prefix || masks[row] >> (j - prefix) & 1);
                        if (!sees)
                            s[mt][i / 4][i & 3] = -INFINITY;
                    }
            }
            // ---- weights
            uint4 p[MT];
            bool moves = false;
            float top[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float v = fmaxf(fmaxf(s[mt][0][2 * r], s[mt][0][2 * r + 1]), fmaxf(s[mt][1][2 * r], s[mt][1][2 * r + 1]));
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
                    top[mt][r] = v;
                    moves |= v * c[mt][r] > (__float_as_uint(z[mt][r]) ? MOE_TREE_SLACK : -INFINITY);
                }
            if (__any_sync(0xFFFFFFFFu, moves)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float keep[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float by = top[mt][r] * c[mt][r];
                        const bool none = __float_as_uint(z[mt][r]) == 0;
                        const bool up = by > (none ? -INFINITY : MOE_TREE_SLACK);
                        const float less = up ? top[mt][r] : 0.0f;
                        keep[r] = up && !none ? ex2(-by) : 1.0f;
                        z[mt][r] = up ? -(top[mt][r] + (0.0f - z[mt][r])) : z[mt][r];  // (never +0)
                        l[mt][r] *= keep[r];
#pragma unroll
                        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                            for (int i = 2 * r; i < 2 * r + 2; ++i)
                                s[mt][nb][i] -= less;
                    }
#pragma unroll
                    for (int j = 0; j < T::NB; ++j) {
                        o[mt][j][0] *= keep[0];
                        o[mt][j][1] *= keep[0];
                        o[mt][j][2] *= keep[1];
                        o[mt][j][3] *= keep[1];
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float e[2][4];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int nb = 0; nb < 2; ++nb)
#pragma unroll
                        for (int i = 2 * r; i < 2 * r + 2; ++i)
                            e[nb][i] = ex2(fmaf(s[mt][nb][i], c[mt][r], MOE_TREE_LIFT));
                    l[mt][r] += (e[0][2 * r] + e[0][2 * r + 1]) + (e[1][2 * r] + e[1][2 * r + 1]);
                }
                p[mt] = make_uint4(pack_h2(e[0][0], e[0][1]), pack_h2(e[0][2], e[0][3]), pack_h2(e[1][0], e[1][1]),
                                   pack_h2(e[1][2], e[1][3]));
            }
            // ---- o += P V: a lane's words of tokens 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9
            {
                const uint8_t *vb = blk + T::HALF;
                uint32_t vw[4 * T::WV];
#pragma unroll
                for (int i = 0; i < 4 * T::WV; i += 4)
                    *reinterpret_cast<uint4 *>(vw + i) = *reinterpret_cast<const uint4 *>(vb + i * 128 + lane * 16);
                const uint32_t *vs = reinterpret_cast<const uint32_t *>(vb + 16 * T::RB);  // pairs of tokens
                const int at2 = g * T::GR / 8 * 8 + t4;
                __half2 vd[2], vm[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    vd[x] = h2(vs[at2 + 4 * x]);
                    if (FMT == MOE_KV_Q4)
                        vm[x] = h2(vs[T::GR * 8 + at2 + 4 * x]);
                }
                if (masked) {  // bytes past the length, of no page or of a token that no row sees are anything: 0 as values
                    unsigned long long seen = ~0ull;
                    if (a.mask) {
                        seen = masks[lane & (T::ROWS - 1)] | (T::ROWS > 32 ? masks[lane + T::ROWS - 32] : 0);
                        seen = __reduce_or_sync(0xFFFFFFFFu, (uint32_t)seen) |
                               (unsigned long long)__reduce_or_sync(0xFFFFFFFFu, (uint32_t)(seen >> 32)) << 32;
                    }
                    auto in = [&](int j) { return j < it.len && (j < prefix || seen >> (j - prefix) & 1); };
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int j = first + 8 * x + 2 * t4;
                        const uint32_t keep = gone ? 0u : (in(j) ? 0xFFFFu : 0u) | (in(j + 1) ? 0xFFFF0000u : 0u);
                        vd[x] = h2(h2(vd[x]) & keep);
                        if (FMT == MOE_KV_Q4)
                            vm[x] = h2(h2(vm[x]) & keep);
                    }
                }
                if (FMT == MOE_KV_Q8) {
#pragma unroll
                    for (int w = 0; w < T::WV; ++w) {
                        uint32_t b[2][4];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t w0 = vw[(2 * x) * T::WV + w], w1 = vw[(2 * x + 1) * T::WV + w];
                            const uint32_t a0 = __byte_perm(w0, w1, 0x5140), a1 = __byte_perm(w0, w1, 0x7362);
                            b[x][0] = q8_pair(a0, 0x5140, vd[x]);
                            b[x][1] = q8_pair(a0, 0x5342, vd[x]);
                            b[x][2] = q8_pair(a1, 0x5140, vd[x]);
                            b[x][3] = q8_pair(a1, 0x5342, vd[x]);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
                                mma16816(o[mt][4 * w + i], p[mt], b[0][i], b[1][i]);
                    }
                } else {
#pragma unroll
                    for (int w = 0; w < T::WV; ++w)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // codes 2 i, 2 i + 1 of the word
                            uint32_t b[2][2];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t w0 = (vw[(2 * x) * T::WV + w] >> (4 * i) & 0x000F000Fu) | 0x64006400u;
                                const uint32_t w1 = (vw[(2 * x + 1) * T::WV + w] >> (4 * i) & 0x000F000Fu) | 0x64006400u;
                                b[x][0] = q4_pair(__byte_perm(w0, w1, 0x5410), vd[x], vm[x]);
                                b[x][1] = q4_pair(__byte_perm(w0, w1, 0x7632), vd[x], vm[x]);
                            }
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                mma16816(o[mt][8 * w + 2 * i], p[mt], b[0][0], b[1][0]);
                                mma16816(o[mt][8 * w + 2 * i + 1], p[mt], b[0][1], b[1][1]);
                            }
                        }
                }
            }
            __syncwarp();  // the stage has been read
            if (ok && asked < mine)
                ask(stage);
            if (++stage == stages) {
                stage = 0;
                phase ^= 1;
            }
        }

        // ---- join the warps: rows' references and sums, then o of warps 2, 3 into 0, 1 and 1 into 0
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[mt][r] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][r], 1);
                l[mt][r] += __shfl_xor_sync(0xFFFFFFFFu, l[mt][r], 2);
                z[mt][r] = __float_as_uint(z[mt][r]) ? -z[mt][r] : -INFINITY;  // the reference itself from here on
                if (t4 == 0) {
                    wm[warp * T::ROWS + mt * 16 + r * 8 + g] = z[mt][r];
                    wl[warp * T::ROWS + mt * 16 + r * 8 + g] = l[mt][r];
                }
            }
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = mt * 16 + r * 8 + g;
                float up = -INFINITY, sum = 0.0f;
                for (int w = 0; w < MOE_TREE_WARPS; ++w)
                    up = fmaxf(up, wm[w * T::ROWS + row]);
                for (int w = 0; w < MOE_TREE_WARPS; ++w) {
                    const float v = wm[w * T::ROWS + row];
                    sum += wl[w * T::ROWS + row] * (v == -INFINITY ? 1.0f : ex2((v - up) * c[mt][r]));  // a NaN sum stays
                }
                const float keep = z[mt][r] == -INFINITY ? 1.0f : ex2((z[mt][r] - up) * c[mt][r]);
                z[mt][r] = up;
                l[mt][r] = sum;
#pragma unroll
                for (int j = 0; j < T::NB; ++j) {
                    o[mt][j][2 * r] *= keep;
                    o[mt][j][2 * r + 1] *= keep;
                }
            }
        auto give = [&](int slot) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < T::NB; ++j)
                    merge[(slot * MT * T::NB + mt * T::NB + j) * 32 + lane] =
                        make_float4(o[mt][j][0], o[mt][j][1], o[mt][j][2], o[mt][j][3]);
        };
        auto take = [&](int slot) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < T::NB; ++j) {
                    const float4 v = merge[(slot * MT * T::NB + mt * T::NB + j) * 32 + lane];
                    o[mt][j][0] += v.x;
                    o[mt][j][1] += v.y;
                    o[mt][j][2] += v.z;
                    o[mt][j][3] += v.w;
                }
        };
        if (warp >= 2)
            give(warp - 2);
        __syncthreads();
        if (warp < 2)
            take(warp);
        __syncthreads();
        if (warp == 1)
            give(0);
        __syncthreads();
        const long long item_end = it.lo + it.units;
        const bool whole = u == it.lo && end == item_end;
        if (warp == 0) {
            take(0);
            if (whole) {
                tree_store<D, MT>(a, it, o, l, lane);
            } else {  // a partial: slot 0 is the run's first item, 1 its last
                float *part = a.part + ((size_t)blockIdx.x * 2 + (u == lo ? 0 : 1)) * T::PART;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int row = mt * 16 + r * 8 + g;
                        float4 *p = reinterpret_cast<float4 *>(part) + t4 * (D / 16) * T::ROWS + row;
#pragma unroll
                        for (int e = 0; e < D / 4; e += 4) {  // column 2 t4 of block j is dimension 2 t4 D / 8 + j
                            const int c = 2 * r + e / (D / 8), j = e % (D / 8);
                            p[e / 4 * T::ROWS] = make_float4(o[mt][j][c], o[mt][j + 1][c], o[mt][j + 2][c], o[mt][j + 3][c]);
                        }
                        if (t4 == 0) {
                            part[T::ROWS * D + row] = z[mt][r] * c[mt][r];  // as an exponent of 2
                            part[T::ROWS * D + T::ROWS + row] = l[mt][r];
                        }
                    }
            }
        }
        if (end == hi && tid == 0)
            tree_cut<T::ROWS, MOE_TREE_COST>(a, it, items, lo, run);
        u = end;
    }
    if (!ok)  // a copy did not arrive in time: wait for those in flight (bounded) before the memory is given back
        for (int k = max(0, asked - stages); k < asked; ++k)
            mbar_wait(bar + k % stages, (uint32_t)(k / stages) & 1u, a.ctrl + MOE_CTRL_STATUS, max(a.wait_ns, MOE_TREE_DRAIN_NS));
}

}  // namespace moe

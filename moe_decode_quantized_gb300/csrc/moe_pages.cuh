// moe_pages.cuh -- the care of a cache's pages on the device: reference counts
// and page tables (whole numbers, the same whatever the timing), and the copy of
// the pages' contents.
//
// The bookkeeping is one CTA's: pages are taken lowest first, in order of rows
// and entries, by one pass over the counts with a running count of the free ones
// (four counts a thread, a scan over the CTA a step), which ends where enough
// were found. Bound by latency: a round of loads and a scan for each 4096 counts
// that are passed over (the last page of 4096, 65536, 2^20 and 2^24 given and freed
// in 10.5, 16.5, 190 and 3070 us, call after call; a compaction's list 12.6, 45, 670 and
// 15600). The copies are bound by bytes.
#pragma once
#include "moe_common.cuh"

namespace moe {

#define MOE_PAGES_THREADS 1024
#define MOE_PAGES_MAX_ROWS 1024
#define MOE_PAGES_MAX_COPIES (1 << 30)          // pairs, whose numbers are counted in 31 bits
#define MOE_PAGES_STEP (4 * MOE_PAGES_THREADS)  // counts of a step of the pass

struct PagesArgs {
    int32_t *refs;
    int n_pages, page;
    int32_t *table;
    long long stride;
    int table_pages, rows;
    const int32_t *len, *source, *target;  // fork: lengths of the rows; free: target
    int n;
    int32_t *copies;
    int max_copies;
    int32_t *n_copies, *refs_out, *table_out;  // compact
    uint32_t *status;
};

__device__ __forceinline__ void pages_flag(const PagesArgs &a, uint32_t bits)
{
    if (a.status)
        atomicOr(a.status, bits);
}

// the sum of v over the CTA's threads before this one; total: over all. scan: [33]
__device__ __forceinline__ int pages_scan(int v, int *scan, int &total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, incl, m);
        incl += lane >= m ? u : 0;
    }
    __syncthreads();  // the last scan's numbers have been read
    if (lane == 31)
        scan[warp] = incl;
    __syncthreads();
    const int mine = scan[lane];
    int sums = mine;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, sums, m);
        sums += lane >= m ? u : 0;
    }
    total = __shfl_sync(0xFFFFFFFFu, sums, 31);
    return incl - v + __shfl_sync(0xFFFFFFFFu, sums - mine, warp);
}

// four counts from page p on (those past the end: -1, neither free nor held)
__device__ __forceinline__ int4 pages_counts(const int32_t *refs, int n_pages, int p)
{
    if (p + 4 <= n_pages && (reinterpret_cast<uintptr_t>(refs) & 15) == 0)
        return *reinterpret_cast<const int4 *>(refs + p);
    return make_int4(p < n_pages ? refs[p] : -1, p + 1 < n_pages ? refs[p + 1] : -1, p + 2 < n_pages ? refs[p + 2] : -1,
                     p + 3 < n_pages ? refs[p + 3] : -1);
}

// give(k, page) for the `need` lowest free pages in order, k = 0 ..; returns how many there were
template <typename F>
__device__ __forceinline__ int pages_take(const PagesArgs &a, int need, int *scan, F give)
{
    int found = 0;
    for (int p0 = 0; p0 < a.n_pages && found < need; p0 += MOE_PAGES_STEP) {
        const int p = p0 + 4 * threadIdx.x;
        const int4 c = pages_counts(a.refs, a.n_pages, p);
        const int f[4] = {c.x == 0, c.y == 0, c.z == 0, c.w == 0};
        int total;
        int k = found + pages_scan(f[0] + f[1] + f[2] + f[3], scan, total);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (f[i]) {
                if (k < need)
                    give(k, p + i);
                ++k;
            }
        found += total;
    }
    return min(found, need);
}

__global__ void __launch_bounds__(MOE_PAGES_THREADS) moe_pages_grow_kernel(const __grid_constant__ PagesArgs a)
{
    __shared__ int scan[33], held[MOE_PAGES_MAX_ROWS], want[MOE_PAGES_MAX_ROWS], before[MOE_PAGES_MAX_ROWS + 1];
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    for (int r = tid >> 5; r < a.rows; r += MOE_PAGES_THREADS / 32) {
        const int32_t *row = a.table + r * a.stride;
        const int len = a.len[r], pages = (int)(((long long)len + a.page - 1) / a.page);
        const bool fits = len >= 0 && pages <= a.table_pages;
        if (!fits && lane == 0)
            pages_flag(a, MOE_WS_INDEX);
        // the first entry that is -1, by 32 places at a time
        int lo = 0, hi = fits ? pages : 0;
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const int c = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && row[at] >= 0));
            if (c == 0)
                break;
            hi = step == 1 ? lo + c : min(hi, lo + c * step);
            lo = step == 1 ? hi : lo + (c - 1) * step + 1;
        }
        if (lane == 0) {
            held[r] = lo;
            want[r] = fits ? max(pages - lo, 0) : 0;
        }
    }
    __syncthreads();
    int need;
    const int mine = tid < a.rows ? want[tid] : 0;
    const int at = pages_scan(mine, scan, need);
    if (tid < a.rows)
        before[tid] = at;
    if (tid == 0)
        before[a.rows] = need;
    __syncthreads();
    const int got = pages_take(a, need, scan, [&](int k, int page) {
        int x = 0, y = a.rows;  // before[x] <= k < before[y]
        while (y - x > 1) {
            const int z = (x + y) / 2;
            if (before[z] <= k)
                x = z;
            else
                y = z;
        }
        a.table[x * a.stride + held[x] + k - before[x]] = page;
        a.refs[page] = 1;
    });
    if (got < need && tid == 0)
        pages_flag(a, MOE_WS_PAGES);
}

__global__ void __launch_bounds__(MOE_PAGES_THREADS) moe_pages_fork_kernel(const __grid_constant__ PagesArgs a)
{
    __shared__ int scan[33], owner[MOE_PAGES_MAX_ROWS], fresh[MOE_PAGES_MAX_ROWS], whole[MOE_PAGES_MAX_ROWS],
        rank[MOE_PAGES_MAX_ROWS];
    const int tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    for (int r = tid; r < a.rows; r += MOE_PAGES_THREADS)
        owner[r] = 0x7FFFFFFF;
    __syncthreads();
    int s = -1, t = -1;
    if (tid < a.n) {
        s = a.source[tid];
        t = a.target[tid];
        if (t >= 0 && t < a.rows)
            atomicMin(owner + t, tid);
    }
    __syncthreads();
    // a thread a pair: refused ones keep whole -1
    int part = 0, last = -1;
    if (tid < a.n) {
        whole[tid] = -1;
        bool ok = s >= 0 && s < a.rows && t >= 0 && t < a.rows && owner[t] == tid && owner[s] == 0x7FFFFFFF;
        if (ok) {
            const int len = a.len[s];
            ok = len >= 0 && (len + a.page - 1ll) / a.page <= a.table_pages;
            if (ok) {
                whole[tid] = len / a.page;
                if (len % a.page) {
                    last = a.table[s * a.stride + whole[tid]];
                    part = last >= 0 && last < a.n_pages;
                    if (!part)
                        pages_flag(a, MOE_WS_INDEX);
                }
            }
        }
        if (!ok)
            pages_flag(a, MOE_WS_INDEX);
    }
    int need;
    const int k = pages_scan(part, scan, need);
    if (tid < a.n) {
        rank[tid] = part ? k : -1;
        fresh[tid] = -1;
    }
    __syncthreads();
    // the full pages are shared, a warp a pair
    for (int i = tid >> 5; i < a.n; i += MOE_PAGES_THREADS / 32) {
        const int w = whole[i];
        if (w < 0)
            continue;
        const int32_t *from = a.table + a.source[i] * a.stride;
        int32_t *to = a.table + a.target[i] * a.stride;
        for (int j = lane; j < a.table_pages; j += 32) {
            int page = -1;
            if (j < w) {
                page = from[j];
                if (page >= 0 && page < a.n_pages) {
                    atomicAdd(a.refs + page, 1);
                } else {
                    page = -1;
                    pages_flag(a, MOE_WS_INDEX);
                }
            }
            to[j] = page;
        }
    }
    __syncthreads();
    // and the rest of each gets a page; `rank` of the pairs is ascending, so that pair i finds its page at its rank
    const int got = pages_take(a, need, scan, [&](int k, int page) {
        fresh[k] = page;
        a.refs[page] = 1;
    });
    if (got < need && tid == 0)
        pages_flag(a, MOE_WS_PAGES);
    __syncthreads();
    if (tid < a.n) {
        const int page = rank[tid] >= 0 && rank[tid] < got ? fresh[rank[tid]] : -1;
        if (page >= 0)
            a.table[t * a.stride + whole[tid]] = page;
        a.copies[2 * tid] = page >= 0 ? last : -1;
        a.copies[2 * tid + 1] = page;
    }
}

// a CTA a row; an entry is taken out by an exchange, so that a row that comes twice is freed once
__global__ void __launch_bounds__(256) moe_pages_free_kernel(const __grid_constant__ PagesArgs a)
{
    pdl_wait();
    const int r = a.target[blockIdx.x];
    if (r < 0 || r >= a.rows) {
        if (threadIdx.x == 0)
            pages_flag(a, MOE_WS_INDEX);
        return;
    }
    int32_t *row = a.table + r * a.stride;
    for (int j = threadIdx.x; j < a.table_pages; j += 256) {
        if (row[j] < 0)
            continue;
        const int page = atomicExch(row + j, -1);
        if (page < 0)
            continue;
        if (page >= a.n_pages)
            pages_flag(a, MOE_WS_INDEX);
        else if (atomicSub(a.refs + page, 1) <= 0) {  // it was not held
            atomicAdd(a.refs + page, 1);
            pages_flag(a, MOE_WS_INDEX);
        }
    }
}

__global__ void __launch_bounds__(MOE_PAGES_THREADS) moe_pages_compact_kernel(const __grid_constant__ PagesArgs a)
{
    __shared__ int scan[33];
    const int tid = threadIdx.x;
    pdl_wait();
    int live = 0, held = 0;
    for (int p = 4 * tid; p < a.n_pages; p += MOE_PAGES_STEP) {
        const int4 c = pages_counts(a.refs, a.n_pages, p);
        live += (c.x > 0) + (c.y > 0) + (c.z > 0) + (c.w > 0);
    }
    pages_scan(live, scan, held);
    int holes = 0, moved = 0;  // free pages below `held`, held ones from there on: as many
    for (int p0 = 0; p0 < a.n_pages; p0 += MOE_PAGES_STEP) {
        const int p = p0 + 4 * tid;
        const int4 c = pages_counts(a.refs, a.n_pages, p);
        const int n[4] = {c.x, c.y, c.z, c.w};
        int hole = 0, move = 0, total;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            hole += p + i < held && p + i < a.n_pages && n[i] <= 0;
            move += p + i >= held && n[i] > 0;
        }
        int k = holes + pages_scan(hole, scan, total);
        holes += total;
        int x = moved + pages_scan(move, scan, total);
        moved += total;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (p + i < held && p + i < a.n_pages && n[i] <= 0)
                a.copies[2 * k++ + 1] = p + i;
            if (p + i >= held && n[i] > 0)
                a.copies[2 * x++] = p + i;
        }
    }
    if (tid == 0)
        *a.n_copies = moved;
    __syncthreads();
    for (int i = moved + tid; i < a.max_copies; i += MOE_PAGES_THREADS)
        a.copies[2 * i] = a.copies[2 * i + 1] = -1;
    for (int p = tid; p < a.n_pages; p += MOE_PAGES_THREADS)
        if (p < held)
            a.refs_out[p] = a.refs[p];
    __syncthreads();
    for (int i = tid; i < moved; i += MOE_PAGES_THREADS)
        a.refs_out[a.copies[2 * i + 1]] = a.refs[a.copies[2 * i]];
    __syncthreads();
    for (int p = held + tid; p < a.n_pages; p += MOE_PAGES_THREADS)
        a.refs_out[p] = 0;
}

#define MOE_PAGES_MOVES 8192  // moves whose sources are searched in shared memory

// the table's entries after the moves: those that moved are found among the copies, which ascend
__global__ void __launch_bounds__(256) moe_pages_remap_kernel(const __grid_constant__ PagesArgs a)
{
    __shared__ int from[MOE_PAGES_MOVES];
    pdl_wait();
    const int moved = *a.n_copies, r = blockIdx.y;
    const bool near = moved <= MOE_PAGES_MOVES;  // (one round of loads instead of one for each step of a search)
    for (int i = threadIdx.x; near && i < moved; i += 256)
        from[i] = a.copies[2 * i];
    __syncthreads();
    for (int j = blockIdx.x * 256 + threadIdx.x; j < a.table_pages; j += gridDim.x * 256) {
        int page = a.table[r * a.stride + j];
        if (page >= a.n_pages)
            pages_flag(a, MOE_WS_INDEX);
        int x = 0, y = page < 0 ? 0 : moved;
        while (x < y) {
            const int z = (x + y) / 2;
            if ((near ? from[z] : a.copies[2 * z]) < page)
                x = z + 1;
            else
                y = z;
        }
        if (page >= 0 && x < moved && a.copies[2 * x] == page)
            page = a.copies[2 * x + 1];
        a.table_out[r * a.stride + j] = page;
    }
}

#define MOE_PAGES_COPY_THREADS 256
#define MOE_PAGES_PIECE 16384  // bytes of a unit of the copies

struct CopyArgs {
    char *pages;
    long long layer_stride, page_bytes;
    int layers, n_pages, pieces;  // units of a page
    const int32_t *copies;
    int n;
    const int32_t *n_copies;
    uint32_t *status;
};

__global__ void __launch_bounds__(MOE_PAGES_COPY_THREADS) moe_pages_copy_kernel(const __grid_constant__ CopyArgs a)
{
    pdl_wait();
    const int n = a.n_copies ? min(a.n, *a.n_copies) : a.n;
    const long long units = (long long)n * a.layers * a.pieces;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const long long rest = u / a.pieces;
        const int piece = (int)(u - rest * a.pieces), layer = (int)(rest % a.layers), i = (int)(rest / a.layers);
        const int from = a.copies[2 * i], to = a.copies[2 * i + 1];
        if (from < 0 || to < 0)
            continue;
        if (from >= a.n_pages || to >= a.n_pages) {
            if (threadIdx.x == 0 && a.status)
                atomicOr(a.status, (uint32_t)MOE_WS_INDEX);
            continue;
        }
        const long long off = (long long)piece * MOE_PAGES_PIECE, bytes = min((long long)MOE_PAGES_PIECE, a.page_bytes - off);
        char *base = a.pages + layer * a.layer_stride;
        const uint4 *src = reinterpret_cast<const uint4 *>(base + from * a.page_bytes + off);
        uint4 *dst = reinterpret_cast<uint4 *>(base + to * a.page_bytes + off);
        const int words = (int)(bytes / 16);
        constexpr int U = MOE_PAGES_PIECE / 16 / MOE_PAGES_COPY_THREADS;
        uint4 v[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (k * MOE_PAGES_COPY_THREADS + threadIdx.x < words)
                v[k] = src[k * MOE_PAGES_COPY_THREADS + threadIdx.x];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (k * MOE_PAGES_COPY_THREADS + threadIdx.x < words)
                dst[k * MOE_PAGES_COPY_THREADS + threadIdx.x] = v[k];
    }
}

}  // namespace moe

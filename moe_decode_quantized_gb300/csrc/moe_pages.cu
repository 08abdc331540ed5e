// moe_pages.cu -- the entry points of libmoe.so for the care of a cache's pages
// (declared and documented in include/moe.h): argument checks and launches.
#include <algorithm>

#include "moe_launch.cuh"
#include "moe_pages.cuh"

using namespace moe;

namespace {

int check_pool(const moe_page_pool *pool, const char *call, const int32_t *table, int64_t stride, int table_pages,
               int rows, const uint32_t *status, PagesArgs &a)
{
    if (!pool || !pool->refs)
        return host_fail(MOE_EINVAL, "%s: the pool or its counts are NULL", call);
    if (pool->n_pages < 1 || pool->page_size < 1)
        return host_fail(MOE_EINVAL, "%s: n_pages (%lld) and page_size (%d) must be positive", call,
                         (long long)pool->n_pages, pool->page_size);
    if (pool->n_pages > 1 << 24)
        return host_fail(MOE_EUNSUPPORTED, "%s: n_pages (%lld) <= 2^24", call, (long long)pool->n_pages);
    if (rows < 0 || table_pages < 1 || (rows > 1 && stride < table_pages))
        return host_fail(MOE_EINVAL, "%s: rows (%d) must not be negative, table_pages (%d) positive and at most "
                         "table_stride (%lld)", call, rows, table_pages, (long long)stride);
    if (rows > MOE_PAGES_MAX_ROWS)
        return host_fail(MOE_EUNSUPPORTED, "%s: rows (%d) <= %d", call, rows, MOE_PAGES_MAX_ROWS);
    if (rows > 0 && !table)
        return host_fail(MOE_EINVAL, "%s: the table is NULL", call);
    if (!aligned(pool->refs, 4) || !aligned(table, 4) || !aligned(status, 4))
        return host_fail(MOE_EINVAL, "%s: an argument is not aligned to its type", call);
    a.refs = pool->refs;
    a.n_pages = (int)pool->n_pages;
    a.page = pool->page_size;
    a.table = const_cast<int32_t *>(table);
    a.stride = stride;
    a.table_pages = table_pages;
    a.rows = rows;
    a.status = const_cast<uint32_t *>(status);
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_pages_grow(const moe_page_pool *pool, int32_t *table_dev, int64_t table_stride, int table_pages, int rows,
                   const int32_t *len_dev, uint32_t *status_dev, moe_stream_t stream)
{
    PagesArgs a{};
    const int rc = check_pool(pool, "moe_pages_grow", table_dev, table_stride, table_pages, rows, status_dev, a);
    if (rc || rows == 0)
        return rc;
    if ((long long)rows * table_pages > 0x7FFFFFFFll)  // (the entries that lengths may ask for are counted in 32 bits)
        return host_fail(MOE_EUNSUPPORTED, "moe_pages_grow: rows (%d) * table_pages (%d) < 2^31", rows, table_pages);
    if (!len_dev || !aligned(len_dev, 4))
        return host_fail(MOE_EINVAL, "moe_pages_grow: the lengths are NULL or not aligned to their type");
    a.len = len_dev;
    MOE_CUDA_OK(launch(moe_pages_grow_kernel, dim3(1), MOE_PAGES_THREADS, 0, stream, a));
    return MOE_OK;
}

int moe_pages_fork(const moe_page_pool *pool, int32_t *table_dev, int64_t table_stride, int table_pages, int rows,
                   const int32_t *kv_len_dev, const int32_t *source_dev, const int32_t *target_dev, int n,
                   int32_t *copies_dev, uint32_t *status_dev, moe_stream_t stream)
{
    PagesArgs a{};
    const int rc = check_pool(pool, "moe_pages_fork", table_dev, table_stride, table_pages, rows, status_dev, a);
    if (rc)
        return rc;
    if (n < 0)
        return host_fail(MOE_EINVAL, "moe_pages_fork: n (%d) < 0", n);
    if (n > MOE_PAGES_MAX_ROWS)
        return host_fail(MOE_EUNSUPPORTED, "moe_pages_fork: n (%d) <= %d", n, MOE_PAGES_MAX_ROWS);
    if (n == 0)
        return MOE_OK;
    if (!kv_len_dev || !source_dev || !target_dev || !copies_dev)
        return host_fail(MOE_EINVAL, "moe_pages_fork: NULL argument");
    if (!aligned(kv_len_dev, 4) || !aligned(source_dev, 4) || !aligned(target_dev, 4) || !aligned(copies_dev, 4))
        return host_fail(MOE_EINVAL, "moe_pages_fork: an argument is not aligned to its type");
    a.len = kv_len_dev;
    a.source = source_dev;
    a.target = target_dev;
    a.n = n;
    a.copies = copies_dev;
    MOE_CUDA_OK(launch(moe_pages_fork_kernel, dim3(1), MOE_PAGES_THREADS, 0, stream, a));
    return MOE_OK;
}

int moe_pages_free(const moe_page_pool *pool, int32_t *table_dev, int64_t table_stride, int table_pages, int rows,
                   const int32_t *rows_dev, int n, uint32_t *status_dev, moe_stream_t stream)
{
    PagesArgs a{};
    const int rc = check_pool(pool, "moe_pages_free", table_dev, table_stride, table_pages, rows, status_dev, a);
    if (rc)
        return rc;
    if (n < 0 || (n > 0 && (!rows_dev || !aligned(rows_dev, 4))))
        return host_fail(MOE_EINVAL, "moe_pages_free: n (%d) < 0, or the rows are NULL or not aligned to their type", n);
    if (n == 0)
        return MOE_OK;
    a.target = rows_dev;
    MOE_CUDA_OK(launch(moe_pages_free_kernel, dim3((unsigned)n), 256, 0, stream, a));
    return MOE_OK;
}

int moe_pages_compact(const moe_page_pool *pool, const int32_t *table_dev, int64_t table_stride, int table_pages,
                      int rows, int32_t *refs_out_dev, int32_t *table_out_dev, int32_t *copies_dev, int max_copies,
                      int32_t *n_copies_dev, uint32_t *status_dev, moe_stream_t stream)
{
    PagesArgs a{};
    const int rc = check_pool(pool, "moe_pages_compact", table_dev, table_stride, table_pages, rows, status_dev, a);
    if (rc)
        return rc;
    if (!refs_out_dev || !copies_dev || !n_copies_dev || (rows > 0 && !table_out_dev))
        return host_fail(MOE_EINVAL, "moe_pages_compact: NULL argument");
    if (!aligned(refs_out_dev, 4) || !aligned(table_out_dev, 4) || !aligned(copies_dev, 4) || !aligned(n_copies_dev, 4))
        return host_fail(MOE_EINVAL, "moe_pages_compact: an argument is not aligned to its type");
    if (max_copies < pool->n_pages / 2)
        return host_fail(MOE_EINVAL, "moe_pages_compact: max_copies (%d) must be n_pages / 2 (%lld) at least", max_copies,
                         (long long)pool->n_pages / 2);
    if (max_copies > MOE_PAGES_MAX_COPIES)
        return host_fail(MOE_EUNSUPPORTED, "moe_pages_compact: max_copies (%d) <= 2^30", max_copies);
    a.refs_out = refs_out_dev;
    a.table_out = table_out_dev;
    a.copies = copies_dev;
    a.max_copies = max_copies;
    a.n_copies = n_copies_dev;
    MOE_CUDA_OK(launch(moe_pages_compact_kernel, dim3(1), MOE_PAGES_THREADS, 0, stream, a));
    if (rows > 0)
        MOE_CUDA_OK(launch(moe_pages_remap_kernel, dim3((unsigned)std::min(8, (table_pages + 255) / 256), (unsigned)rows),
                           256, 0, stream, a));
    return MOE_OK;
}

int moe_pages_copy(void *pages_dev, int64_t layer_stride, int layers, int64_t n_pages, int64_t page_bytes,
                   const int32_t *copies_dev, int n, const int32_t *n_copies_dev, uint32_t *status_dev,
                   moe_stream_t stream)
{
    if (n < 0 || layers < 0 || n_pages < 1 || page_bytes < 1 || n_pages > 0x7FFFFFFF)
        return host_fail(MOE_EINVAL, "moe_pages_copy: n (%d) and layers (%d) must not be negative, n_pages (%lld) and "
                         "page_bytes (%lld) positive, n_pages below 2^31", n, layers, (long long)n_pages, (long long)page_bytes);
    if (n > MOE_PAGES_MAX_COPIES)
        return host_fail(MOE_EUNSUPPORTED, "moe_pages_copy: n (%d) <= 2^30", n);
    if (n == 0 || layers == 0)
        return MOE_OK;
    if (!pages_dev || !copies_dev)
        return host_fail(MOE_EINVAL, "moe_pages_copy: NULL argument");
    if (!aligned(pages_dev, 16) || page_bytes % 16 || (layers > 1 && layer_stride % 16))
        return host_fail(MOE_EINVAL, "moe_pages_copy: pages, layer_stride and page_bytes must be multiples of 16");
    if (page_bytes > 1ll << 32)
        return host_fail(MOE_EUNSUPPORTED, "moe_pages_copy: page_bytes (%lld) <= 2^32", (long long)page_bytes);
    if (layers > 1 && (layer_stride < 0 || layer_stride / page_bytes < n_pages))
        return host_fail(MOE_EINVAL, "moe_pages_copy: layer_stride (%lld) is below n_pages (%lld) pages of %lld bytes",
                         (long long)layer_stride, (long long)n_pages, (long long)page_bytes);
    if (!aligned(copies_dev, 4) || !aligned(n_copies_dev, 4) || !aligned(status_dev, 4))
        return host_fail(MOE_EINVAL, "moe_pages_copy: an argument is not aligned to its type");
    CopyArgs a{};
    a.pages = static_cast<char *>(pages_dev);
    a.layer_stride = layers > 1 ? layer_stride : 0;
    a.page_bytes = page_bytes;
    a.layers = layers;
    a.n_pages = (int)n_pages;
    a.pieces = (int)((page_bytes + MOE_PAGES_PIECE - 1) / MOE_PAGES_PIECE);
    a.copies = copies_dev;
    a.n = n;
    a.n_copies = n_copies_dev;
    a.status = status_dev;
    // (some 32 CTAs an SM, so that an SM's last ones end together: 2052 pages of 73728 bytes in 2 layers with their list
    // 55.5 us, by 8 an SM 60; by 128, each of which may find nothing to do, 24 rows' 46.7 for 44.5)
    const long long units = (long long)n * layers * a.pieces;
    MOE_CUDA_OK(launch(moe_pages_copy_kernel, dim3((unsigned)std::min(units, 152ll * 32)), MOE_PAGES_COPY_THREADS, 0,
                       stream, a));
    return MOE_OK;
}

}  // extern "C"

// moe_spec.cu -- the entry points of libmoe.so for speculative decoding
// (declared and documented in include/moe.h): the quantised cache, attention
// of drafted tokens over it and their verification. Argument checks,
// workspace layout and launches.
#include <algorithm>
#include <mutex>

#include "moe_common.cuh"
#include "moe_host.cuh"
#include "moe_kv.cuh"
#include "moe_tree_attn.cuh"
#include "moe_tree_tc.cuh"
#include "moe_verify.cuh"

using namespace moe;

namespace {

#define SPEC_CUDA_OK(expr)                                                                              \
    do {                                                                                                \
        cudaError_t e_ = (expr);                                                                        \
        if (e_ != cudaSuccess)                                                                          \
            return host_fail(MOE_ECUDA, "%s: %s (%s)", #expr, cudaGetErrorString(e_), cudaGetErrorName(e_)); \
    } while (0)

// Launches behind the stream's last kernel while that still runs (the kernels wait for its end before they touch
// memory): one token over 511, call after call, 12.0 us a call, launched the plain way 16.4.
template <typename... A>
cudaError_t launch(void (*kernel)(A...), dim3 grid, int threads, size_t shared, moe_stream_t stream, A... args)
{
    cudaLaunchConfig_t lc{};
    lc.gridDim = grid;
    lc.blockDim = dim3((unsigned)threads);
    lc.dynamicSmemBytes = shared;
    lc.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, args...);
}

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

#define SPEC_CTRL_BYTES 256  // control words: the status is word MOE_CTRL_STATUS

int check_shape(const moe_kv_cache *c, KvDims &k)
{
    if (!c)
        return host_fail(MOE_EINVAL, "cache is NULL");
    if (c->format != MOE_KV_Q8 && c->format != MOE_KV_Q4)
        return host_fail(MOE_EINVAL, "cache format %d", c->format);
    if (c->head_dim < 1 || c->n_kv_heads < 1 || c->page_size < 1)
        return host_fail(MOE_EINVAL, "head_dim (%d), n_kv_heads (%d) and page_size (%d) must be positive", c->head_dim,
                         c->n_kv_heads, c->page_size);
    if ((c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) || c->n_kv_heads > 256 ||
        c->page_size % MOE_KV_BLOCK || c->page_size > 1024)
        return host_fail(MOE_EUNSUPPORTED, "head_dim (%d) of 64, 128 or 256, n_kv_heads (%d) <= 256, page_size (%d) a "
                         "multiple of 16 up to 1024", c->head_dim, c->n_kv_heads, c->page_size);
    k.dim = c->head_dim;
    k.heads = c->n_kv_heads;
    k.page = c->page_size;
    k.fmt = c->format;
    return MOE_OK;
}

int check_cache(const moe_kv_cache *c, KvDims &k)
{
    const int rc = check_shape(c, k);
    if (rc)
        return rc;
    if (!c->pages || !aligned(c->pages, 16))
        return host_fail(MOE_EINVAL, "the cache's pages are NULL or not 16-byte aligned");
    if (c->n_pages < 1 || c->n_pages > 0x7FFFFFFFll / c->page_size)
        return host_fail(MOE_EINVAL, "n_pages (%lld) must be positive and n_pages * page_size below 2^31",
                         (long long)c->n_pages);
    return MOE_OK;
}

// ---- the cache's kernels

// KvArgs::per_page
unsigned long long kv_per_page(const KvDims &k) { return ((1ull << 36) + k.page / 16 - 1) / (k.page / 16); }

using KvKernel = void (*)(KvArgs);

template <int FMT, int D>
KvKernel kv_read_kernel(bool f32, bool wide)
{
    if (f32)
        return wide ? moe_kv_read_kernel<FMT, D, true, true> : moe_kv_read_kernel<FMT, D, true, false>;
    return wide ? moe_kv_read_kernel<FMT, D, false, true> : moe_kv_read_kernel<FMT, D, false, false>;
}

// f<format, head size>() of the cache's
template <typename F>
auto with_kv(const KvDims &k, F &&f)
{
    if (k.fmt == MOE_KV_Q8)
        return k.dim == 64 ? f(IntC<MOE_KV_Q8>{}, IntC<64>{}) : k.dim == 128 ? f(IntC<MOE_KV_Q8>{}, IntC<128>{})
                                                                              : f(IntC<MOE_KV_Q8>{}, IntC<256>{});
    return k.dim == 64 ? f(IntC<MOE_KV_Q4>{}, IntC<64>{}) : k.dim == 128 ? f(IntC<MOE_KV_Q4>{}, IntC<128>{})
                                                                          : f(IntC<MOE_KV_Q4>{}, IntC<256>{});
}

// ---- verification

using VerifyKernel = void (*)(VerifyArgs);

template <bool AHEAD>
VerifyKernel verify_kernel(bool f32, bool wide)
{
    return f32 ? (wide ? moe_verify_kernel<true, true, AHEAD> : moe_verify_kernel<true, false, AHEAD>)
               : (wide ? moe_verify_kernel<false, true, AHEAD> : moe_verify_kernel<false, false, AHEAD>);
}

VerifyKernel verify_kernel(bool f32, bool wide, bool ahead)
{
    return ahead ? verify_kernel<true>(f32, wide) : verify_kernel<false>(f32, wide);
}

// The rows ahead pay where the walk would go through most of them: chains (4 rows of 32000: 7.2 us, in the walk 11.5;
// 48 x 8 of 131072: 38 and 50), and trees of few bytes (8 rows of 128000: 11 and 15 us; 24 of 100003 in f32, 9.6 MB:
// 14.2 and 14.8; 48 rows 15.4 and 16.4). Larger trees: 96 rows 17.2 and 13.4, 384 (154 MB) 40 and 18.5.
#define MOE_VERIFY_AHEAD_BYTES (20u << 20)

// ---- tree attention: instances and their launch shape

using TreeKernel = void (*)(TreeArgs, int);

struct TreeInstance {
    TreeKernel kernel;
    int rows;
    size_t fixed, stage;  // bytes of shared memory: beside the ring and the list; of a stage of all warps
    int ctas;             // an SM, by registers
};

template <int FMT, int D, int MT>
TreeInstance tree_instance()
{
    using T = TreeShape<FMT, D, MT>;
    return {moe_tree_attn_kernel<FMT, D, MT>, T::ROWS, (size_t)T::FIXED, (size_t)MOE_TREE_WARPS * T::BLOCK, T::CTAS};
}

#define MOE_TREE_MAX_GRID 640  // runs; the workspace holds two partials each
#define MOE_TTC_MAX_GRID 160   // of the tensor-core kernel
#define MOE_TREE_MAX_DEVICES 64

std::mutex g_tree_mu;

// The instance for (format, head size) with at least `rows` rows a block where there is one, else the largest: a block
// of the cache is then turned into numbers once (64 sequences of 12000 tokens, Q8, 32 rows of 128: 386 us, as two row
// blocks 502; of 16000, 64 rows of 64: 497 us, as two 631, as four 790). Heads of 256 leave registers for 16 rows.
int tree_choose(int fmt, int dim, int rows)
{
    const int mt = rows <= 16 ? 0 : rows <= 32 ? 1 : 2;
    const int first = dim == 64 ? 0 : dim == 128 ? 3 : 5, most = dim == 64 ? 2 : dim == 128 ? 1 : 0;
    return (fmt == MOE_KV_Q8 ? 0 : 6) + first + std::min(mt, most);
}

#define MOE_TREE_INSTANCES 12

// the tensor-core kernels' instances, by format
struct TtcInstance {
    TreeKernel kernel;
    size_t fixed, stage;
};

template <int FMT>
TtcInstance ttc_instance()
{
    using T = TtcShape<FMT>;
    return {moe_tree_tc_kernel<FMT>, 1024 + (size_t)T::RAW_AT + T::SMALL, (size_t)T::STAGE};
}

struct TreeDevice {
    int sms = 0;
    size_t per_sm = 0, optin = 0;  // shared memory
    TreeInstance inst[MOE_TREE_INSTANCES];
    TtcInstance tc[2];
};

int tree_device(TreeDevice **out)
{
    static TreeDevice dev[MOE_TREE_MAX_DEVICES];
    int d = 0;
    SPEC_CUDA_OK(cudaGetDevice(&d));
    if (d < 0 || d >= MOE_TREE_MAX_DEVICES)
        return host_fail(MOE_EUNSUPPORTED, "device ordinal %d", d);
    std::lock_guard<std::mutex> lk(g_tree_mu);
    TreeDevice &D = dev[d];
    if (!D.sms) {
        const TreeInstance all[MOE_TREE_INSTANCES] = {
            tree_instance<MOE_KV_Q8, 64, 1>(),  tree_instance<MOE_KV_Q8, 64, 2>(),  tree_instance<MOE_KV_Q8, 64, 4>(),
            tree_instance<MOE_KV_Q8, 128, 1>(), tree_instance<MOE_KV_Q8, 128, 2>(), tree_instance<MOE_KV_Q8, 256, 1>(),
            tree_instance<MOE_KV_Q4, 64, 1>(),  tree_instance<MOE_KV_Q4, 64, 2>(),  tree_instance<MOE_KV_Q4, 64, 4>(),
            tree_instance<MOE_KV_Q4, 128, 1>(), tree_instance<MOE_KV_Q4, 128, 2>(), tree_instance<MOE_KV_Q4, 256, 1>()};
        int n = 0, per_sm = 0, optin = 0;
        SPEC_CUDA_OK(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d));
        SPEC_CUDA_OK(cudaDeviceGetAttribute(&per_sm, cudaDevAttrMaxSharedMemoryPerMultiprocessor, d));
        SPEC_CUDA_OK(cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, d));
        for (int i = 0; i < MOE_TREE_INSTANCES; ++i) {
            SPEC_CUDA_OK(cudaFuncSetAttribute(all[i].kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin));
            D.inst[i] = all[i];
        }
        const TtcInstance tc[2] = {ttc_instance<MOE_KV_Q8>(), ttc_instance<MOE_KV_Q4>()};
        for (int i = 0; i < 2; ++i) {
            SPEC_CUDA_OK(cudaFuncSetAttribute(tc[i].kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin));
            D.tc[i] = tc[i];
        }
        D.per_sm = per_sm;
        D.optin = optin;
        D.sms = n;
    }
    *out = &D;
    return MOE_OK;
}

// The second kernel of a call. items: about how many there are; the runs that
// each may span decide on the instance (one sequence of 8000 tokens, 8 items of
// 57 parts: 21.5 us with the small one, 15.7 with the large; 2 items of 228: 65
// and 33; 8 of 19, heads of 256: 17.7 and 15.9; two row blocks of 4 heads over 152
// runs: 124 and 125, 16 items over 152 runs: 24.5 and 30.8; one sequence of 511,
// whose 8 items have 4 parts and could have had 57: 11.2 and 11.7). The large
// one's CTAs, four an SM, go through several runs each.
using JoinKernel = void (*)(TreeArgs, int, int);

template <int D>
JoinKernel join_kernel(bool deep)
{
    return deep ? moe_tree_join_kernel<D, 256, 8, 8> : moe_tree_join_kernel<D, 256, D / 4, D == 64 ? 2 : 4>;
}

int tree_join(const TreeArgs &a, const TreeDevice &dev, int runs, int rows, long long items, moe_stream_t stream)
{
    const bool deep = runs / items >= 24;
    const int blocks = rows / MOE_TREE_JOIN_ROWS, slices = deep ? a.k.dim / 32 : 1;
    const dim3 grid(deep ? std::max(1, std::min(runs, 4 * dev.sms / (blocks * slices))) : runs, blocks, slices);
    const JoinKernel kernel = a.k.dim == 64 ? join_kernel<64>(deep) : a.k.dim == 128 ? join_kernel<128>(deep)
                                                                                      : join_kernel<256>(deep);
    SPEC_CUDA_OK(launch(kernel, grid, 256, 0, stream, a, rows, runs));
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_kv_page_bytes(const moe_kv_cache *cache, size_t *bytes)
{
    KvDims k;
    const int rc = check_shape(cache, k);
    if (rc)
        return rc;
    if (!bytes)
        return host_fail(MOE_EINVAL, "bytes is NULL");
    *bytes = k.page_bytes();
    return MOE_OK;
}

int moe_kv_append(const moe_kv_cache *cache, const void *k_dev, int64_t k_token_stride, int64_t k_head_stride,
                  const void *v_dev, int64_t v_token_stride, int64_t v_head_stride, const int32_t *slots_dev,
                  int n_tokens, uint32_t *status_dev, moe_stream_t stream)
{
    KvArgs a{};
    const int rc = check_cache(cache, a.k);
    if (rc)
        return rc;
    if (n_tokens < 0 || (n_tokens > 0 && (!k_dev || !v_dev || !slots_dev)))
        return host_fail(MOE_EINVAL, "moe_kv_append: NULL argument or n_tokens (%d) < 0", n_tokens);
    if (!aligned(k_dev, 2) || !aligned(v_dev, 2) || !aligned(slots_dev, 4) || !aligned(status_dev, 4))
        return host_fail(MOE_EINVAL, "moe_kv_append: an argument is not aligned to its type");
    if (n_tokens == 0)
        return MOE_OK;
    a.pages = static_cast<uint8_t *>(cache->pages);
    a.n_slots = cache->n_pages * cache->page_size;
    a.per_page = kv_per_page(a.k);
    a.src[0] = static_cast<const uint16_t *>(k_dev);
    a.src[1] = static_cast<const uint16_t *>(v_dev);
    a.tok_stride[0] = k_token_stride;
    a.tok_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride;
    a.head_stride[1] = v_head_stride;
    a.slots = slots_dev;
    a.tokens = n_tokens;
    a.status = status_dev;
    int align = 32;  // bytes that every row starts at a multiple of, 32, 16 or 2
    while (align > 2 && !(aligned(k_dev, align) && aligned(v_dev, align) &&
                          (k_token_stride | k_head_stride | v_token_stride | v_head_stride) * 2 % align == 0))
        align = align == 32 ? 16 : 2;
    KvKernel kernel = nullptr;
    int per = 0;  // tokens of a warp
    with_kv(a.k, [&](auto f, auto d) {
        constexpr int F = decltype(f)::value, D = decltype(d)::value;
        kernel = align == 32   ? moe_kv_append_kernel<F, D, 32>
                 : align == 16 ? moe_kv_append_kernel<F, D, 16>
                               : moe_kv_append_kernel<F, D, 2>;
        per = align == 2 ? kv_append_tokens<D, 2>() : kv_append_tokens<D, 16>();
        return 0;
    });
    const long long all = ((long long)n_tokens + per - 1) / per;  // warps a head
    const int warps = (int)std::min<long long>(MOE_KV_THREADS / 32, all);
    SPEC_CUDA_OK(launch(kernel, dim3((unsigned)((all + warps - 1) / warps), 2 * a.k.heads), warps * 32, 0, stream, a));
    return MOE_OK;
}

int moe_kv_read(const moe_kv_cache *cache, const int32_t *slots_dev, int n_tokens, void *k_out_dev, void *v_out_dev,
                int out_type, uint32_t *status_dev, moe_stream_t stream)
{
    KvArgs a{};
    const int rc = check_cache(cache, a.k);
    if (rc)
        return rc;
    if (n_tokens < 0 || (n_tokens > 0 && (!k_out_dev || !v_out_dev || !slots_dev)))
        return host_fail(MOE_EINVAL, "moe_kv_read: NULL argument or n_tokens (%d) < 0", n_tokens);
    if (out_type != MOE_BF16 && out_type != MOE_F32)
        return host_fail(MOE_EINVAL, "moe_kv_read: out_type %d", out_type);
    if (!aligned(k_out_dev, 16) || !aligned(v_out_dev, 16) || !aligned(slots_dev, 4) || !aligned(status_dev, 4))
        return host_fail(MOE_EINVAL, "moe_kv_read: outputs must be 16-byte aligned, slots and status 4-byte");
    if (n_tokens == 0)
        return MOE_OK;
    a.pages = static_cast<uint8_t *>(cache->pages);
    a.n_slots = cache->n_pages * cache->page_size;
    a.per_page = kv_per_page(a.k);
    a.slots = slots_dev;
    a.out[0] = k_out_dev;
    a.out[1] = v_out_dev;
    a.tokens = n_tokens;
    a.status = status_dev;
    const bool f32 = out_type == MOE_F32, wide = aligned(k_out_dev, 32) && aligned(v_out_dev, 32);
    KvKernel kernel = nullptr;
    int per = 0;  // the more threads that K's or V's tile of eight tokens takes
    with_kv(a.k, [&](auto f, auto d) {
        constexpr int F = decltype(f)::value, D = decltype(d)::value;
        kernel = kv_read_kernel<F, D>(f32, wide);
        per = std::max(kv_read_threads<F, D, false>(), kv_read_threads<F, D, true>());
        return 0;
    });
    const long long threads = (n_tokens + 7ll) / 8 * per;
    const dim3 grid((unsigned)((threads + MOE_KV_THREADS - 1) / MOE_KV_THREADS), 2 * a.k.heads);
    SPEC_CUDA_OK(launch(kernel, grid, MOE_KV_THREADS, 0, stream, a));
    return MOE_OK;
}

static int tree_ws(const moe_kv_cache *cache, int n_q_heads, int batch, int n_tokens, KvDims &k, size_t &bytes)
{
    const int rc = check_shape(cache, k);
    if (rc)
        return rc;
    if (n_q_heads < 1 || n_q_heads % k.heads || batch < 0 || n_tokens < 0)
        return host_fail(MOE_EINVAL, "n_q_heads (%d) must be a positive multiple of n_kv_heads (%d), batch (%d) and "
                         "n_tokens (%d) not negative", n_q_heads, k.heads, batch, n_tokens);
    if (n_q_heads / k.heads > 64 || batch > 1024 || n_tokens > batch * MOE_MAX_DRAFT)
        return host_fail(MOE_EUNSUPPORTED, "n_q_heads / n_kv_heads (%d) <= 64, batch (%d) <= 1024, n_tokens (%d) <= "
                         "%d a sequence", n_q_heads / k.heads, batch, n_tokens, MOE_MAX_DRAFT);
    // control words, cuts, and two partials of the largest row block a run
    const size_t rows = k.dim == 64 ? (size_t)MOE_TREE_MAX_GRID * 64
                        : k.dim == 128 ? (size_t)MOE_TTC_MAX_GRID * MOE_TTC_ROWS : (size_t)MOE_TREE_MAX_GRID * 16;
    bytes = SPEC_CTRL_BYTES + sizeof(TreeCut) * MOE_TREE_MAX_GRID + rows * 2 * 4 * (k.dim + 2);
    return MOE_OK;
}

int moe_tree_attention_workspace_bytes(const moe_kv_cache *cache, int n_q_heads, int batch, int n_tokens,
                                       size_t *bytes)
{
    if (!bytes)
        return host_fail(MOE_EINVAL, "bytes is NULL");
    KvDims k;
    return tree_ws(cache, n_q_heads, batch, n_tokens, k, *bytes);
}

int moe_tree_attention(const moe_kv_cache *cache, const void *q_dev, int64_t q_token_stride, int64_t q_head_stride,
                       void *out_dev, int64_t out_token_stride, int64_t out_head_stride, int n_q_heads,
                       const int32_t *q_start_dev, const int32_t *kv_len_dev, const int32_t *table_dev,
                       int64_t table_stride, int table_pages, const uint64_t *mask_dev, int batch, int n_tokens,
                       float scale, void *ws_dev, size_t ws_bytes, moe_stream_t stream)
{
    TreeArgs a{};
    int rc = check_cache(cache, a.k);
    if (rc)
        return rc;
    size_t need;
    if ((rc = tree_ws(cache, n_q_heads, batch, n_tokens, a.k, need)))
        return rc;
    if (batch == 0 || n_tokens == 0)
        return MOE_OK;
    if (!q_dev || !out_dev || !q_start_dev || !kv_len_dev || !table_dev || !ws_dev)
        return host_fail(MOE_EINVAL, "moe_tree_attention: NULL argument");
    if (!aligned(q_dev, 2) || !aligned(out_dev, 2) || !aligned(q_start_dev, 4) || !aligned(kv_len_dev, 4) ||
        !aligned(table_dev, 4) || !aligned(mask_dev, 8) || !aligned(ws_dev, 256))
        return host_fail(MOE_EINVAL, "moe_tree_attention: an argument is not aligned to its type, or ws_dev not to 256 "
                         "bytes");
    if (ws_bytes < need)
        return host_fail(MOE_EINVAL, "moe_tree_attention: the workspace holds %zu bytes, %zu are needed", ws_bytes, need);
    if (table_pages < 1 || (batch > 1 && table_stride < table_pages) || !(scale >= -3.0e38f && scale <= 3.0e38f))
        return host_fail(MOE_EINVAL, "moe_tree_attention: table_pages (%d) must be positive and at most table_stride "
                         "(%lld), scale finite", table_pages, (long long)table_stride);
    a.pages = static_cast<const uint8_t *>(cache->pages);
    a.n_pages = (int)cache->n_pages;
    a.q = static_cast<const uint16_t *>(q_dev);
    a.q_tok = q_token_stride;
    a.q_head = q_head_stride;
    a.out = static_cast<uint16_t *>(out_dev);
    a.o_tok = out_token_stride;
    a.o_head = out_head_stride;
    a.q_start = q_start_dev;
    a.kv_len = kv_len_dev;
    a.table = table_dev;
    a.table_stride = table_stride;
    a.max_len = (int)std::min((long long)table_pages * a.k.page, (long long)MOE_TREE_MAX_LEN);
    a.mask = reinterpret_cast<const unsigned long long *>(mask_dev);
    a.batch = batch;
    a.tokens = n_tokens;
    a.group = n_q_heads / a.k.heads;
    a.scale = scale;
    a.q_wide = aligned(q_dev, 16) && (q_token_stride | q_head_stride) % 8 == 0;
    a.o_wide = aligned(out_dev, 16) && (out_token_stride | out_head_stride) % 8 == 0;
    a.min_units = 2 * MOE_TREE_WARPS;  // (a sequence of 511 tokens: 11.7 us, with twice that 13.0; of 8000: 15.7, 16.3)
    a.ctrl = static_cast<uint32_t *>(ws_dev);
    a.cuts = reinterpret_cast<TreeCut *>(a.ctrl + SPEC_CTRL_BYTES / 4);
    a.part = reinterpret_cast<float *>(a.cuts + MOE_TREE_MAX_GRID);
    a.wait_ns = host_wait_ns();
    // the row block from the mean rows of a sequence (the lengths themselves are on the device)
    TreeDevice *dev;
    if ((rc = tree_device(&dev)))
        return rc;
    const int rows = (n_tokens + batch - 1) / batch * a.group;
    // The tensor-core kernel from where the warps' own products cost more than its longer steps (64 sequences of 12000
    // tokens, Q8, 32 rows: 386 us by warps, 586 us by it; 16 of up to 16000, Q4, 32 rows: 90 and 117 us; 16 of 4000, 48
    // rows in Q8 84 and 68 us, 64 in Q4 92 and 69 us)
    if (a.k.dim == 128 && rows > 32) {
        const TtcInstance &t = dev->tc[a.k.fmt == MOE_KV_Q8 ? 0 : 1];
        const size_t used = t.fixed + 12 * ((size_t)batch + 1);
        const int stages = (int)std::min<size_t>(4, (dev->optin - used) / t.stage);
        a.min_units = 2;
        const int grid = std::min(dev->sms, MOE_TTC_MAX_GRID);
        SPEC_CUDA_OK(launch(t.kernel, dim3(grid), MOE_TTC_THREADS, used + stages * t.stage, stream, a, stages));
        return tree_join(a, *dev, grid, MOE_TTC_ROWS, (long long)batch * a.k.heads * ((rows + MOE_TTC_ROWS - 1) / MOE_TTC_ROWS),
                         stream);
    }
    const TreeInstance &t = dev->inst[tree_choose(a.k.fmt, a.k.dim, rows)];
    // as many CTAs an SM as the registers allow while each ring keeps three stages (64 sequences of 4000 to 24000
    // tokens: three CTAs 264 us, two 324, one 511)
    const size_t list = 12 * ((size_t)batch + 1), used = t.fixed + list;
    int ctas = t.ctas, stages;
    for (;; --ctas) {
        const size_t room = std::min(dev->optin, dev->per_sm / ctas - 1024);
        stages = room > used ? (int)std::min<size_t>(8, (room - used) / t.stage) : 0;
        if (stages >= 3 || ctas == 1)
            break;
    }
    if (stages < 2)
        return host_fail(MOE_EUNSUPPORTED, "moe_tree_attention: %zu bytes of shared memory do not fit", used + 2 * t.stage);
    const int grid = std::min(dev->sms * ctas, MOE_TREE_MAX_GRID);
    SPEC_CUDA_OK(launch(t.kernel, dim3(grid), MOE_TREE_THREADS, used + stages * t.stage, stream, a, stages));
    return tree_join(a, *dev, grid, t.rows, (long long)batch * a.k.heads * ((rows + t.rows - 1) / t.rows), stream);
}

int moe_spec_verify_workspace_bytes(int batch, int n_rows, size_t *bytes)
{
    if (!bytes || batch < 0 || n_rows < 0)
        return host_fail(MOE_EINVAL, "moe_spec_verify_workspace_bytes: bad arguments");
    if (batch > 65535)
        return host_fail(MOE_EUNSUPPORTED, "batch (%d) <= 65535", batch);
    *bytes = SPEC_CTRL_BYTES + (size_t)n_rows * MOE_VERIFY_MAX_SPLITS * sizeof(VerifySlice);
    return MOE_OK;
}

int moe_spec_verify(const void *logits_dev, int logits_type, int64_t logits_stride, const int32_t *q_start_dev,
                    const int32_t *tokens_dev, const int32_t *parents_dev, const float *draft_dev, int64_t draft_stride,
                    const float *temperature_dev, const float *uniforms_dev, const float *noise_dev, int64_t noise_stride,
                    int batch, int n_rows, int vocab, int32_t *n_accepted_dev, int32_t *path_dev,
                    int32_t *next_token_dev, void *ws_dev, size_t ws_bytes, moe_stream_t stream)
{
    size_t need;
    int rc = moe_spec_verify_workspace_bytes(batch, n_rows, &need);
    if (rc)
        return rc;
    if (logits_type != MOE_BF16 && logits_type != MOE_F32)
        return host_fail(MOE_EINVAL, "moe_spec_verify: logits_type %d", logits_type);
    if (vocab < 1 || vocab > (1 << 24))
        return host_fail(vocab < 1 ? MOE_EINVAL : MOE_EUNSUPPORTED, "moe_spec_verify: vocab (%d) of 1 .. 2^24", vocab);
    if (batch == 0)
        return MOE_OK;
    if (!q_start_dev || !n_accepted_dev || !next_token_dev || !ws_dev ||
        (n_rows > 0 && (!logits_dev || !tokens_dev || !path_dev)))
        return host_fail(MOE_EINVAL, "moe_spec_verify: NULL argument");
    if (n_rows > 0 && (uniforms_dev == nullptr) != (noise_dev == nullptr))
        return host_fail(MOE_EINVAL, "moe_spec_verify: uniforms and noise go together");
    if (!aligned(logits_dev, logits_type == MOE_F32 ? 4 : 2) || !aligned(q_start_dev, 4) || !aligned(tokens_dev, 4) ||
        !aligned(parents_dev, 4) || !aligned(draft_dev, 4) || !aligned(temperature_dev, 4) || !aligned(uniforms_dev, 4) ||
        !aligned(noise_dev, 4) || !aligned(n_accepted_dev, 4) || !aligned(path_dev, 4) || !aligned(next_token_dev, 4) ||
        !aligned(ws_dev, 256))
        return host_fail(MOE_EINVAL, "moe_spec_verify: an argument is not aligned to its type, or ws_dev not to 256 bytes");
    if ((n_rows > 1 && (logits_stride < vocab || (draft_dev && draft_stride < vocab))) ||
        (batch > 1 && noise_dev && noise_stride < vocab))
        return host_fail(MOE_EINVAL, "moe_spec_verify: a row stride is below vocab (%d)", vocab);
    if (ws_bytes < need)
        return host_fail(MOE_EINVAL, "moe_spec_verify: the workspace holds %zu bytes, %zu are needed", ws_bytes, need);
    VerifyArgs a{};
    a.logits = logits_dev;
    a.stride = logits_stride;
    a.q_start = q_start_dev;
    a.tokens = tokens_dev;
    a.parents = parents_dev;
    a.draft = draft_dev;
    a.draft_stride = draft_stride;
    a.temperature = temperature_dev;
    a.uniforms = uniforms_dev;
    a.noise = noise_dev;
    a.noise_stride = noise_stride;
    a.rows = n_rows;
    a.vocab = vocab;
    a.n_accepted = n_accepted_dev;
    a.path = path_dev;
    a.next = next_token_dev;
    a.ctrl = static_cast<uint32_t *>(ws_dev);
    const bool f32 = logits_type == MOE_F32;
    const bool wide = aligned(logits_dev, 16) && logits_stride % (f32 ? 4 : 8) == 0 &&
                      (!draft_dev || (aligned(draft_dev, 16) && draft_stride % 4 == 0)) &&
                      (!noise_dev || (aligned(noise_dev, 16) && noise_stride % 4 == 0));
    // a cluster of CTAs a sequence: as many as are on the GPU together (three an SM; 512 chains of 3 drafts over 32000: 63
    // us, with eight CTAs each 93), with 2048 values a CTA at least (48 of 7 over 131072: 38 us, with one CTA each 99)
    const int ranks = std::max(1, std::min({MOE_VERIFY_MAX_CLUSTER, 456 / batch, vocab / 2048}));
    a.slice = ((vocab + ranks - 1) / ranks + 7) / 8 * 8;
    // all rows ahead where that is little, else as the walk reaches them
    const size_t all = (size_t)n_rows * vocab * (f32 ? 4 : 2);
    const bool ahead = n_rows > 0 && (all <= MOE_VERIFY_AHEAD_BYTES || !parents_dev);
    if (ahead) {
        a.batch = batch;
        // parts of 16384 values, of down to 2048 where the rows are few (4 rows of 32000: 7.2 us, as two parts 9.0; 384
        // of 131072: 38 us, in parts of 2048 109)
        a.splits = std::max(1, std::min({MOE_VERIFY_MAX_SPLITS, vocab / 2048, std::max(608 / n_rows, vocab / 16384)}));
        a.split = ((vocab + a.splits - 1) / a.splits + 7) / 8 * 8;
        a.stats = reinterpret_cast<VerifySlice *>(static_cast<char *>(ws_dev) + SPEC_CTRL_BYTES);
        const auto rows = f32 ? (wide ? moe_verify_rows_kernel<true, true> : moe_verify_rows_kernel<true, false>)
                              : (wide ? moe_verify_rows_kernel<false, true> : moe_verify_rows_kernel<false, false>);
        SPEC_CUDA_OK(launch(rows, dim3((unsigned)n_rows * a.splits), MOE_VERIFY_STAT_THREADS, 0, stream, a));
    }
    const auto kernel = verify_kernel(f32, wide, ahead);
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)batch * ranks);
    lc.blockDim = dim3(MOE_VERIFY_THREADS);
    lc.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 2;
    SPEC_CUDA_OK(cudaLaunchKernelEx(&lc, kernel, a));
    return MOE_OK;
}

}  // extern "C"

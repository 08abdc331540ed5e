// moe_latent.cu -- the entry points of libmoe.so for rotary positions, the cache
// of latent vectors and attention over it (declared and documented in
// include/moe.h). Argument checks, workspace layout and launches.
#include <math.h>

#include <algorithm>
#include <mutex>

#include "moe_latent_tc.cuh"
#include "moe_launch.cuh"
#include "moe_prompt.cuh"

using namespace moe;

namespace {

#define LATENT_CTRL_BYTES 256  // control words: the status is word MOE_CTRL_STATUS

int check_shape(const moe_latent_cache *c)
{
    if (!c)
        return host_fail(MOE_EINVAL, "cache is NULL");
    if (c->latent_dim < 1 || c->rope_dim < 1 || c->page_size < 1)
        return host_fail(MOE_EINVAL, "latent_dim (%d), rope_dim (%d) and page_size (%d) must be positive", c->latent_dim,
                         c->rope_dim, c->page_size);
    if ((c->latent_dim != 128 && c->latent_dim != 256 && c->latent_dim != 512) || c->rope_dim % 8 || c->rope_dim > 64 ||
        c->page_size % 16 || c->page_size > 1024)
        return host_fail(MOE_EUNSUPPORTED, "latent_dim (%d) of 128, 256 or 512, rope_dim (%d) a multiple of 8 up to 64, "
                         "page_size (%d) a multiple of 16 up to 1024", c->latent_dim, c->rope_dim, c->page_size);
    return MOE_OK;
}

int check_cache(const moe_latent_cache *c)
{
    const int rc = check_shape(c);
    if (rc)
        return rc;
    if (!c->pages || !aligned(c->pages, 16))
        return host_fail(MOE_EINVAL, "the cache's pages are NULL or not 16-byte aligned");
    if (c->n_pages < 1 || c->n_pages > 0x7FFFFFFFll / c->page_size)
        return host_fail(MOE_EINVAL, "n_pages (%lld) must be positive and n_pages * page_size below 2^31",
                         (long long)c->n_pages);
    return MOE_OK;
}

bool wide_rows(const void *p, int64_t s0, int64_t s1) { return aligned(p, 16) && (s0 | s1) % 8 == 0; }

// rows of the latent cache, in or out
int latent_rows(bool read, LatentRows &a, const moe_latent_cache *cache, moe_stream_t stream)
{
    a.pages = static_cast<uint16_t *>(cache->pages);
    a.n_slots = cache->n_pages * cache->page_size;
    a.latent = cache->latent_dim;
    a.rope = cache->rope_dim;
    a.c_wide = wide_rows(a.c, a.c_stride, 0);
    a.kr_wide = wide_rows(a.kr, a.kr_stride, 0);
    const long long per = MOE_LATENT_PIECES * MOE_LATENT_THREADS, n = a.tokens;
    a.c_blocks = (unsigned)((n * (a.latent / 8) + per - 1) / per);
    const dim3 grid(a.c_blocks + (unsigned)((n * (a.rope / 8) + per - 1) / per));
    MOE_CUDA_OK(launch(read ? moe_latent_rows_kernel<true> : moe_latent_rows_kernel<false>, grid, MOE_LATENT_THREADS, 0,
                       stream, a));
    return MOE_OK;
}

// ---- absorbed attention: instances, maps of the cache, the join of cut items

#define MOE_LTC_MAX_PAIRS 80  // the workspace holds two partials each
#define MOE_LATENT_MAX_DEVICES 64

std::mutex g_latent_mu;

struct LatentInstance {
    void (*kernel)(LatentArgs, int);
    size_t fixed, stage;  // bytes of shared memory beside the ring and the list; of a stage
    void (*join)(TreeArgs), (*join_long)(TreeArgs, int, int);  // of many items, of few long ones
};

template <int L>
LatentInstance latent_instance()
{
    using T = LtcShape<L>;
    return {moe_latent_tc_kernel<L>, (size_t)T::RING_AT + T::SMALL, (size_t)T::STAGE,
            moe_latent_join_kernel<L>, moe_tree_join_kernel<L, 256, 8, 8>};
}

struct LatentDevice {
    int pairs = 0;
    size_t optin = 0;
    LatentInstance inst[3];
};

int latent_device(LatentDevice **out)
{
    static LatentDevice dev[MOE_LATENT_MAX_DEVICES];
    int d = 0;
    MOE_CUDA_OK(cudaGetDevice(&d));
    if (d < 0 || d >= MOE_LATENT_MAX_DEVICES)
        return host_fail(MOE_EUNSUPPORTED, "device ordinal %d", d);
    std::lock_guard<std::mutex> lk(g_latent_mu);
    LatentDevice &D = dev[d];
    if (!D.pairs) {
        int n = 0, optin = 0;
        MOE_CUDA_OK(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, d));
        MOE_CUDA_OK(cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, d));
        const LatentInstance all[3] = {latent_instance<128>(), latent_instance<256>(), latent_instance<512>()};
        for (int i = 0; i < 3; ++i) {
            MOE_CUDA_OK(cudaFuncSetAttribute(all[i].kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin));
            D.inst[i] = all[i];
        }
        D.optin = optin;
        D.pairs = std::min(n / 2, MOE_LTC_MAX_PAIRS);
    }
    *out = &D;
    return MOE_OK;
}

// the cache's rows as tensor maps: boxes of 32 tokens and all chunks of 64 dimensions where pages are of whole 32
// tokens, else of 16 tokens and a chunk
int latent_maps(const moe_latent_cache *c, LatentArgs &a)
{
    const uint64_t row = 2ull * (c->latent_dim + c->rope_dim), slots = (uint64_t)c->n_pages * c->page_size;
    const uint32_t chunks = c->latent_dim / 64, tokens = a.big ? 32 : 16;
    const uint64_t dims[3] = {64, slots, chunks}, strides[2] = {row, 128};
    const uint64_t rope_dims[2] = {(uint64_t)c->rope_dim, slots};
    const uint32_t keys[3] = {64, tokens, a.big ? chunks : 1}, values[3] = {64, tokens, a.big ? chunks / 2 : 1};
    const uint32_t ropes[2] = {64, tokens};
    int rc = host_map_bf16(&a.keys, c->pages, 3, dims, strides, keys);
    if (!rc)
        rc = host_map_bf16(&a.values, c->pages, 3, dims, strides, values);
    if (!rc)
        rc = host_map_bf16(&a.ropes, static_cast<const char *>(c->pages) + 2 * c->latent_dim, 2, rope_dims, strides, ropes);
    return rc;
}

// ---- expanded attention

#define MOE_PROMPT_SMALL 512  // bytes of shared memory beside the queries and the ring

// rows [tokens, heads, dims] as a tensor map: boxes of `box` tokens of one head and 64 dimensions
int prompt_map(CUtensorMap *m, const void *base, int64_t token_stride, int64_t head_stride, int tokens, int heads, int dims,
               uint32_t box)
{
    const bool one = heads == 1 || head_stride == 0;
    const uint64_t size[3] = {(uint64_t)dims, one ? 1ull : (uint64_t)heads, (uint64_t)tokens};
    const uint64_t strides[2] = {one ? 16ull : 2 * (uint64_t)head_stride, tokens == 1 ? 16ull : 2 * (uint64_t)token_stride};
    const uint32_t boxes[3] = {64, 1, box};
    return host_map_bf16(m, base, 3, size, strides, boxes);
}

struct PromptDevice {
    int sms = 0;
    int clusters[2][4];  // [nope_dim 64, 128][i]: clusters of 2^i CTAs that run at once (i 1 to 3)
};

size_t prompt_shared(int nope_dim) { return (2 * (nope_dim / 64 + 1) + MOE_PROMPT_PLACES) * (size_t)MOE_PROMPT_PLACE + MOE_PROMPT_SMALL; }

// the kernel's launch: clusters of `split` CTAs
struct PromptLaunch {
    cudaLaunchConfig_t lc{};
    cudaLaunchAttribute at[2];
    PromptLaunch(dim3 grid, int nope_dim, int split, moe_stream_t stream)
    {
        lc.gridDim = grid;
        lc.blockDim = dim3(MOE_PROMPT_THREADS);
        lc.dynamicSmemBytes = prompt_shared(nope_dim);
        lc.stream = (cudaStream_t)stream;
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = split;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        lc.attrs = at;
        lc.numAttrs = split > 1 ? 2 : 1;
    }
};

// shared memory of the kernel, and what of it runs at once, asked for once a device
int prompt_device(PromptDevice **out)
{
    static PromptDevice dev[MOE_LATENT_MAX_DEVICES];
    int d = 0, optin = 0, sms = 0;
    MOE_CUDA_OK(cudaGetDevice(&d));
    if (d < 0 || d >= MOE_LATENT_MAX_DEVICES)
        return host_fail(MOE_EUNSUPPORTED, "device ordinal %d", d);
    std::lock_guard<std::mutex> lk(g_latent_mu);
    PromptDevice &D = dev[d];
    if (!D.sms) {
        MOE_CUDA_OK(cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, d));
        MOE_CUDA_OK(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d));
        for (int k = 0; k < 2; ++k) {
            const auto kernel = k ? moe_prompt_kernel<128> : moe_prompt_kernel<64>;
            MOE_CUDA_OK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin));
            for (int i = 1; i < 4; ++i) {
                PromptLaunch l(dim3(1u << i), 64 << k, 1 << i, nullptr);
                MOE_CUDA_OK(cudaOccupancyMaxActiveClusters(&D.clusters[k][i], kernel, &l.lc));
            }
        }
        D.sms = sms;
    }
    *out = &D;
    return MOE_OK;
}

using RopeKernel = void (*)(RopeArgs);

template <bool F32, bool WIDE>
RopeKernel rope_kernel(bool inter)
{
    return inter ? moe_rope_kernel<F32, WIDE, true> : moe_rope_kernel<F32, WIDE, false>;
}

}  // namespace

extern "C" {

int moe_rope_table(const moe_rope_cfg *cfg, uint64_t *table_host, float *magnitude_host)
{
    if (!cfg || !table_host)
        return host_fail(MOE_EINVAL, "moe_rope_table: NULL argument");
    const int dim = cfg->dim;
    if (dim < 2 || dim % 2)
        return host_fail(MOE_EINVAL, "moe_rope_table: dim (%d) must be even and positive", dim);
    if (dim > 1024)
        return host_fail(MOE_EUNSUPPORTED, "moe_rope_table: dim (%d) <= 1024", dim);
    if (cfg->scaling < MOE_ROPE_PLAIN || cfg->scaling > MOE_ROPE_PARTS)
        return host_fail(MOE_EINVAL, "moe_rope_table: scaling %d", cfg->scaling);
    const bool scaled = cfg->scaling != MOE_ROPE_PLAIN, parts = cfg->scaling == MOE_ROPE_PARTS;
    if (!(cfg->base >= 1.0 && cfg->base < 1e30) || (scaled && !(cfg->factor >= 1.0 && cfg->factor < 1e30)))
        return host_fail(MOE_EINVAL, "moe_rope_table: base (%g) and factor (%g) must be at least 1 and finite", cfg->base,
                         cfg->factor);
    if (cfg->scaling == MOE_ROPE_BASE && dim == 2)
        return host_fail(MOE_EINVAL, "moe_rope_table: dim 2 has no base to scale");
    if (parts && !(cfg->slow >= 0.0 && cfg->fast > cfg->slow && cfg->fast < 1e30 && cfg->original > 0.0 &&
                   cfg->original < 1e30))
        return host_fail(MOE_EINVAL, "moe_rope_table: 0 <= slow (%g) < fast (%g) and original (%g) > 0", cfg->slow,
                         cfg->fast, cfg->original);
    const double turn = 6.283185307179586476925286766559;
    const double base = cfg->scaling == MOE_ROPE_BASE ? cfg->base * pow(cfg->factor, (double)dim / (dim - 2)) : cfg->base;
    for (int i = 0; i < dim / 2; ++i) {
        double f = pow(base, -2.0 * i / dim);
        if (cfg->scaling == MOE_ROPE_LINEAR)
            f /= cfg->factor;
        if (parts) {
            const double r = cfg->original * f / turn;
            const double k = std::min(std::max((r - cfg->slow) / (cfg->fast - cfg->slow), 0.0), 1.0);
            f *= k + (1.0 - k) / cfg->factor;
        }
        table_host[i] = (uint64_t)rint(f / turn * 18446744073709551616.0);  // below 2^62: f is 1 at most
    }
    if (magnitude_host)
        *magnitude_host = parts ? (float)(0.1 * log(cfg->factor) + 1.0) : 1.0f;
    return MOE_OK;
}

int moe_rope(const void *x_dev, int64_t x_token_stride, int64_t x_head_stride, void *out_dev, int64_t out_token_stride,
             int64_t out_head_stride, int type, int tokens, int heads, int head_dim, int offset, int rope_dim, int layout,
             const int32_t *positions_dev, const uint64_t *table_dev, float magnitude, int transposed, moe_stream_t stream)
{
    if (type != MOE_BF16 && type != MOE_F32)
        return host_fail(MOE_EINVAL, "moe_rope: type %d", type);
    if (layout != MOE_ROPE_HALF && layout != MOE_ROPE_INTERLEAVED)
        return host_fail(MOE_EINVAL, "moe_rope: layout %d", layout);
    if (tokens < 0 || heads < 0 || head_dim < 1 || offset < 0 || rope_dim < 2 || rope_dim % 2 || rope_dim > head_dim ||
        offset > head_dim - rope_dim)
        return host_fail(MOE_EINVAL, "moe_rope: tokens (%d) and heads (%d) must not be negative, rope_dim (%d) even, from 2 "
                         "to head_dim (%d) - offset (%d)", tokens, heads, rope_dim, head_dim, offset);
    if (head_dim > 1024 || heads > 65536)
        return host_fail(MOE_EUNSUPPORTED, "moe_rope: head_dim (%d) <= 1024, heads (%d) <= 65536", head_dim, heads);
    if (!(magnitude >= -3.0e38f && magnitude <= 3.0e38f))
        return host_fail(MOE_EINVAL, "moe_rope: magnitude must be finite");
    if (tokens == 0 || heads == 0)
        return MOE_OK;
    if (!x_dev || !out_dev || !positions_dev || !table_dev)
        return host_fail(MOE_EINVAL, "moe_rope: NULL argument");
    const bool f32 = type == MOE_F32;
    const int size = f32 ? 4 : 2;
    if (!aligned(x_dev, size) || !aligned(out_dev, size) || !aligned(positions_dev, 4) || !aligned(table_dev, 8))
        return host_fail(MOE_EINVAL, "moe_rope: an argument is not aligned to its type");
    const bool in_place = x_dev == out_dev;
    if (in_place && ((tokens > 1 && x_token_stride != out_token_stride) || (heads > 1 && x_head_stride != out_head_stride)))
        return host_fail(MOE_EINVAL, "moe_rope: in place, the strides of x and out must be the same");
    const bool inter = layout == MOE_ROPE_INTERLEAVED;
    const int v = 16 / size;
    const bool wide = aligned(x_dev, 16) && aligned(out_dev, 16) && head_dim % v == 0 && offset % v == 0 &&
                      (inter ? rope_dim : rope_dim / 2) % v == 0 &&
                      (x_token_stride | x_head_stride | out_token_stride | out_head_stride) % v == 0;
    RopeArgs a{};
    a.x = x_dev;
    a.out = out_dev;
    a.x_tok = x_token_stride;
    a.x_head = x_head_stride;
    a.o_tok = out_token_stride;
    a.o_head = out_head_stride;
    a.tokens = tokens;
    a.heads = heads;
    a.dim = head_dim;
    a.offset = offset;
    a.rope = rope_dim;
    a.positions = positions_dev;
    a.table = reinterpret_cast<const unsigned long long *>(table_dev);
    a.magnitude = magnitude;
    a.sign = transposed ? -1.0f : 1.0f;
    a.turned = wide ? (inter ? rope_dim : rope_dim / 2) / v : rope_dim / 2;
    a.items = a.turned + (in_place ? 0 : (head_dim - rope_dim) / (wide ? v : 1));
    a.heads_cta = std::min(heads, MOE_ROPE_HEADS);
    // a CTA some 2048 pieces (16384 tokens of 32 heads in bf16 and 4099 of 12 in f32: 67.2 and 10.9 us; 1024: 75.9 and 14.2;
    // 4096: 67.1 and 12.0), but four CTAs an SM first (8 tokens of 40 heads in a graph 2.1 us, else 4.7; 2000 of one head 2.1
    // and 5.3)
    const long long per = (long long)a.heads_cta * a.items;
    a.tokens_cta = (int)std::max(1ll, std::min({2048 / per, tokens / 608ll, MOE_ROPE_SMEM / (4ll * rope_dim)}));
    const dim3 grid((unsigned)(((long long)tokens + a.tokens_cta - 1) / a.tokens_cta),
                    (unsigned)((heads + a.heads_cta - 1) / a.heads_cta));
    const RopeKernel kernel = f32 ? (wide ? rope_kernel<true, true>(inter) : rope_kernel<true, false>(inter))
                                  : (wide ? rope_kernel<false, true>(inter) : rope_kernel<false, false>(inter));
    MOE_CUDA_OK(launch(kernel, grid, MOE_ROPE_THREADS, (size_t)a.tokens_cta * rope_dim * 4, stream, a));
    return MOE_OK;
}

int moe_latent_page_bytes(const moe_latent_cache *cache, size_t *bytes)
{
    const int rc = check_shape(cache);
    if (rc)
        return rc;
    if (!bytes)
        return host_fail(MOE_EINVAL, "bytes is NULL");
    *bytes = (size_t)cache->page_size * (cache->latent_dim + cache->rope_dim) * 2;
    return MOE_OK;
}

int moe_latent_append(const moe_latent_cache *cache, const void *c_dev, int64_t c_stride, const void *kr_dev,
                      int64_t kr_stride, const int32_t *slots_dev, int n_tokens, const int32_t *positions_dev,
                      const uint64_t *table_dev, int layout, float magnitude, uint32_t *status_dev, moe_stream_t stream)
{
    const int rc = check_cache(cache);
    if (rc)
        return rc;
    if (n_tokens < 0 || (n_tokens > 0 && (!c_dev || !kr_dev || !slots_dev)))
        return host_fail(MOE_EINVAL, "moe_latent_append: NULL argument or n_tokens (%d) < 0", n_tokens);
    if ((positions_dev == nullptr) != (table_dev == nullptr))
        return host_fail(MOE_EINVAL, "moe_latent_append: positions and table go together");
    if (layout != MOE_ROPE_HALF && layout != MOE_ROPE_INTERLEAVED)
        return host_fail(MOE_EINVAL, "moe_latent_append: layout %d", layout);
    if (!(magnitude >= -3.0e38f && magnitude <= 3.0e38f))
        return host_fail(MOE_EINVAL, "moe_latent_append: magnitude must be finite");
    if (!aligned(c_dev, 2) || !aligned(kr_dev, 2) || !aligned(slots_dev, 4) || !aligned(positions_dev, 4) ||
        !aligned(table_dev, 8) || !aligned(status_dev, 4))
        return host_fail(MOE_EINVAL, "moe_latent_append: an argument is not aligned to its type");
    if (n_tokens == 0)
        return MOE_OK;
    LatentRows a{};
    a.c = static_cast<uint16_t *>(const_cast<void *>(c_dev));
    a.kr = static_cast<uint16_t *>(const_cast<void *>(kr_dev));
    a.c_stride = c_stride;
    a.kr_stride = kr_stride;
    a.slots = slots_dev;
    a.tokens = n_tokens;
    a.positions = positions_dev;
    a.table = reinterpret_cast<const unsigned long long *>(table_dev);
    a.layout = layout;
    a.magnitude = magnitude;
    a.status = status_dev;
    return latent_rows(false, a, cache, stream);
}

int moe_latent_read(const moe_latent_cache *cache, const int32_t *slots_dev, int n_tokens, void *c_out_dev,
                    int64_t c_stride, void *kr_out_dev, int64_t kr_stride, uint32_t *status_dev, moe_stream_t stream)
{
    const int rc = check_cache(cache);
    if (rc)
        return rc;
    if (n_tokens < 0 || (n_tokens > 0 && (!c_out_dev || !kr_out_dev || !slots_dev)))
        return host_fail(MOE_EINVAL, "moe_latent_read: NULL argument or n_tokens (%d) < 0", n_tokens);
    if (!aligned(c_out_dev, 2) || !aligned(kr_out_dev, 2) || !aligned(slots_dev, 4) || !aligned(status_dev, 4))
        return host_fail(MOE_EINVAL, "moe_latent_read: an argument is not aligned to its type");
    if (n_tokens > 1 && (c_stride < cache->latent_dim || kr_stride < cache->rope_dim))
        return host_fail(MOE_EINVAL, "moe_latent_read: a row stride is below the row's length");
    if (n_tokens == 0)
        return MOE_OK;
    LatentRows a{};
    a.c = static_cast<uint16_t *>(c_out_dev);
    a.kr = static_cast<uint16_t *>(kr_out_dev);
    a.c_stride = c_stride;
    a.kr_stride = kr_stride;
    a.slots = slots_dev;
    a.tokens = n_tokens;
    a.status = status_dev;
    return latent_rows(true, a, cache, stream);
}

static int latent_ws(const moe_latent_cache *cache, int heads, int batch, int n_tokens, size_t &bytes)
{
    const int rc = check_shape(cache);
    if (rc)
        return rc;
    if (heads < 1 || batch < 0 || n_tokens < 0)
        return host_fail(MOE_EINVAL, "heads (%d) must be positive, batch (%d) and n_tokens (%d) not negative", heads, batch,
                         n_tokens);
    if (heads > 128 || batch > 1024 || n_tokens > batch * MOE_MAX_DRAFT)
        return host_fail(MOE_EUNSUPPORTED, "heads (%d) <= 128, batch (%d) <= 1024, n_tokens (%d) <= %d a sequence", heads,
                         batch, n_tokens, MOE_MAX_DRAFT);
    // control words, cuts, and two partials of a row block a run
    bytes = LATENT_CTRL_BYTES + sizeof(TreeCut) * MOE_LTC_MAX_PAIRS +
            (size_t)MOE_LTC_MAX_PAIRS * 2 * MOE_LTC_ROWS * 4 * (cache->latent_dim + 2);
    return MOE_OK;
}

int moe_latent_attention_workspace_bytes(const moe_latent_cache *cache, int heads, int batch, int n_tokens, size_t *bytes)
{
    if (!bytes)
        return host_fail(MOE_EINVAL, "bytes is NULL");
    return latent_ws(cache, heads, batch, n_tokens, *bytes);
}

int moe_latent_attention(const moe_latent_cache *cache, const void *q_dev, int64_t q_token_stride, int64_t q_head_stride,
                         const void *qr_dev, int64_t qr_token_stride, int64_t qr_head_stride, void *out_dev,
                         int64_t out_token_stride, int64_t out_head_stride, int heads, const int32_t *q_start_dev,
                         const int32_t *kv_len_dev, const int32_t *table_dev, int64_t table_stride, int table_pages,
                         const uint64_t *mask_dev, int batch, int n_tokens, float scale, void *ws_dev, size_t ws_bytes,
                         moe_stream_t stream)
{
    int rc = check_cache(cache);
    if (rc)
        return rc;
    size_t need;
    if ((rc = latent_ws(cache, heads, batch, n_tokens, need)))
        return rc;
    if (batch == 0 || n_tokens == 0)
        return MOE_OK;
    if (!q_dev || !qr_dev || !out_dev || !q_start_dev || !kv_len_dev || !table_dev || !ws_dev)
        return host_fail(MOE_EINVAL, "moe_latent_attention: NULL argument");
    if (!aligned(q_dev, 2) || !aligned(qr_dev, 2) || !aligned(out_dev, 2) || !aligned(q_start_dev, 4) ||
        !aligned(kv_len_dev, 4) || !aligned(table_dev, 4) || !aligned(mask_dev, 8) || !aligned(ws_dev, 256))
        return host_fail(MOE_EINVAL, "moe_latent_attention: an argument is not aligned to its type, or ws_dev not to 256 "
                         "bytes");
    if (ws_bytes < need)
        return host_fail(MOE_EINVAL, "moe_latent_attention: the workspace holds %zu bytes, %zu are needed", ws_bytes, need);
    if (table_pages < 1 || (batch > 1 && table_stride < table_pages) || !(scale >= -3.0e38f && scale <= 3.0e38f))
        return host_fail(MOE_EINVAL, "moe_latent_attention: table_pages (%d) must be positive and at most table_stride "
                         "(%lld), scale finite", table_pages, (long long)table_stride);
    LatentArgs a{};
    TreeArgs &t = a.t;
    t.k = {cache->latent_dim, 1, cache->page_size, 0};
    t.pages = static_cast<const uint8_t *>(cache->pages);
    t.n_pages = (int)cache->n_pages;
    t.q = static_cast<const uint16_t *>(q_dev);
    t.q_tok = q_token_stride;
    t.q_head = q_head_stride;
    a.qr = static_cast<const uint16_t *>(qr_dev);
    a.qr_tok = qr_token_stride;
    a.qr_head = qr_head_stride;
    a.rope = cache->rope_dim;
    t.out = static_cast<uint16_t *>(out_dev);
    t.o_tok = out_token_stride;
    t.o_head = out_head_stride;
    t.q_start = q_start_dev;
    t.kv_len = kv_len_dev;
    t.table = table_dev;
    t.table_stride = table_stride;
    t.max_len = (int)std::min((long long)table_pages * t.k.page, (long long)MOE_TREE_MAX_LEN);
    t.mask = reinterpret_cast<const unsigned long long *>(mask_dev);
    t.batch = batch;
    t.tokens = n_tokens;
    t.group = heads;
    // exponents of 2 are scores (of the scale's sign) times join_c; where the scale is too small for that, all alike
    const float c = std::min(fabsf(scale) * 1.4426950408889634f, 3.0e38f);
    t.scale = c == 0.0f ? 0.0f : scale;
    t.join_c = c == 0.0f ? 1.0f : c;
    t.q_wide = wide_rows(q_dev, q_token_stride, q_head_stride);
    a.qr_wide = wide_rows(qr_dev, qr_token_stride, qr_head_stride);
    t.o_wide = wide_rows(out_dev, out_token_stride, out_head_stride);
    t.min_units = 2;  // (one sequence of 4000 tokens: 18.3 us, with one tile a run 20.7)
    t.ctrl = static_cast<uint32_t *>(ws_dev);
    t.cuts = reinterpret_cast<TreeCut *>(t.ctrl + LATENT_CTRL_BYTES / 4);
    t.part = reinterpret_cast<float *>(t.cuts + MOE_LTC_MAX_PAIRS);
    t.wait_ns = host_wait_ns();
    a.big = t.k.page % 32 == 0;
    a.per_page = ((1ull << 36) + t.k.page / 16 - 1) / (t.k.page / 16);
    if ((rc = latent_maps(cache, a)))
        return rc;
    LatentDevice *dev;
    if ((rc = latent_device(&dev)))
        return rc;
    const int latent = cache->latent_dim;
    const LatentInstance &inst = dev->inst[latent == 128 ? 0 : latent == 256 ? 1 : 2];
    const size_t used = inst.fixed + 12 * ((size_t)batch + 1);
    const int stages = (int)std::min<size_t>(MOE_LTC_MAX_STAGES, (dev->optin - used) / inst.stage);
    cudaLaunchConfig_t lc{};
    lc.gridDim = dim3((unsigned)dev->pairs * 2);
    lc.blockDim = dim3(MOE_LTC_THREADS);
    lc.dynamicSmemBytes = used + stages * inst.stage;
    lc.stream = (cudaStream_t)stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    lc.attrs = at;
    lc.numAttrs = 2;
    MOE_CUDA_OK(cudaLaunchKernelEx(&lc, inst.kernel, a, stages));
    // the join, by the parts that an item may have: of a run each, and of two tiles (one sequence of 511 tokens and 128 heads,
    // 8 parts: 19 us by the one, 26 by the other; of 100003 and 16 heads, 76 parts: 53 and 42)
    const int rows = (n_tokens + batch - 1) / batch * heads, runs = dev->pairs;
    const long long items = (long long)batch * ((rows + MOE_LTC_ROWS - 1) / MOE_LTC_ROWS);
    if (std::min(runs / items, (long long)t.max_len / (2 * MOE_LTC_TOKENS) + 1) >= 24) {
        const int blocks = std::min((rows + MOE_TREE_JOIN_ROWS - 1) / MOE_TREE_JOIN_ROWS, MOE_LTC_ROWS / MOE_TREE_JOIN_ROWS);
        const dim3 grid((unsigned)runs, (unsigned)(batch == 1 ? blocks : MOE_LTC_ROWS / MOE_TREE_JOIN_ROWS),
                        (unsigned)(latent / 32));
        MOE_CUDA_OK(launch(inst.join_long, grid, 256, 0, stream, t, MOE_LTC_ROWS, runs));
    } else {
        MOE_CUDA_OK(launch(inst.join, dim3((unsigned)runs, (unsigned)(latent / 32)), MOE_LTC_JOIN_THREADS, 0, stream, t));
    }
    return MOE_OK;
}

int moe_latent_prompt_attention(const void *q_dev, int64_t q_token_stride, int64_t q_head_stride, const void *k_dev,
                                int64_t k_token_stride, int64_t k_head_stride, const void *kr_dev, int64_t kr_stride,
                                const void *v_dev, int64_t v_token_stride, int64_t v_head_stride, void *out_dev,
                                int64_t out_token_stride, int64_t out_head_stride, int heads, int nope_dim, int rope_dim,
                                const int32_t *q_start_dev, const int32_t *kv_start_dev, int batch, int q_tokens,
                                int kv_tokens, int causal, float scale, uint32_t *status_dev, moe_stream_t stream)
{
    if (heads < 1 || nope_dim < 1 || rope_dim < 1 || batch < 0 || q_tokens < 0 || kv_tokens < 0)
        return host_fail(MOE_EINVAL, "moe_latent_prompt_attention: heads (%d), nope_dim (%d) and rope_dim (%d) must be "
                         "positive, batch (%d), q_tokens (%d) and kv_tokens (%d) not negative", heads, nope_dim, rope_dim,
                         batch, q_tokens, kv_tokens);
    if ((nope_dim != 64 && nope_dim != 128) || rope_dim % 8 || rope_dim > 64 || heads > 1024 || batch > 1024)
        return host_fail(MOE_EUNSUPPORTED, "moe_latent_prompt_attention: nope_dim (%d) of 64 or 128, rope_dim (%d) a "
                         "multiple of 8 up to 64, heads (%d) and batch (%d) <= 1024", nope_dim, rope_dim, heads, batch);
    if (q_tokens > 1 << 23 || kv_tokens > 1 << 30)
        return host_fail(MOE_EUNSUPPORTED, "moe_latent_prompt_attention: q_tokens (%d) <= 2^23, kv_tokens (%d) <= 2^30", q_tokens,
                         kv_tokens);
    if (!(scale >= -3.0e38f && scale <= 3.0e38f))
        return host_fail(MOE_EINVAL, "moe_latent_prompt_attention: scale must be finite");
    if (batch == 0 || q_tokens == 0)
        return MOE_OK;
    if (!q_dev || !out_dev || !q_start_dev || !kv_start_dev || (kv_tokens > 0 && (!k_dev || !kr_dev || !v_dev)))
        return host_fail(MOE_EINVAL, "moe_latent_prompt_attention: NULL argument");
    if (!aligned(q_dev, 2) || !aligned(out_dev, 2) || !aligned(q_start_dev, 4) || !aligned(kv_start_dev, 4) ||
        !aligned(status_dev, 4))
        return host_fail(MOE_EINVAL, "moe_latent_prompt_attention: an argument is not aligned to its type");
    if (!aligned(k_dev, 16) || !aligned(kr_dev, 16) || !aligned(v_dev, 16) ||
        (k_token_stride | k_head_stride | kr_stride | v_token_stride | v_head_stride) % 8)
        return host_fail(MOE_EINVAL, "moe_latent_prompt_attention: k, kr and v must start on 16-byte boundaries and have "
                         "strides of multiples of 8");
    if (kv_tokens > 1 && (k_token_stride < 1 || kr_stride < 1 || v_token_stride < 1))
        return host_fail(MOE_EINVAL, "moe_latent_prompt_attention: k's, kr's and v's token strides must be positive");
    if (heads > 1 && (k_head_stride < 0 || v_head_stride < 0))
        return host_fail(MOE_EINVAL, "moe_latent_prompt_attention: k's and v's head strides must not be negative");
    PromptArgs a{};
    a.q = static_cast<const uint16_t *>(q_dev);
    a.v = static_cast<const uint16_t *>(v_dev);
    a.out = static_cast<uint16_t *>(out_dev);
    a.q_tok = q_token_stride;
    a.q_head = q_head_stride;
    a.v_tok = v_token_stride;
    a.v_head = v_head_stride;
    a.o_tok = out_token_stride;
    a.o_head = out_head_stride;
    a.q_start = q_start_dev;
    a.kv_start = kv_start_dev;
    a.batch = batch;
    a.rope = rope_dim;
    a.q_tokens = q_tokens;
    a.kv_tokens = kv_tokens;
    a.causal = causal;
    // (TMA takes the queries where it can)
    a.q_wide = wide_rows(q_dev, q_token_stride, q_head_stride) && (q_tokens == 1 || q_token_stride > 0) &&
               (heads == 1 || q_head_stride > 0);
    a.o_wide = !wide_rows(out_dev, out_token_stride, out_head_stride) ? 0
               : aligned(out_dev, 32) && (out_token_stride | out_head_stride) % 16 == 0 ? 2 : 1;
    a.one_k = heads == 1 || k_head_stride == 0;
    a.one_v = heads == 1 || v_head_stride == 0;
    a.scale = scale;
    a.status = status_dev;
    a.wait_ns = host_wait_ns();
    int rc = MOE_OK;
    if (kv_tokens > 0) {
        const uint64_t dims[2] = {(uint64_t)rope_dim, (uint64_t)kv_tokens}, strides[1] = {kv_tokens == 1 ? 16ull : 2 * (uint64_t)kr_stride};
        const uint32_t box[2] = {64, MOE_PROMPT_TOKENS};
        if ((rc = prompt_map(&a.keys, k_dev, k_token_stride, k_head_stride, kv_tokens, heads, nope_dim, MOE_PROMPT_TOKENS)) ||
            (rc = prompt_map(&a.values, v_dev, v_token_stride, v_head_stride, kv_tokens, heads, nope_dim,
                             MOE_PROMPT_TOKENS / (nope_dim / 64))) ||
            (rc = host_map_bf16(&a.ropes, kr_dev, 2, dims, strides, box)))
            return rc;
    }
    if (a.q_wide && (rc = prompt_map(&a.queries, q_dev, q_token_stride, q_head_stride, q_tokens, heads, nope_dim + rope_dim, 128)))
        return rc;
    PromptDevice *dev;
    if ((rc = prompt_device(&dev)))
        return rc;
    // Where blocks are few, clusters share each one's tokens, as far as the clusters run at once (128 rows of 4 heads after 30000
    // tokens: 63 us, by a CTA a block 385; 512 of 32 after 16000: 139 and 252; 128 of 19 after 8000 by clusters of 4: 39.5 us, by
    // 19 of 8, some of which wait for others' end, 54); but parts of two tiles at least, and of 6
    // where a CTA to every 128 rows does instead (512 rows of 16 heads, no tokens before: 15 us, shared out 19; 2048 of 8: 34
    // and 30.5): so too where the SMs are enough for that alone (1024 rows of 16: 22 us, 26 with 256 a CTA). (How the rows
    // are spread over the sequences is not known here: blocks that end short of 256 rows count for less than they are.)
    const long long blocks = (long long)heads * std::max((q_tokens + MOE_PROMPT_ROWS - 1) / MOE_PROMPT_ROWS, std::min(batch, q_tokens));
    const int least = (q_tokens <= (long long)batch * (MOE_PROMPT_ROWS / 2) ? 2 : 6) * MOE_PROMPT_TOKENS;
    a.split = 1;
    for (int i = 1; a.split * 2 <= std::min(MOE_PROMPT_SPLIT, nope_dim / 16) && blocks <= dev->clusters[nope_dim / 128][i] &&
                    kv_tokens >= (long long)batch * a.split * 2 * least;
         ++i)
        a.split *= 2;
    a.block = a.split == 1 && (long long)heads * ((q_tokens + 127) / 128) <= dev->sms ? MOE_PROMPT_ROWS / 2 : MOE_PROMPT_ROWS;
    const PromptLaunch l(dim3((unsigned)(heads * a.split), (unsigned)(q_tokens / a.block + batch)), nope_dim, a.split, stream);
    MOE_CUDA_OK(cudaLaunchKernelEx(&l.lc, nope_dim == 64 ? moe_prompt_kernel<64> : moe_prompt_kernel<128>, a));
    return MOE_OK;
}

}  // extern "C"

/*
 * moe.h -- C ABI of libmoe.so, the GB300 (sm_103a) engine for one decode step
 * of a DeepSeek-style mixture-of-experts layer whose routed experts stay in
 * raw Q2_K (gate, up) and Q3_K (down) blocks.
 *
 * Sources (web pages of the "spark_model" crate, cited by page and item):
 *   [moe_v41]  spark_model/layers/moe_v41.rs -- module doc (the layer's math),
 *              struct MoeV41Cfg, struct MoeV41LayerWeights, struct Kernels,
 *              struct MoeV41 (buffers), fn shared_side, fn softplus,
 *              fn route_from_logits, fn bf16_bytes.
 *   [route]    spark_model/layers/moe_v41/device_route.rs -- module doc,
 *              fn header_words, fn arena_of, fn route_select_launch,
 *              fn slot_table_update, fn parse_header, fn route_device_m1,
 *              fn device_route_check.
 *   [step_seg] spark_model/layers/deepseek_v41_layer/step_seg.rs -- module
 *              doc (the step captured as CUDA graphs over layers).
 *
 * Conventions for every entry point:
 *  - Pointers named *_dev or documented "device" are device pointers; the
 *    caller owns every buffer (the library allocates no device memory on the
 *    hot path). Host pointers are documented as such.
 *  - Calls only ENQUEUE work on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream) and return at once; nothing synchronises implicitly.
 *    Results are valid once the stream reaches the call.
 *  - Return 0 (MOE_OK) or a negative MOE_E* code; moe_last_error() then
 *    returns a message for the calling thread. Argument errors are detected
 *    on the host before anything is enqueued.
 *  - Calls that share a workspace must be ordered on one stream.
 *  - bf16 tensors are passed as raw 16-bit patterns (uint16_t storage).
 *
 * Shapes supported: dim and inter in {256, 512, 1024, 2048, 4096, 8192};
 * 1 <= topk <= 8; topk <= n_routed <= 1024; 1 <= m <= max_tokens <= 8;
 * m * dim <= 32768. Other shapes return MOE_EUNSUPPORTED (or MOE_EINVAL for
 * values that are wrong for any engine, e.g. topk = 0 or a non-multiple of 256).
 */
#ifndef MOE_H
#define MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *moe_stream_t; /* == cudaStream_t */

#define MOE_OK 0
#define MOE_EINVAL (-1)       /* an argument is invalid                       */
#define MOE_EUNSUPPORTED (-2) /* valid, but outside the shapes built here     */
#define MOE_ECUDA (-3)        /* a CUDA call failed (message has the error)   */
#define MOE_ECAPTURE (-4)     /* graph capture or instantiation failed        */

#define MOE_SLOT_TABLE_LAYERS 64 /* rows of the slot table ([route] slot table) */
#define MOE_MAX_TOPK 8
#define MOE_MAX_TOKENS 8
#define MOE_MAX_ROUTED 1024

/* Status bits in word 0 of each token's header row. */
#define MOE_HDR_MISS 1      /* a pick had slot -1: its pointers use slot 0 ([route] module doc) */
#define MOE_HDR_NONFINITE 2 /* a logit or key of the token was NaN or infinite                  */

/* Bits of the workspace status word (moe_read_status). */
#define MOE_WS_TIMEOUT 1   /* a bounded wait inside a kernel gave up           */
#define MOE_WS_PLAN 2      /* a plan exceeded a kernel's capacity; work skipped */
#define MOE_WS_TRIPLE 4    /* moe_slot_table_set met a triple outside the table */
#define MOE_WS_INDEX 8     /* a slot, page, length or token read on the device lay outside its table */
#define MOE_WS_NONFINITE 16 /* a value to be quantised or a logit was NaN or infinite                */
#define MOE_WS_PAGES 32    /* the pool had no free page left for an entry      */

/* Layer configuration ([moe_v41] struct MoeV41Cfg). norm_topk_prob is 0/1. */
typedef struct {
    int32_t dim, inter, n_routed, topk, norm_topk_prob, max_tokens;
    float gate_temp, route_scale, swiglu_limit;
} moe_cfg;

/* The expert arena: expert slot s holds gate (Q2_K [inter, dim]), up (Q2_K
 * [inter, dim]) and down (Q3_K [dim, inter]) blocks at base + s * slot_bytes
 * + {gate,up,down}_off ([route] fn arena_of). base and the three offsets
 * must be 16-byte aligned, slot_bytes a multiple of 16. Device memory. */
typedef struct {
    const void *base;
    uint64_t slot_bytes, gate_off, up_off, down_off;
} moe_arena;

/* Formats of the shared expert ([moe_v41] struct MoeV41LayerWeights: "bf16
 * or the GGUF's Q2_K (w1, w3) / Q3_K (w2) blocks on the routed experts'
 * kernels"). */
#define MOE_SHARED_BF16 0   /* w1, w3 bf16 [inter, dim]; w2 bf16 [dim, inter]   */
#define MOE_SHARED_KQUANT 1 /* w1, w3 Q2_K [inter, dim]; w2 Q3_K [dim, inter],
                               laid out as a routed expert's gate, up, down   */

/* One layer's resident weights ([moe_v41] struct MoeV41LayerWeights), all
 * device pointers: router_w bf16 [n_routed, dim] row-major; bias f32
 * [n_routed]; slot_row i32 [n_routed] (this layer's slot-table row, -1 = not
 * resident); sh_w1, sh_w3, sh_w2 the shared expert in format sh_format
 * (MOE_SHARED_*; all three NULL = no shared expert). 16-byte aligned. */
typedef struct {
    const void *router_w;
    const float *bias;
    const int32_t *slot_row;
    const void *sh_w1, *sh_w3, *sh_w2;
    int32_t sh_format;
} moe_layer;

/* Words (int32) of the route header for m tokens. Layout, k = topk:
 *   row t (t < m), 1 + 3k words ([route] fn header_words, module doc):
 *     [0] status bits (MOE_HDR_*); [1..k] picks in pick order;
 *     [k+1..2k] the weights' f32 bit patterns, pick order; [2k+1..3k] the
 *     slots of the token's picks in ascending expert id (-1 reported as 0)
 *   then the plan over all m tokens (distinct picked experts, ascending id):
 *     [m(1+3k)] ne; [+1 .. +1+m*k] pair_start[0..ne] (ne+1 used);
 *     [+2+m*k .. +1+2*m*k] plan_expert[0..ne-1]. */
int moe_header_words(const moe_cfg *cfg, int m);

/* Bytes of the device workspace for up to cfg->max_tokens tokens. */
int moe_workspace_bytes(const moe_cfg *cfg, size_t *bytes);

/* Zeroes a workspace (its counters must start at zero). Call once after
 * allocating it, on the stream that will use it, and again after a call whose
 * status has MOE_WS_TIMEOUT (a wait that gave up can leave counters mid-count). */
int moe_workspace_init(void *ws_dev, size_t bytes, moe_stream_t stream);

/* Router logits ([moe_v41] module doc: an f32-accumulated product of the bf16
 * input and the bf16 gate weight; struct Kernels router_gemv):
 *   logits[t, e] = sum_j x[t, j] * w[e, j], bf16 products exact in f32, f32
 *   accumulation in a fixed order that does not depend on m.
 * x_dev bf16 [m, dim]; w_dev bf16 [n_routed, dim]; logits_dev f32 [m, n_routed]. */
int moe_router_logits(const moe_cfg *cfg, const void *x_dev, const void *w_dev,
                      float *logits_dev, int m, moe_stream_t stream);

/* q8_1 quantisation of m bf16 rows ([moe_v41] module doc: the activation
 * quantised to q8_1; struct Kernels q8_rows): per 32 values d = amax / 127
 * (f32), q = round-half-away(x / d), stored as f16 d, f16 d * sum q, int8
 * q[32] (36 bytes). out_dev: m * dim / 32 blocks. */
int moe_quantize_q8_1(const moe_cfg *cfg, const void *x_dev, int m, void *out_dev,
                      moe_stream_t stream);

/* Device selection ([moe_v41] fn route_from_logits; [route] fn
 * route_select_launch, module doc): per token, scores s = the f32 chain
 * sqrt(ln_1p(exp(t))), t = l / temp, each step correctly rounded (t itself
 * in place of ln_1p(exp(t)) for t > 20; [moe_v41] fn softplus), picks = the top k of
 * s + bias with ties to the lower id, weights = picked scores divided by
 * (their f32 sum in pick order + 1e-20) when norm_topk_prob and k > 1, times
 * route_scale; then the plan, the plan weights and rows (pair-major:
 * experts ascending, tokens ascending within one), and the pointer table
 * ptrs[0..cap) gate, [cap..2cap) up, [2cap..3cap) down with cap = m * topk,
 * pointer = base + slot * slot_bytes + offset, slot -1 -> slot 0 and the
 * MOE_HDR_MISS bit. Scores, picks and weights are bit-identical to the
 * definition (each rounding of the score decided exactly).
 * logits_dev f32 [m, n_routed]; bias_dev f32 [n_routed]; slot_row_dev i32
 * [n_routed]; arena by value (host struct, device base); header_dev i32
 * [moe_header_words]; plan_w_dev f32 [m*topk]; plan_rows_dev i32 [m*topk];
 * ptrs_dev u64 [3*m*topk]. */
int moe_route_select(const moe_cfg *cfg, const float *logits_dev, const float *bias_dev,
                     const int32_t *slot_row_dev, const moe_arena *arena, int m,
                     int32_t *header_dev, float *plan_w_dev, int32_t *plan_rows_dev,
                     uint64_t *ptrs_dev, moe_stream_t stream);

/* The routing score of each logit ([moe_v41] fn softplus, fn
 * route_from_logits): t = f32(logits[i] / gate_temp); for t > 20
 * scores[i] = f32(sqrt(t)), else e = f32(e^t), p = f32(ln(1 + e)),
 * scores[i] = f32(sqrt(p)), each rounding to nearest as a correctly rounded
 * operation -- the score the router and the selection use. The roundings
 * are decided in float-float single precision, in double and then
 * double-double precision when that cannot decide them. logits_dev,
 * scores_dev f32 [count], count >= 0 (0: nothing is launched). */
int moe_route_scores(const moe_cfg *cfg, const float *logits_dev, int count, float *scores_dev,
                     moe_stream_t stream);

/* The routed experts of one call ([moe_v41] module doc: three K-quant GEMVs
 * per expert on the raw blocks, gate and up Q2_K, down Q3_K, q8_1 activation;
 * struct Kernels mmvq_q2k_experts / swiglu_q8 / mmvq_q3k_experts /
 * accumulate): for every plan expert p and each of its tokens t
 *   g, u = Q2_K(gate_p, up_p) . q8_1(x_t);  h = silu(min(g, L)) * clamp(u, -L, L)
 *   down = Q3_K(down_p) . q8_1(h);  acc_t = sum over t's plan, ascending id,
 *   of w * down (f32). Reads the plan from header_dev (moe_route_select).
 * acc_dev f32 [m, dim]; ws_dev: workspace (intermediates g, u, down stay there). */
int moe_expert_step(const moe_cfg *cfg, const void *x_dev, const uint64_t *ptrs_dev,
                    const float *plan_w_dev, const int32_t *plan_rows_dev,
                    const int32_t *header_dev, int m, float *acc_dev, void *ws_dev,
                    moe_stream_t stream);

/* Clamped SwiGLU and the q8_1 of its output ([moe_v41] struct Kernels
 * swiglu_q8): h[i] = silu(min(g, L)) * clamp(u, -L, L) in f32 (L <= 0: no
 * clamp); h_q8 as moe_quantize_q8_1. g_dev, u_dev, h_dev f32 [rows, inter];
 * hq8_dev rows * inter / 32 blocks (h_dev may be NULL). */
int moe_swiglu_q8(const moe_cfg *cfg, const float *g_dev, const float *u_dev, int rows,
                  float *h_dev, void *hq8_dev, moe_stream_t stream);

/* One whole MoE layer step for m tokens ([moe_v41] module doc and fn
 * shared_side; [route] module doc): router logits, selection, routed experts,
 * the shared expert (bf16: gs, us = W1 x, W3 x; hs = bf16(SwiGLU); sd = W2 hs;
 * K-quant: gs, us = Q2_K(W1, W3) . q8_1(x), hs = SwiGLU in f32, sd =
 * Q3_K(W2) . q8_1(hs), as a routed expert of weight 1 -- [moe_v41] struct
 * MoeV41 sh_q8),
 * acc = routed sum (ascending id) + sd added last, residual += acc,
 * x_next = bf16 round-to-nearest-even of residual ([moe_v41] fn bf16_bytes).
 * Launched as three kernels chained with programmatic dependent launch.
 * x_dev bf16 [m, dim]; residual_dev f32 [m, dim] (in/out); x_next_dev bf16
 * [m, dim] (may equal x_dev); header_dev i32 [moe_header_words]; acc, the
 * plan, pointers and intermediates are left in ws_dev (moe_ws_view). */
int moe_layer_step(const moe_cfg *cfg, const moe_layer *layer, const moe_arena *arena,
                   const void *x_dev, float *residual_dev, void *x_next_dev,
                   int32_t *header_dev, int m, void *ws_dev, moe_stream_t stream);

/* moe_layer_step without a caller workspace and without any device
 * allocation. The pages have no counterpart of this call: it exists for
 * callers that cannot allocate device memory (a plain C host program linking
 * only this library, with no device allocator of its own; a serving loop that
 * must not allocate once it runs, since cudaMalloc and cudaFree can
 * synchronise the device and can fail under memory pressure).
 * The workspace is a 4 MiB array in the library's device memory, one per
 * device. The first call on a device (with that device current) looks it up
 * with cudaGetSymbolAddress and zeroes it; make that first call before any
 * stream capture (a first call on a capturing stream returns
 * MOE_EUNSUPPORTED). The looked-up address is kept for the life of the
 * process: do not use this call across cudaDeviceReset of that device.
 * Every call clears the array's control words and counters on `stream`
 * first, then runs the same kernels as moe_layer_step.
 * Arguments as moe_layer_step; status_host: NULL, or a host word that
 * receives the workspace status (MOE_WS_*) of this call once `stream`
 * reaches the end of the call (pinned memory keeps the copy asynchronous).
 * The array is shared by every call on the device: calls that overlap in
 * time (other streams, other host threads) race on it and must be
 * serialised by the caller. Errors: MOE_EUNSUPPORTED when the configuration
 * needs more than 4 MiB of workspace (moe_workspace_bytes); MOE_EINVAL for
 * bad arguments; MOE_ECUDA when the look-up or a launch fails. */
int moe_layer_step_static(const moe_cfg *cfg, const moe_layer *layer, const moe_arena *arena,
                          const void *x_dev, float *residual_dev, void *x_next_dev,
                          int32_t *header_dev, int m, uint32_t *status_host, moe_stream_t stream);

/* Same step with HOST buffers: copies x (bf16 [m, dim], host) and residual
 * (f32 [m, dim], host) in, runs moe_layer_step, copies residual, x_next and
 * the header back to host buffers, all on `stream` (pinned host memory makes
 * the copies asynchronous). io_dev: device scratch of
 * moe_host_io_bytes(cfg, m) bytes. */
int moe_host_io_bytes(const moe_cfg *cfg, int m, size_t *bytes);
int moe_layer_step_host(const moe_cfg *cfg, const moe_layer *layer, const moe_arena *arena,
                        const void *x_host, float *residual_host, void *x_next_host,
                        int32_t *header_host, int m, void *io_dev, void *ws_dev,
                        moe_stream_t stream);

/* Where the intermediates of the last call live inside a workspace (device
 * pointers into ws_dev), for inspection. */
typedef struct {
    float *logits;      /* [m, n_routed]                                   */
    float *plan_w;      /* [m*topk]                                        */
    int32_t *plan_rows; /* [m*topk]                                        */
    uint64_t *ptrs;     /* [3*m*topk]                                      */
    float *g, *u;       /* [m*topk, inter] per plan pair                   */
    float *gs, *us;     /* [m, inter] shared expert                        */
    float *down;        /* [m*topk, dim] per plan pair                     */
    float *sd;          /* [m, dim] shared expert output                   */
    float *acc;         /* [m, dim] routed sum + shared                    */
    uint32_t *status;   /* one word, MOE_WS_* bits                         */
} moe_ws_view;
int moe_workspace_view(const moe_cfg *cfg, void *ws_dev, moe_ws_view *view);

/* Reads the workspace status word (MOE_WS_* bits) to a host variable; this
 * synchronises `stream`. */
int moe_read_status(void *ws_dev, uint32_t *status_host, moe_stream_t stream);

/* Sets the bound, in nanoseconds, on every wait inside the kernels (a wait
 * on a shared-memory barrier, on another CTA's count, or on the selection's
 * plan) for the calls enqueued after it; a graph keeps the bound it was
 * captured with. 0 restores the default of 2 s. Process-wide. When a wait
 * runs out, the kernel records MOE_WS_TIMEOUT in the workspace status and
 * returns instead of waiting on (page step_seg.rs has no counterpart: a
 * device wait there is unbounded). */
int moe_set_wait_limit_ns(uint64_t ns);

/* Failure-handling check, not a step of the layer: launches the two expert
 * kernels of a layer step as moe_layer_step does, but with no router kernel
 * before them, so the gate/up producers' bounded wait for the selection's
 * plan-ready word can only end by running out. header_dev must hold an empty
 * plan (zeros: ne = 0), so that no expert is read. After the stream reaches
 * it, the workspace status has MOE_WS_TIMEOUT and the workspace must be
 * initialised again (moe_workspace_init). x_dev bf16 [m, dim]. */
int moe_expert_step_unreleased(const moe_cfg *cfg, const void *x_dev, const int32_t *header_dev, int m,
                               void *ws_dev, moe_stream_t stream);

/* Slot-table update ([route] fn slot_table_update, struct Kernels
 * slot_table_set): for each of n (layer, expert, slot) int32 triples,
 * table[layer * n_routed + expert] = slot. The triples are applied in
 * parallel, so the caller must pass at most one triple per (layer, expert)
 * (moe_dedupe_triples gives the last-write-wins set). A triple outside
 * [0, 64) x [0, n_routed) is skipped and sets MOE_WS_TRIPLE in
 * *status_dev (may be NULL). table_dev i32 [64, n_routed]; triples_dev i32
 * [n, 3]. */
int moe_slot_table_set(int32_t *table_dev, int n_routed, const int32_t *triples_dev, int n,
                       uint32_t *status_dev, moe_stream_t stream);

/* Host helper: keeps only the last triple of each (layer, expert) key, in
 * place, preserving the order of first appearance of the kept keys; *n_out
 * = the count kept. Host pointer. */
int moe_dedupe_triples(int32_t *triples_host, int n, int *n_out);

/* Host helper ([route] fn parse_header): token t's status word, picks and
 * weights out of a header copied to the host. Fails (MOE_EINVAL) when a pick
 * lies outside 0..n_routed-1. picks_host i32 [topk], weights_host f32 [topk]. */
int moe_parse_header(const moe_cfg *cfg, const int32_t *header_host, int m, int t,
                     int32_t *status_host, int32_t *picks_host, float *weights_host);

/* Options of moe_graph_create. */
#define MOE_GRAPH_SNAPSHOTS 1       /* copy each layer's input (x and residual) to snapshot memory
                                       before the layer, inside the graph ([step_seg] module doc:
                                       a snapshot a layer, ~75 KB there), so the step can be rerun
                                       from a layer (moe_graph_rerun_from, moe_graph_step_cached) */
#define MOE_GRAPH_EAGER_FALLBACK 2  /* if capture or instantiation fails, the object runs the layers
                                       eagerly instead ([step_seg] fn close_or_disable: graph mode off) */
#define MOE_GRAPH_TEST_FAIL_CAPTURE 4 /* failure-handling check: treat the capture as failed (no capture
                                       is attempted), to exercise MOE_GRAPH_EAGER_FALLBACK */

/* A whole-step CUDA graph ([step_seg] module doc: the step captured once and
 * replayed, one read-back of the headers per launch): n_layers layer steps
 * chained, layer l reading x from x_a (l even) or x_b (l odd) and writing the
 * other, except that the last layer writes x_a, so each launch continues from
 * the previous launch's output; residual_dev carries between layers; layer
 * l's header lands at headers_dev + l * moe_header_words(cfg, m). layers is a
 * host array of n_layers structs (copied; their device pointers are baked
 * in); every buffer must outlive the graph. snap_dev: moe_graph_snapshot_bytes
 * of device memory with MOE_GRAPH_SNAPSHOTS, else may be NULL. flags:
 * MOE_GRAPH_*. Without MOE_GRAPH_EAGER_FALLBACK a failed capture returns
 * MOE_ECAPTURE and no object. */
int moe_graph_snapshot_bytes(const moe_cfg *cfg, int m, int n_layers, size_t *bytes);
int moe_graph_create(const moe_cfg *cfg, const moe_layer *layers, int n_layers,
                     const moe_arena *arena, int m, void *x_a_dev, void *x_b_dev,
                     float *residual_dev, int32_t *headers_dev, void *ws_dev, void *snap_dev,
                     unsigned flags, void **graph);
/* *eager = 1 when the object runs its layers eagerly (capture failed). */
int moe_graph_is_eager(void *graph, int *eager);
/* Restores layer `layer`'s snapshot into that layer's input buffers and runs
 * layers layer .. n_layers - 1 eagerly on `stream` (snapshots refreshed on
 * the way). Needs MOE_GRAPH_SNAPSHOTS. */
int moe_graph_rerun_from(void *graph, int layer, moe_stream_t stream);
int moe_graph_launch(void *graph, moe_stream_t stream);
int moe_graph_destroy(void *graph);

/* One graph launch with HOST buffers: copies x (bf16 [m, dim]) and residual
 * (f32 [m, dim]) from host memory into the graph's x_a / residual buffers,
 * launches the graph, and copies the output x (x_a), the residual and every
 * layer's header back to host memory, all on `stream` (pinned host memory
 * makes the copies asynchronous). headers_host: n_layers * moe_header_words. */
int moe_graph_launch_host(void *graph, const void *x_host, const float *residual_host, void *x_out_host,
                          float *residual_out_host, int32_t *headers_host, moe_stream_t stream);

/* Measurement entry point: the same layer step as moe_layer_step, but the
 * three kernels run back to back without overlap, bracketed by CUDA events on
 * `stream`; synchronises `stream` and writes the durations in milliseconds to
 * ms_host[0] (router + selection), ms_host[1] (gate/up GEMVs incl. the shared
 * W1/W3 rows), ms_host[2] (down GEMVs incl. shared W2, accumulate, residual). */
int moe_layer_step_profiled(const moe_cfg *cfg, const moe_layer *layer, const moe_arena *arena,
                            const void *x_dev, float *residual_dev, void *x_next_dev, int32_t *header_dev,
                            int m, void *ws_dev, moe_stream_t stream, float *ms_host);

/* Dense GEMM on the tensor cores (tcgen05.mma, f32 accumulator in tensor
 * memory, operands by TMA): d[n * ldd + r] = sum_k a[r, k] * b[n, k], a bf16
 * [M, K] and b bf16 [N, K] row-major (bf16 products exact, f32 sums) --
 * the contraction of the router and of the bf16 shared expert when many
 * tokens run at once ([moe_v41] struct Kernels gemm / gemm_f32out). K a
 * positive multiple of 64, ldd >= M, a and b 16-byte aligned with row
 * strides K * 2 a multiple of 16. Device pointers. */
int moe_gemm_bf16(const void *a_dev, const void *b_dev, float *d_dev, int M, int N, int K, int ldd,
                  moe_stream_t stream);

/* The batched (prefill) arm: one MoE layer step for m tokens at once
 * ([moe_v41] struct Kernels gather, scatter_add, sum_rows, quant_d2s6 /
 * quant_d4, mmq_q2k_*, mmq_q3k_*, gemm; struct MoeV41 a_rows, a_q8: an
 * expert group's gathered rows and their q8_1 activations). The arithmetic
 * is moe_layer_step's; the routed experts run as GEMMs over each expert's
 * group of tokens, on tensor cores:
 *   logits = router GEMM; scores, picks and weights as the decode selection;
 *   pairs (token, pick) grouped by expert in ascending id, tokens ascending;
 *   per expert g, u = Q2_K(gate, up) . q8_1(x) over its group, h = SwiGLU,
 *   q8_1(h), down = Q3_K(down) . q8_1(h), each times the pair's weight;
 *   the bf16 shared expert as dense GEMMs; acc = the pairs in ascending
 *   expert id then sd; residual += acc; x_next = bf16(residual).
 * The GEMM operands are the dequantised weights and the dequantised q8_1
 * activations rounded to fp16 (the products then differ from the exact
 * dequantise-then-dot by about 2^-12 relative per operand); accumulation
 * f32. Shapes: dim a multiple of 1024, inter of 2048 (the row strides of
 * the Q2_K / Q3_K blocks must be multiples of 16 bytes for TMA), the shared
 * expert bf16 or absent, 0 <= m <= 65536 (cfg->max_tokens is not used).
 * arena_slots: slots in the arena (the tensor maps cover that many). x_dev
 * bf16 [m, dim], 16-byte aligned (a TMA operand; otherwise MOE_EINVAL before
 * any launch); residual_dev f32 [m, dim] (in/out); x_next_dev bf16 [m, dim]
 * (16- and 8-byte alignment of these take the wider accesses); picks_dev i32 [m, topk], weights_dev f32 [m, topk] (pick
 * order); ws_dev: moe_prefill_workspace_bytes bytes (no initialisation
 * needed). Errors: MOE_EUNSUPPORTED for the shapes above; a picked expert
 * whose slot is -1 uses slot 0 and sets MOE_WS_PLAN (moe_prefill_status). */
int moe_prefill_workspace_bytes(const moe_cfg *cfg, int m, size_t *bytes);
int moe_prefill_step(const moe_cfg *cfg, const moe_layer *layer, const moe_arena *arena, int64_t arena_slots,
                     const void *x_dev, float *residual_dev, void *x_next_dev, int32_t *picks_dev,
                     float *weights_dev, int m, void *ws_dev, size_t ws_bytes, moe_stream_t stream);

/* Measurement entry point: moe_prefill_step with CUDA events between its
 * stages on `stream`; synchronises `stream` and writes milliseconds to
 * ms_host[0..8]: router GEMM; scores, top-k and grouping; q8_1 of x and the
 * gathers; gate GEMM; up GEMM; SwiGLU + q8_1(h); down GEMM; shared expert
 * (three GEMMs and its SwiGLU); finish. */
int moe_prefill_step_profiled(const moe_cfg *cfg, const moe_layer *layer, const moe_arena *arena,
                              int64_t arena_slots, const void *x_dev, float *residual_dev, void *x_next_dev,
                              int32_t *picks_dev, float *weights_dev, int m, void *ws_dev, size_t ws_bytes,
                              moe_stream_t stream, float *ms_host);

/* The status word (MOE_WS_* bits) of the last moe_prefill_step on ws_dev;
 * synchronises `stream`. */
int moe_prefill_status(const moe_cfg *cfg, int m, void *ws_dev, uint32_t *status_host, moe_stream_t stream);

/* Expert residency ([moe_v41] module doc: the ExpertLru gathers the picked
 * experts' raw slices into device-visible slots, misses read from the
 * source; [route] module doc and fn slot_table_update: the host touches the
 * picks, fetches the misses and uploads the slot changes to the device
 * table). A cache owns n_slots slots of the arena for layers 0 .. n_layers-1
 * of the slot table at slot_table_dev ([64][n_routed], row l for layer l; NULL
 * keeps the table on the host only), least recently used out first, and
 * fetches a missing expert with fetch(user, layer, expert, slot address,
 * slot_bytes, stream) -- which must enqueue the copy of the expert's slot
 * image on `stream` and return 0. Creating the cache marks every entry of its
 * rows not resident (-1). */
typedef int (*moe_expert_fetch_fn)(void *user, int layer, int expert, void *slot_dev, uint64_t slot_bytes,
                                   moe_stream_t stream);
int moe_cache_create(int n_layers, int n_routed, int n_slots, const moe_arena *arena, int32_t *slot_table_dev,
                     moe_expert_fetch_fn fetch, void *user, void **cache);
int moe_cache_destroy(void *cache);
/* Makes the experts (host array of n ids of one layer; repeats allowed)
 * resident: hits become most recently used, misses take the least recently
 * used slots (their previous experts marked -1) and are fetched; the changed
 * table rows are uploaded on `stream`. *n_fetched (may be NULL) = misses.
 * MOE_EUNSUPPORTED when more distinct experts are asked at once than slots. */
int moe_cache_ensure(void *cache, int layer, const int32_t *experts_host, int n, int *n_fetched,
                     moe_stream_t stream);
/* The slot of (layer, expert), -1 when not resident. */
int moe_cache_slot_of(void *cache, int layer, int expert, int32_t *slot);
int moe_cache_stats(void *cache, uint64_t *hits, uint64_t *misses, uint64_t *evictions);

/* An expert source over host memory: images_host[layer * n_routed + expert]
 * = host address of that expert's slot image (image_bytes; pinned memory
 * keeps the copies asynchronous). moe_fetch_host_images is its fetch
 * function (pass the source as `user`). */
int moe_host_source_create(const void *const *images_host, int n_layers, int n_routed, uint64_t image_bytes,
                           void **source);
int moe_host_source_destroy(void *source);
int moe_fetch_host_images(void *source, int layer, int expert, void *slot_dev, uint64_t slot_bytes,
                          moe_stream_t stream);

/* One launch of a graph with snapshots whose layers take their experts from
 * a cache (layer l using row l of the cache's table): launch, read the
 * headers; at the first layer whose header has MOE_HDR_MISS, make that
 * layer's picks resident, restore its snapshot and run the rest eagerly,
 * layer by layer, a layer with a miss fetched and rerun from its snapshot
 * ([step_seg] module doc and fn step_seg: restore, the layer's ffn eagerly,
 * eager to the end). On return (the stream synchronised) the graph's buffers
 * hold the result and headers_host (host, n_layers header rows) the final
 * headers; *layers_rerun (may be NULL) = layers run again. */
int moe_graph_step_cached(void *graph, void *cache, int32_t *headers_host, int *layers_rerun,
                          moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Speculative decoding around the layer step: a quantised paged cache of keys
 * and values, attention of drafted tokens over it, and their verification.
 * The pages have no counterpart of these calls: a layer step of several tokens
 * of one sequence (m > 1) needs tokens drafted ahead, and these judge them.
 * All calls only enqueue on `stream`; bf16 as raw 16-bit patterns. */

/* Formats of the cache: per 32 consecutive values of a row (one token, one kv
 * head), clamped to +-60000 (NaN is held as 0 and sets MOE_WS_NONFINITE, as
 * do infinities),
 *   Q8: d = f16(max|x| / 127) rounded up, code = rint(x / d) + 128 in 8 bits,
 *       value d * (code - 128);
 *   Q4: m = f16(min x) rounded down, d = f16((max x - m) / 15) rounded up,
 *       code = rint((x - m) / d) in 4 bits, value d * code + m
 * (quotients in f32, rint to even, code 0 of the quotient where d = 0), so
 * |x - value| <= d / 2. */
#define MOE_KV_Q8 0
#define MOE_KV_Q4 1

#define MOE_MAX_DRAFT 64 /* query rows of one sequence in one call: the last token and 63 drafted */

/* A cache of one layer: n_pages pages of page_size tokens, of which slot s is
 * token s % page_size of page s / page_size. Per page, kv head and 16 tokens
 * one block, blocks in that order (page, head, 16 tokens):
 *   K codes [16 RB] | K scales | V codes [16 RB] | V scales,
 * RB = head_dim (Q8) or head_dim / 2 (Q4) bytes. With t the token in the
 * block, i a byte of its row and x a count of bytes, a code byte lies at
 * x / 16 * 512 + lane * 16 + x % 16:
 *   K: lane = t % 8 * 4 + i / (RB / 4), x = t / 8 * (RB / 4) + i % (RB / 4)
 *   V: lane = i / (RB / 8) * 4 + t % 8 / 2,
 *      x = (t / 8 * 2 + t % 2) * (RB / 8) + i % (RB / 8)
 * Four bytes hold eight Q4 codes (a little-endian word), code c of them at bit
 * c / 2 * 4 + c % 2 * 16. Scales are f16: K [t][group][d or d, m], V [d or
 * d, m][group][t]. pages: device memory, 16-byte aligned, n_pages *
 * moe_kv_page_bytes bytes. head_dim 64, 128 or 256; page_size a multiple of 16
 * up to 1024; n_kv_heads 1 .. 256; n_pages * page_size below 2^31. */
typedef struct {
    void *pages;
    int64_t n_pages;
    int32_t head_dim, n_kv_heads, page_size, format;
} moe_kv_cache;

/* Bytes of one page (pages and n_pages of the struct are not looked at). */
int moe_kv_page_bytes(const moe_kv_cache *cache, size_t *bytes);

/* Quantises n_tokens rows of keys and values into the cache: token t's row of
 * head h is k_dev + t * k_token_stride + h * k_head_stride (bf16, strides in
 * elements, so views of a fused projection's output can be passed), written
 * to slot slots_dev[t] (i32; -1: the token is skipped; the caller passes a
 * slot at most once). Rows that all start on 32-byte (16-byte) boundaries are
 * loaded that wide, others slower. *status_dev (NULL, or a device
 * word) receives MOE_WS_INDEX for a slot outside the cache (skipped) and
 * MOE_WS_NONFINITE. */
int moe_kv_append(const moe_kv_cache *cache, const void *k_dev, int64_t k_token_stride, int64_t k_head_stride,
                  const void *v_dev, int64_t v_token_stride, int64_t v_head_stride, const int32_t *slots_dev,
                  int n_tokens, uint32_t *status_dev, moe_stream_t stream);

/* Types of a call's floating-point argument. */
#define MOE_BF16 0
#define MOE_F32 1

/* Reads rows back: k_out_dev, v_out_dev [n_tokens, n_kv_heads, head_dim] of
 * out_type (MOE_BF16: rounded once; MOE_F32), 16-byte aligned; slot -1 (or one
 * outside the cache, which sets MOE_WS_INDEX) gives zeros. */
int moe_kv_read(const moe_kv_cache *cache, const int32_t *slots_dev, int n_tokens, void *k_out_dev,
                void *v_out_dev, int out_type, uint32_t *status_dev, moe_stream_t stream);

/* Attention of drafted tokens. Sequence b has the query rows (tokens)
 * q_start_dev[b] .. q_start_dev[b + 1] - 1 (i32 [batch + 1], at most
 * MOE_MAX_DRAFT rows each, n_tokens in all) and kv_len_dev[b] (i32, at most
 * 2^31 - 256) tokens in the cache, its query rows' own keys and values among
 * them as the last ones; token j of it is in slot j % page_size of page
 * table_dev[b * table_stride + j / page_size] (i32, table_pages entries a
 * sequence). Query row i of the sequence sees the tokens before the sequence's
 * query rows, and of those row j when bit j of mask_dev[q_start + i] (u64) is
 * set; mask_dev NULL: rows 0 .. i (a chain). A single token: one row, mask_dev
 * NULL. Per query head h, kv head h / (n_q_heads / n_kv_heads):
 *   out = sum_j softmax_j(scale q . K_j | j seen) V_j,
 * a row that sees nothing gives 0, and a drafted token that no row of its
 * sequence sees need not be in the cache. Products of f16 roundings of the
 * cache's values (2^-11 relative) and of the query's bf16 values times the
 * power of two that brings the row's largest into [2^13, 2^14) (exact down to
 * 2^-30 of the largest, below that within 2^-25 of the scaled value), f32 sums;
 * the softmax in f32, its weights rounded to f16 (2^-11) for the second
 * product. q, out bf16, row stride *_token_stride and head stride
 * *_head_stride in elements, dimensions contiguous. n_q_heads a multiple of
 * n_kv_heads, at most 64 a kv head. ws_dev: moe_tree_attention_workspace_bytes
 * bytes, initialised once (moe_workspace_init); moe_read_status gives
 * MOE_WS_INDEX where lengths (the sequence's rows are 0), or a page (its
 * tokens are not seen) lay outside. batch 0 .. 1024. */
int moe_tree_attention_workspace_bytes(const moe_kv_cache *cache, int n_q_heads, int batch, int n_tokens,
                                       size_t *bytes);
int moe_tree_attention(const moe_kv_cache *cache, const void *q_dev, int64_t q_token_stride, int64_t q_head_stride,
                       void *out_dev, int64_t out_token_stride, int64_t out_head_stride, int n_q_heads,
                       const int32_t *q_start_dev, const int32_t *kv_len_dev, const int32_t *table_dev,
                       int64_t table_stride, int table_pages, const uint64_t *mask_dev, int batch, int n_tokens,
                       float scale, void *ws_dev, size_t ws_bytes, moe_stream_t stream);

/* Verification of drafted tokens from given random numbers. Sequence b has
 * rows q_start_dev[b] .. q_start_dev[b + 1] - 1 of logits (logits_type;
 * n_rows rows of vocab values, row stride logits_stride elements): row 0 of
 * its last accepted token, row j of drafted node j (at most MOE_MAX_DRAFT
 * rows). tokens_dev i32 [n_rows]: node j's token (row 0's is not read);
 * parents_dev i32 [n_rows]: node j's parent, an earlier row of the sequence
 * (NULL: j - 1, a chain); draft_dev f32 [n_rows, vocab], row stride
 * draft_stride: the probabilities that node j's token was drawn from (NULL:
 * the token was chosen, not drawn). Let p_j = softmax(logits_j /
 * temperature_dev[b]) (NULL: 1; not above 0: all on the largest logit, the
 * lowest index of equals). From cur = 0, r = p_0, Z = 1, for j = 1 .. in order
 * where parent_j = cur: with x = token_j and q = draft row j (NULL: 1 at x),
 *   uniforms_dev[row j] * Z * q(x) < r(x): accepted, cur = j, r = p_j, Z = 1;
 *   else r = max(r - Z q, 0), Z = sum r.
 * next_token = the index of the largest r(i) / noise_dev[b * noise_stride + i]
 * (lowest of equals; r = p_cur where Z = 0): with noise from the exponential
 * distribution a sample of r / Z, so that the tokens follow the target's
 * distribution whatever the draft's. uniforms_dev f32 [n_rows] in [0, 1),
 * noise_dev f32 [batch, vocab] > 0; both NULL: every sequence greedy.
 * Outputs: n_accepted_dev i32 [batch]; path_dev i32 [n_rows], the accepted
 * nodes of sequence b from q_start[b] on, then -1; next_token_dev i32 [batch]
 * (-1 where the last row has no finite logit, or no rows). A logit of NaN or
 * +infinity counts as -infinity and sets MOE_WS_NONFINITE, a token outside the
 * vocabulary is passed over and sets MOE_WS_INDEX. ws_dev: initialised once.
 * batch 0 .. 65535, vocab 1 .. 2^24; n_rows 0: the rows' arguments may be NULL. */
int moe_spec_verify_workspace_bytes(int batch, int n_rows, size_t *bytes);
int moe_spec_verify(const void *logits_dev, int logits_type, int64_t logits_stride, const int32_t *q_start_dev,
                    const int32_t *tokens_dev, const int32_t *parents_dev, const float *draft_dev,
                    int64_t draft_stride, const float *temperature_dev, const float *uniforms_dev,
                    const float *noise_dev, int64_t noise_stride, int batch, int n_rows, int vocab,
                    int32_t *n_accepted_dev, int32_t *path_dev, int32_t *next_token_dev, void *ws_dev,
                    size_t ws_bytes, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions, attention with keys and values from one shared latent
 * vector a token, and the care of a cache's pages. The pages that the rest of
 * this header cites have no counterpart of these calls: they are what surrounds
 * the layer step in a layer of this kind. All calls only enqueue on `stream`;
 * status words (NULL, or a device word) receive MOE_WS_* bits. */

/* Frequencies of rotary positions: pair i of dim / 2 turns by f_i = base^(-2i /
 * dim) radians a position, scaled for contexts longer than the model's own by
 *   MOE_ROPE_PLAIN   nothing;
 *   MOE_ROPE_LINEAR  f_i / factor;
 *   MOE_ROPE_BASE    the base times factor^(dim / (dim - 2)) (dim > 2);
 *   MOE_ROPE_PARTS   f_i (k + (1 - k) / factor), k = clamp((r - slow) / (fast -
 *                    slow), 0, 1) with r = original f_i / 2 pi the pair's turns
 *                    in `original` positions, and the magnitude 0.1 ln(factor) + 1
 *                    (else 1) for both results of a turn. The ramp is over a
 *                    pair's turns. Code that ramps over its index i, between two
 *                    whole indices, gives other frequencies to the pairs between
 *                    them, and may use another magnitude: a caller that needs
 *                    those fills the table and gives the magnitude itself. */
#define MOE_ROPE_PLAIN 0
#define MOE_ROPE_LINEAR 1
#define MOE_ROPE_BASE 2
#define MOE_ROPE_PARTS 3
typedef struct {
    int32_t dim, scaling;
    double base, factor, original, slow, fast;
} moe_rope_cfg;

/* Host: table_host[i] (dim / 2 of them) = f_i / 2 pi, the part of a turn that a
 * position adds, times 2^64 and rounded, so that position p stands at p *
 * table[i] mod 2^64 of a turn, exactly, for any int32 p. Copied to the device by
 * the caller. dim even, 2 .. 1024; base, factor >= 1 (f_i of less than a turn);
 * 0 <= slow < fast, original > 0 for MOE_ROPE_PARTS. *magnitude_host may be NULL. */
int moe_rope_table(const moe_rope_cfg *cfg, uint64_t *table_host, float *magnitude_host);

/* Which dimensions are a pair: i and i + rope_dim / 2, or 2i and 2i + 1. */
#define MOE_ROPE_HALF 0
#define MOE_ROPE_INTERLEAVED 1

/* Rotary positions on part of each head: of x [tokens, heads, head_dim] (type
 * MOE_BF16 or MOE_F32; token and head strides in elements, dimensions
 * contiguous), dimensions offset .. offset + rope_dim - 1 of each row, in pairs
 * (a, b) with angle t of the row's position (positions_dev i32 [tokens], any
 * sign) and the pair (table_dev u64 [rope_dim / 2]):
 *   a' = magnitude (a cos t - b sin t), b' = magnitude (a sin t + b cos t);
 * transposed != 0: -t, the gradient's way back (with magnitude 1 also the
 * inverse). In f32: the angle, from half a turn back to half a turn on, rounded
 * to 2^-32 of a turn and then to f32 (an error of 2^-26 + 2^-33 of a turn at most,
 * near half a turn; less with the angle), results rounded once.
 * Other dimensions are copied. out may be x with the same strides (in place:
 * other dimensions are not touched); it must not overlap x in another way.
 * head_dim 1 .. 1024, rope_dim even, 2 .. head_dim - offset. Rows that start on
 * 16-byte boundaries, with offset and half a rope_dim (MOE_ROPE_INTERLEAVED: a
 * rope_dim) of whole 16-byte pieces, are moved in such pieces, others value by
 * value. tokens or heads 0: nothing is launched. */
int moe_rope(const void *x_dev, int64_t x_token_stride, int64_t x_head_stride, void *out_dev,
             int64_t out_token_stride, int64_t out_head_stride, int type, int tokens, int heads, int head_dim,
             int offset, int rope_dim, int layout, const int32_t *positions_dev, const uint64_t *table_dev,
             float magnitude, int transposed, moe_stream_t stream);

/* A cache of one layer's latent vectors: n_pages pages of page_size rows
 * (tokens), a row latent_dim + rope_dim bf16 values, the latent vector and the
 * part of the key that turns; slot s is row s, token s % page_size of page s /
 * page_size. pages: device memory, 16-byte
 * aligned, n_pages * moe_latent_page_bytes bytes. latent_dim 128, 256 or 512;
 * rope_dim a multiple of 8 from 8 to 64; page_size a multiple of 16 up to 1024;
 * n_pages * page_size below 2^31. */
typedef struct {
    void *pages;
    int64_t n_pages;
    int32_t latent_dim, rope_dim, page_size;
} moe_latent_cache;

/* Bytes of one page (pages and n_pages of the struct are not looked at). */
int moe_latent_page_bytes(const moe_latent_cache *cache, size_t *bytes);

/* Writes n_tokens rows: latent vector c_dev + t * c_stride and key part kr_dev
 * + t * kr_stride (bf16, strides in elements) to slot slots_dev[t] (i32; -1: the
 * token is skipped; the caller passes a slot at most once; a slot outside the
 * cache is skipped and sets MOE_WS_INDEX). positions_dev i32 [n_tokens] and
 * table_dev u64 [rope_dim / 2]: the key part is turned as by moe_rope with
 * `layout` and `magnitude` on its way; both NULL: written as it is. */
int moe_latent_append(const moe_latent_cache *cache, const void *c_dev, int64_t c_stride, const void *kr_dev,
                      int64_t kr_stride, const int32_t *slots_dev, int n_tokens, const int32_t *positions_dev,
                      const uint64_t *table_dev, int layout, float magnitude, uint32_t *status_dev,
                      moe_stream_t stream);

/* Reads rows back (for the expanded form, another pool or a check): c_out_dev
 * [n_tokens, latent_dim], kr_out_dev [n_tokens, rope_dim] bf16, row strides in
 * elements; slot -1 (or one outside the cache, which sets MOE_WS_INDEX) gives
 * zeros. */
int moe_latent_read(const moe_latent_cache *cache, const int32_t *slots_dev, int n_tokens, void *c_out_dev,
                    int64_t c_stride, void *kr_out_dev, int64_t kr_stride, uint32_t *status_dev,
                    moe_stream_t stream);

/* Latent attention, absorbed form: one token, a chain or a tree of drafted
 * tokens a sequence, all heads over the sequence's shared rows of the cache.
 * Sequences, lengths, page table and masks are as for moe_tree_attention
 * (q_start, kv_len, table, mask; at most MOE_MAX_DRAFT rows a sequence). For row
 * i and head h, over the tokens j that row i sees:
 *   out[i, h] = sum_j softmax_j(scale (q[i, h] . c_j + qr[i, h] . kr_j)) c_j,
 * q, out [n_tokens, heads, latent_dim], qr [n_tokens, heads, rope_dim] bf16 with
 * token and head strides in elements: q is the query times the keys'
 * up-projection, out goes through the values' one. A row that sees nothing, or
 * nothing but scores of -inf, gives 0; a drafted token that no row of its
 * sequence sees need not be in the cache, and a NaN or infinity in a token's row
 * reaches only query rows that see the token: all of the row where the token's
 * score is NaN or +inf, and where it is -inf the token's dimensions that are not
 * finite, as NaN. bf16 products in f32 sums, the softmax in f32, its weights rounded to bf16 (2^-8)
 * for the second product and added up as rounded. heads 1 .. 128, batch 0 ..
 * 1024. ws_dev: moe_latent_attention_workspace_bytes bytes, initialised once
 * (moe_workspace_init); moe_read_status gives MOE_WS_INDEX where lengths (the
 * sequence's rows are 0), or a page (its tokens are not seen) lay outside. */
int moe_latent_attention_workspace_bytes(const moe_latent_cache *cache, int heads, int batch, int n_tokens,
                                         size_t *bytes);
int moe_latent_attention(const moe_latent_cache *cache, const void *q_dev, int64_t q_token_stride,
                         int64_t q_head_stride, const void *qr_dev, int64_t qr_token_stride, int64_t qr_head_stride,
                         void *out_dev, int64_t out_token_stride, int64_t out_head_stride, int heads,
                         const int32_t *q_start_dev, const int32_t *kv_len_dev, const int32_t *table_dev,
                         int64_t table_stride, int table_pages, const uint64_t *mask_dev, int batch, int n_tokens,
                         float scale, void *ws_dev, size_t ws_bytes, moe_stream_t stream);

/* Latent attention, expanded form, for prompts: sequence b has the query rows
 * q_start_dev[b] .. q_start_dev[b + 1] - 1 (i32 [batch + 1]) and the tokens
 * kv_start_dev[b] .. kv_start_dev[b + 1] - 1 of k, kr and v, its query rows the
 * last of them (earlier parts of the prompt come before). Row i of n over t
 * tokens sees tokens 0 .. t - n + i (causal != 0) or all:
 *   out[i, h] = sum_j softmax_j(scale (q[i, h] . [k[j, h] | kr[j]])) v[j, h],
 * q [q_tokens, heads, nope_dim + rope_dim], k, v [kv_tokens, heads, nope_dim],
 * kr [kv_tokens, rope_dim], out [q_tokens, heads, nope_dim], all bf16, strides
 * in elements. A row that sees nothing gives 0 (a causal one of a sequence with
 * fewer tokens than rows); a NaN or infinity in a token that a row does not see
 * does not reach it, and a row that sees an infinite value is infinite or NaN
 * there, whatever its score. Products as for moe_latent_attention. nope_dim 64 or 128,
 * rope_dim a multiple of 8 from 8 to 64, heads 1 .. 1024, batch 0 .. 1024,
 * q_tokens up to 2^23, kv_tokens up to 2^30. k, kr and v must start on 16-byte
 * boundaries and have strides of multiples of 8, those of tokens positive, those
 * of heads positive or 0 (keys, values that all heads share). Rows that no
 * sequence has are not written. The order in which a row's products are added up
 * goes by heads, batch, q_tokens, kv_tokens, nope_dim and the kind of GPU, never
 * by timing: the same call gives the same bits, another batch around a sequence
 * need not.
 * *status_dev receives MOE_WS_INDEX where a sequence's q_start or kv_start fall
 * or lie outside q_tokens or kv_tokens, or its q_start lies before an earlier
 * sequence's (its rows within q_tokens are 0, but those that are a sequence's
 * whose starts hold), and MOE_WS_TIMEOUT. */
int moe_latent_prompt_attention(const void *q_dev, int64_t q_token_stride, int64_t q_head_stride, const void *k_dev,
                                int64_t k_token_stride, int64_t k_head_stride, const void *kr_dev, int64_t kr_stride,
                                const void *v_dev, int64_t v_token_stride, int64_t v_head_stride, void *out_dev,
                                int64_t out_token_stride, int64_t out_head_stride, int heads, int nope_dim,
                                int rope_dim, const int32_t *q_start_dev, const int32_t *kv_start_dev, int batch,
                                int q_tokens, int kv_tokens, int causal, float scale, uint32_t *status_dev,
                                moe_stream_t stream);

/* The care of pages, on the device, so that a captured step can do it. A pool
 * counts for each page how many table entries hold it (refs_dev i32 [n_pages],
 * 0: free; all 0 at first); a table has a row a sequence (i32 [rows, stride],
 * table_pages entries a row; -1: none). One pool and table serve the caches of
 * all layers. New pages are the lowest free ones, in order of rows and entries;
 * where none is left the entry stays -1 and MOE_WS_PAGES is set. An entry, row
 * or length outside its bounds is passed over and sets MOE_WS_INDEX
 * (moe_pages_grow does not look at the pages that a row holds). Calls on
 * one pool must be ordered. n_pages 1 .. 2^24, rows 1 .. 1024. */
typedef struct {
    int32_t *refs;
    int64_t n_pages;
    int32_t page_size;
} moe_page_pool;

/* Gives each row a page for every entry from its first -1 on and below
 * ceil(len_dev[row] / page_size) (i32 [rows]; a row's pages come before its -1
 * entries, as these calls leave them). rows * table_pages below 2^31. */
int moe_pages_grow(const moe_page_pool *pool, int32_t *table_dev, int64_t table_stride, int table_pages, int rows,
                   const int32_t *len_dev, uint32_t *status_dev, moe_stream_t stream);

/* Row target_dev[i] becomes a fork of row source_dev[i] (i < n): it shares the
 * len / page_size full pages of len = kv_len_dev[source] tokens, and gets a page
 * of its own for the rest, if any; its other entries become -1 (what it held
 * must have been freed). copies_dev i32 [n, 2] = (page to copy from, page to copy
 * to) for moe_pages_copy, or (-1, -1). A row may be forked many times; a target
 * that comes twice (after its first), or a source that is also a target, is
 * passed over and sets MOE_WS_INDEX. n 0 .. 1024. */
int moe_pages_fork(const moe_page_pool *pool, int32_t *table_dev, int64_t table_stride, int table_pages, int rows,
                   const int32_t *kv_len_dev, const int32_t *source_dev, const int32_t *target_dev, int n,
                   int32_t *copies_dev, uint32_t *status_dev, moe_stream_t stream);

/* Gives back all entries of rows rows_dev[i] (i < n; a row that comes twice is
 * freed once): they become -1, and pages that no entry holds any more are free. */
int moe_pages_free(const moe_page_pool *pool, int32_t *table_dev, int64_t table_stride, int table_pages, int rows,
                   const int32_t *rows_dev, int n, uint32_t *status_dev, moe_stream_t stream);

/* Moves the pages held to the front of the pool: with L pages held, the held
 * pages from L on go, in order, to the free ones below L. copies_dev i32
 * [max_copies, 2] receives (from, to), then (-1, -1); *n_copies_dev their number;
 * refs_out_dev [n_pages] and table_out_dev (strides and rows as table) the pool's
 * counts and the table afterwards (they may be refs and table themselves). The
 * pages' contents are then moved by moe_pages_copy, for each cache. max_copies
 * n_pages / 2 at least, 2^30 at most. */
int moe_pages_compact(const moe_page_pool *pool, const int32_t *table_dev, int64_t table_stride, int table_pages,
                      int rows, int32_t *refs_out_dev, int32_t *table_out_dev, int32_t *copies_dev, int max_copies,
                      int32_t *n_copies_dev, uint32_t *status_dev, moe_stream_t stream);

/* Copies pages of `layers` caches (of any kind: pages of page_bytes bytes, layer
 * l's at pages_dev + l * layer_stride, n_pages of them): from copies_dev[i, 0]
 * to copies_dev[i, 1], i < n or, where n_copies_dev is not NULL, below that count
 * too. A negative pair is passed over; one outside the cache too, and sets
 * MOE_WS_INDEX. No page may be copied to twice, or be copied both from and to.
 * pages_dev, layer_stride (n_pages * page_bytes at least) and page_bytes multiples
 * of 16; n 0 .. 2^30. */
int moe_pages_copy(void *pages_dev, int64_t layer_stride, int layers, int64_t n_pages, int64_t page_bytes,
                   const int32_t *copies_dev, int n, const int32_t *n_copies_dev, uint32_t *status_dev,
                   moe_stream_t stream);

/* Last error message of the calling thread ("" if none). */
const char *moe_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_H */

"""GB300-native engine for one decode step of a DeepSeek-style MoE layer whose
routed experts stay in raw Q2_K / Q3_K blocks.

Thin Python binding of libmoe.so (include/moe.h): every function only turns
torch tensors into device pointers and calls the C ABI function of the same
name; all arithmetic runs in the CUDA kernels. Tensors must live on the
current CUDA device; work is enqueued on the current torch stream unless a
`stream` (torch.cuda.Stream or raw handle) is given.
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import numpy as np

from . import _lib

MOE_HDR_MISS = 1
MOE_HDR_NONFINITE = 2
MOE_WS_TIMEOUT = 1
MOE_WS_PLAN = 2
MOE_WS_TRIPLE = 4
MOE_WS_INDEX = 8
MOE_WS_NONFINITE = 16
MOE_WS_PAGES = 32
MOE_KV_Q8 = 0
MOE_KV_Q4 = 1
MOE_MAX_DRAFT = 64
MOE_BF16 = 0
MOE_F32 = 1
MOE_ROPE_PLAIN = 0
MOE_ROPE_LINEAR = 1
MOE_ROPE_BASE = 2
MOE_ROPE_PARTS = 3
MOE_ROPE_HALF = 0
MOE_ROPE_INTERLEAVED = 1
MOE_SHARED_BF16 = 0
MOE_SHARED_KQUANT = 1
MOE_GRAPH_SNAPSHOTS = 1
MOE_GRAPH_EAGER_FALLBACK = 2
MOE_GRAPH_TEST_FAIL_CAPTURE = 4
SLOT_TABLE_LAYERS = 64

__all__ = ["Config", "Arena", "Layer", "MoeError", "header_words", "workspace_bytes",
           "workspace_init", "router_logits", "quantize_q8_1", "route_select", "expert_step",
           "swiglu_q8", "layer_step", "host_io_bytes", "layer_step_host", "workspace_view",
           "read_status", "layer_step_profiled", "layer_step_static", "route_scores", "set_wait_limit_ns",
           "expert_step_unreleased", "gemm_bf16", "prefill_workspace_bytes", "prefill_step", "prefill_step_profiled", "prefill_status", "graph_snapshot_bytes", "HostSource",
           "ExpertCache", "slot_table_set", "dedupe_triples", "parse_header", "Graph",
           "KvCache", "kv_page_bytes", "kv_append", "kv_read", "tree_attention_workspace_bytes", "tree_attention",
           "spec_verify_workspace_bytes", "spec_verify",
           "rope_table", "rope", "LatentCache", "latent_page_bytes", "latent_append", "latent_read",
           "latent_attention_workspace_bytes", "latent_attention", "latent_prompt_attention",
           "PagePool", "pages_grow", "pages_fork", "pages_free", "pages_compact", "pages_copy"]


class MoeError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


def _check(rc: int):
    if rc != 0:
        raise MoeError(rc, _lib.moe().moe_last_error().decode())


def _stream(stream):
    if stream is None:
        import torch
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if hasattr(stream, "cuda_stream"):
        return C.c_void_p(stream.cuda_stream)
    return C.c_void_p(int(stream))


def _ptr(t):
    """Device (or host) address of a tensor / array / int; None stays NULL."""
    if t is None:
        return None
    if isinstance(t, int):
        return C.c_void_p(t)
    if isinstance(t, np.ndarray):
        return C.c_void_p(t.ctypes.data)
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return C.c_void_p(t.data_ptr())


@dataclass
class Config:
    """Layer configuration (page spark_model/layers/moe_v41.rs, struct MoeV41Cfg)."""
    dim: int
    inter: int
    n_routed: int
    topk: int
    norm_topk_prob: bool = True
    max_tokens: int = 1
    gate_temp: float = 1.0
    route_scale: float = 2.5
    swiglu_limit: float = 7.0

    def c(self) -> _lib.MoeCfg:
        return _lib.MoeCfg(self.dim, self.inter, self.n_routed, self.topk, int(bool(self.norm_topk_prob)),
                           self.max_tokens, self.gate_temp, self.route_scale, self.swiglu_limit)


@dataclass
class Arena:
    """Device expert arena (page .../moe_v41/device_route.rs, fn arena_of)."""
    base: object
    slot_bytes: int
    gate_off: int
    up_off: int
    down_off: int

    def c(self) -> _lib.MoeArena:
        return _lib.MoeArena(_ptr(self.base), self.slot_bytes, self.gate_off, self.up_off, self.down_off)


@dataclass
class Layer:
    """One layer's resident weights (page spark_model/layers/moe_v41.rs, MoeV41LayerWeights).
    sh_format: MOE_SHARED_BF16 (bf16 w1, w3, w2) or MOE_SHARED_KQUANT (Q2_K w1,
    w3 and Q3_K w2 blocks, laid out as a routed expert's gate, up, down)."""
    router_w: object
    bias: object
    slot_row: object
    sh_w1: object = None
    sh_w3: object = None
    sh_w2: object = None
    sh_format: int = 0

    def c(self) -> _lib.MoeLayer:
        return _lib.MoeLayer(_ptr(self.router_w), _ptr(self.bias), _ptr(self.slot_row), _ptr(self.sh_w1),
                             _ptr(self.sh_w3), _ptr(self.sh_w2), int(self.sh_format))


class HostSource:
    """Expert slot images in host memory (include/moe.h, moe_host_source_create):
    images[layer][expert] -> a host array (pinned torch tensor or numpy), kept alive here."""

    def __init__(self, images, n_layers: int, n_routed: int, image_bytes: int):
        self._keep = images
        ptrs = (C.c_void_p * (n_layers * n_routed))()
        for l in range(n_layers):
            for e in range(n_routed):
                img = images[l][e]
                ptrs[l * n_routed + e] = img.data_ptr() if hasattr(img, "data_ptr") else img.ctypes.data
        h = C.c_void_p()
        _check(_lib.moe().moe_host_source_create(C.cast(ptrs, C.c_void_p), n_layers, n_routed, image_bytes,
                                                 C.byref(h)))
        self._h = h

    def close(self):
        if self._h:
            _lib.moe().moe_host_source_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class ExpertCache:
    """LRU expert slots over an arena (include/moe.h, moe_cache_create). source:
    a HostSource (its fetch runs in the library), or a Python callable
    fetch(layer, expert, slot_address, slot_bytes, stream) -> int, or None."""

    def __init__(self, n_layers: int, n_routed: int, n_slots: int, arena: Arena, slot_table=None, source=None):
        lib = _lib.moe()
        self._keep = (arena, slot_table, source)
        if isinstance(source, HostSource):
            fn = C.cast(lib.moe_fetch_host_images, C.c_void_p)
            user = source._h
        elif source is not None:
            self._cb = _lib.FETCH_FN(lambda u, l, e, d, b, s: int(source(l, e, d, b, s)))
            fn = C.cast(self._cb, C.c_void_p)
            user = None
        else:
            fn, user = None, None
        h = C.c_void_p()
        _check(lib.moe_cache_create(n_layers, n_routed, n_slots, C.byref(arena.c()), _ptr(slot_table), fn, user,
                                    C.byref(h)))
        self._h = h

    def ensure(self, layer: int, experts, stream=None) -> int:
        e = np.ascontiguousarray(experts, dtype=np.int32)
        n = C.c_int(0)
        _check(_lib.moe().moe_cache_ensure(self._h, layer, C.c_void_p(e.ctypes.data), e.size, C.byref(n),
                                           _stream(stream)))
        return n.value

    def slot_of(self, layer: int, expert: int) -> int:
        sl = C.c_int32(0)
        _check(_lib.moe().moe_cache_slot_of(self._h, layer, expert, C.byref(sl)))
        return sl.value

    def stats(self):
        h, m, ev = C.c_uint64(0), C.c_uint64(0), C.c_uint64(0)
        _check(_lib.moe().moe_cache_stats(self._h, C.byref(h), C.byref(m), C.byref(ev)))
        return h.value, m.value, ev.value

    def close(self):
        if self._h:
            _lib.moe().moe_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def header_words(cfg: Config, m: int) -> int:
    n = _lib.moe().moe_header_words(C.byref(cfg.c()), m)
    if n < 0:
        _check(n)
    return n


def workspace_bytes(cfg: Config) -> int:
    b = C.c_size_t(0)
    _check(_lib.moe().moe_workspace_bytes(C.byref(cfg.c()), C.byref(b)))
    return b.value


def workspace_init(ws, stream=None):
    _check(_lib.moe().moe_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def router_logits(cfg: Config, x, w, logits, m: int, stream=None):
    _check(_lib.moe().moe_router_logits(C.byref(cfg.c()), _ptr(x), _ptr(w), _ptr(logits), m, _stream(stream)))


def quantize_q8_1(cfg: Config, x, m: int, out, stream=None):
    _check(_lib.moe().moe_quantize_q8_1(C.byref(cfg.c()), _ptr(x), m, _ptr(out), _stream(stream)))


def route_select(cfg: Config, logits, bias, slot_row, arena: Arena, m: int, header, plan_w, plan_rows, ptrs,
                 stream=None):
    _check(_lib.moe().moe_route_select(C.byref(cfg.c()), _ptr(logits), _ptr(bias), _ptr(slot_row),
                                       C.byref(arena.c()), m, _ptr(header), _ptr(plan_w), _ptr(plan_rows),
                                       _ptr(ptrs), _stream(stream)))


def expert_step(cfg: Config, x, ptrs, plan_w, plan_rows, header, m: int, acc, ws, stream=None):
    _check(_lib.moe().moe_expert_step(C.byref(cfg.c()), _ptr(x), _ptr(ptrs), _ptr(plan_w), _ptr(plan_rows),
                                      _ptr(header), m, _ptr(acc), _ptr(ws), _stream(stream)))


def swiglu_q8(cfg: Config, g, u, rows: int, h, hq8, stream=None):
    _check(_lib.moe().moe_swiglu_q8(C.byref(cfg.c()), _ptr(g), _ptr(u), rows, _ptr(h), _ptr(hq8),
                                    _stream(stream)))


def layer_step(cfg: Config, layer: Layer, arena: Arena, x, residual, x_next, header, m: int, ws, stream=None):
    _check(_lib.moe().moe_layer_step(C.byref(cfg.c()), C.byref(layer.c()), C.byref(arena.c()), _ptr(x),
                                     _ptr(residual), _ptr(x_next), _ptr(header), m, _ptr(ws), _stream(stream)))


def layer_step_static(cfg: Config, layer: Layer, arena: Arena, x, residual, x_next, header, m: int,
                      status=None, stream=None):
    """layer_step on the library's own static device workspace (no allocation).
    status: None, or a host uint32 array of one element that receives the
    workspace status once the stream reaches the end of the call."""
    _check(_lib.moe().moe_layer_step_static(C.byref(cfg.c()), C.byref(layer.c()), C.byref(arena.c()), _ptr(x),
                                            _ptr(residual), _ptr(x_next), _ptr(header), m, _ptr(status),
                                            _stream(stream)))


def set_wait_limit_ns(ns: int):
    """Bound (ns) on every wait inside kernels enqueued from now on; 0 = 2 s."""
    _check(_lib.moe().moe_set_wait_limit_ns(int(ns)))


def expert_step_unreleased(cfg: Config, x, header, m: int, ws, stream=None):
    """The expert kernels with no router before them: their wait for the plan
    can only run out (a failure-handling check; see include/moe.h)."""
    _check(_lib.moe().moe_expert_step_unreleased(C.byref(cfg.c()), _ptr(x), _ptr(header), m, _ptr(ws),
                                                 _stream(stream)))


def route_scores(cfg: Config, logits, scores, count: int, stream=None):
    """scores[i] = the f32 chain sqrt(ln_1p(exp(logits[i] / gate_temp))), each step correctly rounded."""
    _check(_lib.moe().moe_route_scores(C.byref(cfg.c()), _ptr(logits), count, _ptr(scores), _stream(stream)))


def host_io_bytes(cfg: Config, m: int) -> int:
    b = C.c_size_t(0)
    _check(_lib.moe().moe_host_io_bytes(C.byref(cfg.c()), m, C.byref(b)))
    return b.value


def layer_step_host(cfg: Config, layer: Layer, arena: Arena, x_host, residual_host, x_next_host, header_host,
                    m: int, io, ws, stream=None):
    """Host buffers (pinned torch CPU tensors or numpy arrays) in and out."""
    _check(_lib.moe().moe_layer_step_host(C.byref(cfg.c()), C.byref(layer.c()), C.byref(arena.c()),
                                          _ptr(x_host), _ptr(residual_host), _ptr(x_next_host),
                                          _ptr(header_host), m, _ptr(io), _ptr(ws), _stream(stream)))


def layer_step_profiled(cfg: Config, layer: Layer, arena: Arena, x, residual, x_next, header, m: int, ws,
                        stream=None):
    """-> [ms router+select, ms gate/up, ms down] for one layer step (kernels not overlapped)."""
    ms = np.zeros(3, np.float32)
    _check(_lib.moe().moe_layer_step_profiled(C.byref(cfg.c()), C.byref(layer.c()), C.byref(arena.c()), _ptr(x),
                                              _ptr(residual), _ptr(x_next), _ptr(header), m, _ptr(ws),
                                              _stream(stream), C.c_void_p(ms.ctypes.data)))
    return ms


def workspace_view(cfg: Config, ws) -> dict:
    v = _lib.MoeWsView()
    _check(_lib.moe().moe_workspace_view(C.byref(cfg.c()), _ptr(ws), C.byref(v)))
    return {name: getattr(v, name) for name, _ in _lib.MoeWsView._fields_}


def read_status(ws, stream=None) -> int:
    s = C.c_uint32(0)
    _check(_lib.moe().moe_read_status(_ptr(ws), C.byref(s), _stream(stream)))
    return s.value


def slot_table_set(table, n_routed: int, triples, n: int, status=None, stream=None):
    _check(_lib.moe().moe_slot_table_set(_ptr(table), n_routed, _ptr(triples), n, _ptr(status),
                                         _stream(stream)))


def dedupe_triples(triples: np.ndarray) -> np.ndarray:
    """Last-write-wins dedupe of (layer, expert, slot) triples (host)."""
    t = np.ascontiguousarray(triples, dtype=np.int32).reshape(-1, 3).copy()
    n = C.c_int(0)
    _check(_lib.moe().moe_dedupe_triples(C.c_void_p(t.ctypes.data), t.shape[0], C.byref(n)))
    return t[:n.value].copy()


def parse_header(cfg: Config, header_host: np.ndarray, m: int, t: int):
    """-> (status, picks, weights) of token t from a header copied to the host."""
    h = np.ascontiguousarray(header_host, dtype=np.int32)
    st = np.zeros(1, np.int32)
    picks = np.zeros(cfg.topk, np.int32)
    w = np.zeros(cfg.topk, np.float32)
    _check(_lib.moe().moe_parse_header(C.byref(cfg.c()), C.c_void_p(h.ctypes.data), m, t,
                                       C.c_void_p(st.ctypes.data), C.c_void_p(picks.ctypes.data),
                                       C.c_void_p(w.ctypes.data)))
    return int(st[0]), picks, w


def gemm_bf16(a, b, d, M: int, N: int, K: int, ldd: int, stream=None):
    """d[n * ldd + r] = sum_k a[r, k] b[n, k] on the tensor cores (bf16 in, f32 out)."""
    _check(_lib.moe().moe_gemm_bf16(_ptr(a), _ptr(b), _ptr(d), M, N, K, ldd, _stream(stream)))


def prefill_workspace_bytes(cfg: Config, m: int) -> int:
    b = C.c_size_t(0)
    _check(_lib.moe().moe_prefill_workspace_bytes(C.byref(cfg.c()), m, C.byref(b)))
    return b.value


def prefill_step(cfg: Config, layer: Layer, arena: Arena, arena_slots: int, x, residual, x_next, picks, weights,
                 m: int, ws, stream=None):
    """The batched (prefill) layer step for m tokens (include/moe.h, moe_prefill_step)."""
    _check(_lib.moe().moe_prefill_step(C.byref(cfg.c()), C.byref(layer.c()), C.byref(arena.c()), int(arena_slots),
                                       _ptr(x), _ptr(residual), _ptr(x_next), _ptr(picks), _ptr(weights), m,
                                       _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def prefill_step_profiled(cfg: Config, layer: Layer, arena: Arena, arena_slots: int, x, residual, x_next, picks,
                          weights, m: int, ws, stream=None):
    """-> ms of the nine stages of one prefill step (include/moe.h, moe_prefill_step_profiled)."""
    ms = np.zeros(9, np.float32)
    _check(_lib.moe().moe_prefill_step_profiled(C.byref(cfg.c()), C.byref(layer.c()), C.byref(arena.c()),
                                                int(arena_slots), _ptr(x), _ptr(residual), _ptr(x_next), _ptr(picks),
                                                _ptr(weights), m, _ptr(ws), ws.numel() * ws.element_size(),
                                                _stream(stream), C.c_void_p(ms.ctypes.data)))
    return ms


def prefill_status(cfg: Config, m: int, ws, stream=None) -> int:
    s = C.c_uint32(0)
    _check(_lib.moe().moe_prefill_status(C.byref(cfg.c()), m, _ptr(ws), C.byref(s), _stream(stream)))
    return s.value


def graph_snapshot_bytes(cfg: Config, m: int, n_layers: int) -> int:
    b = C.c_size_t(0)
    _check(_lib.moe().moe_graph_snapshot_bytes(C.byref(cfg.c()), m, n_layers, C.byref(b)))
    return b.value


class Graph:
    """A captured multi-layer step (include/moe.h, moe_graph_create). snapshots:
    device memory of graph_snapshot_bytes (with MOE_GRAPH_SNAPSHOTS in flags)."""

    def __init__(self, cfg: Config, layers, arena: Arena, m: int, x_a, x_b, residual, headers, ws, snapshots=None,
                 flags: int = 0):
        arr = (_lib.MoeLayer * len(layers))(*[ly.c() for ly in layers])
        self._keep = (layers, arena, x_a, x_b, residual, headers, ws, snapshots)
        h = C.c_void_p()
        _check(_lib.moe().moe_graph_create(C.byref(cfg.c()), C.cast(arr, C.c_void_p), len(layers),
                                           C.byref(arena.c()), m, _ptr(x_a), _ptr(x_b), _ptr(residual),
                                           _ptr(headers), _ptr(ws), _ptr(snapshots), flags, C.byref(h)))
        self._h = h

    @property
    def eager(self) -> bool:
        e = C.c_int(0)
        _check(_lib.moe().moe_graph_is_eager(self._h, C.byref(e)))
        return bool(e.value)

    def rerun_from(self, layer: int, stream=None):
        _check(_lib.moe().moe_graph_rerun_from(self._h, layer, _stream(stream)))

    def step_cached(self, cache: "ExpertCache", headers_host: np.ndarray, stream=None) -> int:
        """One launch with misses fetched and the rest rerun (moe_graph_step_cached);
        -> layers rerun. headers_host: int32 numpy array of the graph's header rows."""
        n = C.c_int(0)
        _check(_lib.moe().moe_graph_step_cached(self._h, cache._h, C.c_void_p(headers_host.ctypes.data),
                                                C.byref(n), _stream(stream)))
        return n.value

    def launch(self, stream=None):
        _check(_lib.moe().moe_graph_launch(self._h, _stream(stream)))

    def launch_host(self, x_host, residual_host, x_out_host, residual_out_host, headers_host, stream=None):
        _check(_lib.moe().moe_graph_launch_host(self._h, _ptr(x_host), _ptr(residual_host), _ptr(x_out_host),
                                                _ptr(residual_out_host), _ptr(headers_host), _stream(stream)))

    def close(self):
        if self._h:
            _lib.moe().moe_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------ speculative decoding
#
# These calls run between others of a few microseconds each, so their host side
# is kept short: library and torch looked up once, addresses passed as integers.

_rt = None


class _Runtime:
    def __init__(self):
        import torch
        self.lib = _lib.moe()
        self.bf16, self.f32, self.i32 = torch.bfloat16, torch.float32, torch.int32
        self.rows = (torch.bfloat16, torch.int16, torch.uint16)  # bf16 or its bit patterns
        self.bits = (torch.int64, torch.uint64)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device, current = torch.cuda.current_device, torch.cuda.current_stream
        self.stream = (lambda: raw(device())) if raw is not None else (lambda: current().cuda_stream)
        self.raw = raw if raw is not None else (lambda d: current().cuda_stream)
        self.device = getattr(torch._C, "_cuda_getDevice", device)


def _runtime():
    global _rt
    if _rt is None:
        _rt = _Runtime()
    return _rt


def _on(rt, stream):
    if stream is None:
        return rt.stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t, name, dtype, n):
    """Address of a contiguous tensor of at least n values; None stays NULL."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} values, {n} are needed")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _bytes(ws):
    """Address and size of a workspace tensor."""
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _refuse_host(**tensors):
    """Refuses the first host tensor: its address means nothing to the kernels."""
    for name, t in tensors.items():
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU, not on {t.device}")


def _matrix(t, name, dtype, rows, columns):
    """Address and row stride of a [rows, columns] tensor whose rows are contiguous; None: NULL."""
    if t is None:
        return None, 0
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != columns:
        raise ValueError(f"{name} must be [{rows}, {columns}], not {list(t.shape)}")
    if columns > 1 and t.stride(1) != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), t.stride(0)


def _heads(rt, cache, t, name, heads):
    """Address, token stride and head stride of bf16 rows [tokens, heads, head_dim]."""
    if t.dtype not in rt.rows:
        raise ValueError(f"{name} must be bfloat16, not {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != cache.head_dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {cache.head_dim}], not {list(shape)}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), st, sh


@dataclass
class KvCache:
    """A paged cache of quantised keys and values (include/moe.h, moe_kv_cache).
    pages: uint8 device tensor of whole pages (kv_page_bytes each)."""
    pages: object
    head_dim: int
    n_kv_heads: int
    page_size: int = 64
    format: int = MOE_KV_Q8

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_ref", None)

    def __post_init__(self):
        self.ref()

    @property
    def n_pages(self) -> int:
        if self.pages is None:
            return 0
        per, size = kv_page_bytes(self), self.pages.numel() * self.pages.element_size()
        if size % per:
            raise ValueError(f"pages holds {size} bytes, not a multiple of a page's {per}")
        return size // per

    def ref(self):
        """The C struct by reference, made again after a field was set or the pages tensor got other memory."""
        pages = self.pages
        at = None if pages is None else (pages.data_ptr(), pages.numel())
        if self._ref is None or at != self._at:
            n_pages = self.n_pages
            c = _lib.MoeKvCache(_ptr(pages), n_pages, self.head_dim, self.n_kv_heads, self.page_size, self.format)
            object.__setattr__(self, "_ref", C.byref(c))
            object.__setattr__(self, "_at", at)
        return self._ref


def kv_page_bytes(cache: KvCache) -> int:
    b = C.c_size_t(0)
    c = _lib.MoeKvCache(None, 0, cache.head_dim, cache.n_kv_heads, cache.page_size, cache.format)
    _check(_lib.moe().moe_kv_page_bytes(C.byref(c), C.byref(b)))
    return b.value


def kv_append(cache: KvCache, k, v, slots, status=None, stream=None):
    """Quantise rows k, v (bf16 [tokens, n_kv_heads, head_dim], any strides of the
    first two) into slots (int32 [tokens], -1: skipped). status: None, or a
    device word (int32) that receives MOE_WS_* bits."""
    rt = _runtime()
    n, heads = k.shape[0], cache.n_kv_heads
    if n != v.shape[0]:
        raise ValueError("k and v must have the same number of tokens")
    args = (cache.ref(), *_heads(rt, cache, k, "k", heads), *_heads(rt, cache, v, "v", heads),
            _dev(slots, "slots", rt.i32, n), n, _dev(status, "status", rt.i32, 1), _on(rt, stream))
    if not (k.is_cuda and v.is_cuda and slots.is_cuda and cache.pages.is_cuda and (status is None or status.is_cuda)):
        _refuse_host(pages=cache.pages, k=k, v=v, slots=slots, status=status)
    rc = rt.lib.moe_kv_append(*args)
    if rc:
        _check(rc)


def kv_read(cache: KvCache, slots, k_out, v_out, status=None, stream=None):
    """Rows of the cache as numbers: k_out, v_out bf16 or f32 [tokens, n_kv_heads, head_dim]."""
    rt = _runtime()
    n, kind = slots.numel(), k_out.dtype
    if kind is not rt.bf16 and kind is not rt.f32:
        raise ValueError(f"k_out must be bfloat16 or float32, not {kind}")
    size = n * cache.n_kv_heads * cache.head_dim
    args = (cache.ref(), _dev(slots, "slots", rt.i32, n), n, _dev(k_out, "k_out", kind, size),
            _dev(v_out, "v_out", kind, size), MOE_F32 if kind is rt.f32 else MOE_BF16,
            _dev(status, "status", rt.i32, 1), _on(rt, stream))
    if not (slots.is_cuda and k_out.is_cuda and v_out.is_cuda and cache.pages.is_cuda and
            (status is None or status.is_cuda)):
        _refuse_host(pages=cache.pages, slots=slots, k_out=k_out, v_out=v_out, status=status)
    rc = rt.lib.moe_kv_read(*args)
    if rc:
        _check(rc)


def tree_attention_workspace_bytes(cache: KvCache, n_q_heads: int, batch: int, n_tokens: int) -> int:
    b = C.c_size_t(0)
    _check(_lib.moe().moe_tree_attention_workspace_bytes(cache.ref(), n_q_heads, batch, n_tokens, C.byref(b)))
    return b.value


def tree_attention(cache: KvCache, q, out, q_start, kv_len, table, mask, scale: float, ws, stream=None):
    """Attention of each sequence's drafted tokens over the cache (include/moe.h,
    moe_tree_attention): q, out bf16 [tokens, n_q_heads, head_dim], q_start int32
    [batch + 1], kv_len int32 [batch], table int32 [batch, pages], mask int64
    [tokens] of bits, or None for chains and single tokens."""
    rt = _runtime()
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    n, heads = q.shape[:2]
    batch = kv_len.numel()
    if mask is not None and mask.dtype not in rt.bits:
        raise ValueError(f"mask must be int64, not {mask.dtype}")
    tp, ts = _matrix(table, "table", rt.i32, batch, table.shape[-1])
    args = (cache.ref(), *_heads(rt, cache, q, "q", heads), *_heads(rt, cache, out, "out", heads),
            heads, _dev(q_start, "q_start", rt.i32, batch + 1), _dev(kv_len, "kv_len", rt.i32, batch), tp, ts,
            table.shape[1], None if mask is None else _dev(mask, "mask", mask.dtype, n), batch, n, scale,
            *_bytes(ws), _on(rt, stream))
    if not (q.is_cuda and out.is_cuda and q_start.is_cuda and kv_len.is_cuda and table.is_cuda and ws.is_cuda and
            cache.pages.is_cuda and (mask is None or mask.is_cuda)):
        _refuse_host(pages=cache.pages, q=q, out=out, q_start=q_start, kv_len=kv_len, table=table, mask=mask, ws=ws)
    rc = rt.lib.moe_tree_attention(*args)
    if rc:
        _check(rc)


def spec_verify_workspace_bytes(batch: int, n_rows: int) -> int:
    b = C.c_size_t(0)
    _check(_lib.moe().moe_spec_verify_workspace_bytes(batch, n_rows, C.byref(b)))
    return b.value


def spec_verify(logits, q_start, tokens, parents, draft, temperature, uniforms, noise, n_accepted, path, next_token,
                ws, stream=None):
    """Verify drafted tokens from given random numbers (include/moe.h, moe_spec_verify):
    logits bf16 or f32 [rows, vocab], draft f32 [rows, vocab] or None, noise f32
    [batch, vocab]; the other inputs as there. Outputs int32: n_accepted [batch],
    path [rows], next_token [batch]."""
    rt = _runtime()
    kind = logits.dtype
    if kind is not rt.bf16 and kind is not rt.f32:
        raise ValueError(f"logits must be bfloat16 or float32, not {kind}")
    rows, vocab = logits.shape
    batch, i32, f32 = next_token.numel(), rt.i32, rt.f32
    lp, ls = _matrix(logits, "logits", kind, rows, vocab)
    dp, ds = _matrix(draft, "draft", f32, rows, vocab)
    np_, ns = _matrix(noise, "noise", f32, batch, vocab)
    args = (lp, MOE_F32 if kind is f32 else MOE_BF16, ls, _dev(q_start, "q_start", i32, batch + 1),
            _dev(tokens, "tokens", i32, rows), _dev(parents, "parents", i32, rows), dp, ds,
            _dev(temperature, "temperature", f32, batch), _dev(uniforms, "uniforms", f32, rows),
            np_, ns, batch, rows, vocab, _dev(n_accepted, "n_accepted", i32, batch),
            _dev(path, "path", i32, rows), _dev(next_token, "next_token", i32, batch),
            *_bytes(ws), _on(rt, stream))
    if not (logits.is_cuda and q_start.is_cuda and tokens.is_cuda and n_accepted.is_cuda and path.is_cuda and
            next_token.is_cuda and ws.is_cuda and (parents is None or parents.is_cuda) and
            (draft is None or draft.is_cuda) and (temperature is None or temperature.is_cuda) and
            (uniforms is None or uniforms.is_cuda) and (noise is None or noise.is_cuda)):
        _refuse_host(logits=logits, q_start=q_start, tokens=tokens, parents=parents, draft=draft, temperature=temperature,
                 uniforms=uniforms, noise=noise, n_accepted=n_accepted, path=path, next_token=next_token, ws=ws)
    rc = rt.lib.moe_spec_verify(*args)
    if rc:
        _check(rc)


# ------------------------------------------------------------------ positions, latent attention, pages


def _on_gpu(**tensors):
    """Refuses the first tensor that is on the host, or on another GPU than the current one."""
    import torch
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU, not on {t.device}")
        if t.get_device() != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, which is not the current device")


def _here(rt, stream, d):
    """The stream's handle; whether device d (a tensor's get_device, -1 on the host) is the current one."""
    if d < 0:
        return 0, False
    now = rt.device()
    if stream is None:
        return rt.raw(now), d == now
    return (stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)), d == now


def _rows3(t, name, kinds, heads, dim):
    """Address, token stride and head stride of rows [tokens, heads, dim] with contiguous dimensions."""
    if t.dtype not in kinds:
        raise ValueError(f"{name} must be {kinds[0]}, not {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}], not {list(shape)}")
    st, sh, sd = t.stride()
    if sd != 1 and dim > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), st, sh


def _rows2(t, name, kinds, rows, dim):
    """Address and row stride of rows [at least `rows`, dim] with contiguous dimensions."""
    if t.dtype not in kinds:
        raise ValueError(f"{name} must be {kinds[0]}, not {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] < rows or shape[1] != dim:
        raise ValueError(f"{name} must be [{rows}, {dim}], not {list(shape)}")
    sr, sd = t.stride()
    if sd != 1 and dim > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return t.data_ptr(), sr


def _distinct(t, name):
    """Refuses an output whose rows share memory (an expanded tensor)."""
    if 0 in t.stride() and any(s == 0 and n > 1 for s, n in zip(t.stride(), t.shape)):
        raise ValueError(f"{name} is an output: its rows must not share memory")


def rope_table(dim: int, base: float = 10000.0, scaling: int = MOE_ROPE_PLAIN, factor: float = 1.0,
               original: float = 4096.0, slow: float = 1.0, fast: float = 32.0):
    """-> (frequencies uint64 numpy [dim / 2], magnitude): the part of a turn that a position adds, times 2^64
    (include/moe.h, moe_rope_table). On the device: torch.from_numpy(table.view(numpy.int64)).cuda()."""
    table = np.zeros(max(int(dim), 2) // 2, np.uint64)
    magnitude = C.c_float(1.0)
    cfg = _lib.MoeRopeCfg(dim, scaling, base, factor, original, slow, fast)
    _check(_lib.moe().moe_rope_table(C.byref(cfg), C.c_void_p(table.ctypes.data), C.byref(magnitude)))
    return table, magnitude.value


def rope(x, out, positions, table, offset: int = 0, layout: int = MOE_ROPE_HALF, magnitude: float = 1.0,
         transposed: bool = False, stream=None):
    """Rotary positions on dimensions offset .. offset + 2 * table.numel() - 1 of each head (include/moe.h, moe_rope):
    x, out bf16 or f32 [tokens, heads, head_dim], any strides of the first two (out may be x), positions int32
    [tokens], table int64 (rope_table's). transposed: turned back, as a gradient is."""
    rt = _rt or _runtime()
    kind = x.dtype
    if kind is rt.bf16:
        code = MOE_BF16
    elif kind is rt.f32:
        code = MOE_F32
    else:
        raise ValueError(f"x must be bfloat16 or float32, not {kind}")
    shape = x.shape
    if len(shape) != 3 or out.shape != shape:
        raise ValueError(f"x and out must both be [tokens, heads, head_dim], not {list(x.shape)} and {list(out.shape)}")
    if out.dtype is not kind:
        raise ValueError(f"out must be {kind}, not {out.dtype}")
    tokens, heads, dim = shape
    bits = table.dtype
    if bits not in rt.bits:
        raise ValueError(f"table must be int64, not {bits}")
    xt, xh, xd = x.stride()
    ot, oh, od = out.stride()
    if (xd != 1 or od != 1) and dim > 1:
        raise ValueError("the last dimension of x and out must be contiguous")
    if ot == 0 or oh == 0:
        _distinct(out, "out")
    pairs = table.numel()
    d = x.get_device()
    on, here = _here(rt, stream, d)
    args = (x.data_ptr(), xt, xh, out.data_ptr(), ot, oh, code, tokens, heads, dim, offset, 2 * pairs, layout,
            _dev(positions, "positions", rt.i32, tokens), _dev(table, "table", bits, 1), magnitude, 1 if transposed else 0, on)
    if not (here and out.get_device() == d and positions.get_device() == d and table.get_device() == d):
        _on_gpu(x=x, out=out, positions=positions, table=table)
    rc = rt.lib.moe_rope(*args)
    if rc:
        _check(rc)


@dataclass
class LatentCache:
    """A paged cache of latent vectors (include/moe.h, moe_latent_cache). pages: device tensor of whole pages
    (latent_page_bytes each), rows of latent_dim + rope_dim bf16 values."""
    pages: object
    latent_dim: int
    rope_dim: int
    page_size: int = 64

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        object.__setattr__(self, "_ref", None)

    def __post_init__(self):
        self.ref()

    @property
    def n_pages(self) -> int:
        if self.pages is None:
            return 0
        per, size = latent_page_bytes(self), self.pages.numel() * self.pages.element_size()
        if size % per:
            raise ValueError(f"pages holds {size} bytes, not a multiple of a page's {per}")
        return size // per

    def ref(self):
        """The C struct by reference, made again after a field was set or the pages tensor got other memory."""
        pages = self.pages
        at = None if pages is None else (pages.data_ptr(), pages.numel())
        if self._ref is None or at != self._at:
            c = _lib.MoeLatentCache(_ptr(pages), self.n_pages, self.latent_dim, self.rope_dim, self.page_size)
            object.__setattr__(self, "_ref", C.byref(c))
            object.__setattr__(self, "_at", at)
        return self._ref


def latent_page_bytes(cache: LatentCache) -> int:
    b = C.c_size_t(0)
    c = _lib.MoeLatentCache(None, 0, cache.latent_dim, cache.rope_dim, cache.page_size)
    _check(_lib.moe().moe_latent_page_bytes(C.byref(c), C.byref(b)))
    return b.value


def latent_append(cache: LatentCache, c, k_rope, slots, positions=None, table=None, layout: int = MOE_ROPE_HALF,
                  magnitude: float = 1.0, status=None, stream=None):
    """Write rows into slots (int32 [tokens], -1: skipped): latent vectors c [tokens, latent_dim] and key parts k_rope
    [tokens, rope_dim] (bf16, any row strides), the latter turned by positions (int32 [tokens]) and table (rope_table's)
    where they are given. status: None, or a device word (int32) that receives MOE_WS_* bits."""
    rt = _runtime()
    n = c.shape[0]
    if n != k_rope.shape[0]:
        raise ValueError("c and k_rope must have the same number of tokens")
    if table is not None and (table.dtype not in rt.bits or 2 * table.numel() != cache.rope_dim):
        raise ValueError(f"table must be int64 of {cache.rope_dim // 2} values, not {table.dtype} of {table.numel()}")
    d = c.get_device()
    on, here = _here(rt, stream, d)
    args = (cache.ref(), *_rows2(c, "c", rt.rows, n, cache.latent_dim),
            *_rows2(k_rope, "k_rope", rt.rows, n, cache.rope_dim), _dev(slots, "slots", rt.i32, n), n,
            _dev(positions, "positions", rt.i32, n), None if table is None else _dev(table, "table", table.dtype, 1),
            layout, magnitude, _dev(status, "status", rt.i32, 1), on)
    if not (here and cache.pages.get_device() == d and k_rope.get_device() == d and slots.get_device() == d and
            (positions is None or positions.get_device() == d) and (table is None or table.get_device() == d) and
            (status is None or status.get_device() == d)):
        _on_gpu(pages=cache.pages, c=c, k_rope=k_rope, slots=slots, positions=positions, table=table, status=status)
    rc = rt.lib.moe_latent_append(*args)
    if rc:
        _check(rc)


def latent_read(cache: LatentCache, slots, c_out, k_rope_out, status=None, stream=None):
    """Rows of the cache: c_out [tokens, latent_dim], k_rope_out [tokens, rope_dim], bf16, any row strides."""
    rt = _runtime()
    n = slots.numel()
    for t, name in ((c_out, "c_out"), (k_rope_out, "k_rope_out")):
        _distinct(t, name)
    d = c_out.get_device()
    on, here = _here(rt, stream, d)
    args = (cache.ref(), _dev(slots, "slots", rt.i32, n), n, *_rows2(c_out, "c_out", rt.rows, n, cache.latent_dim),
            *_rows2(k_rope_out, "k_rope_out", rt.rows, n, cache.rope_dim), _dev(status, "status", rt.i32, 1), on)
    if not (here and cache.pages.get_device() == d and k_rope_out.get_device() == d and slots.get_device() == d and
            (status is None or status.get_device() == d)):
        _on_gpu(pages=cache.pages, slots=slots, c_out=c_out, k_rope_out=k_rope_out, status=status)
    rc = rt.lib.moe_latent_read(*args)
    if rc:
        _check(rc)


def latent_attention_workspace_bytes(cache: LatentCache, heads: int, batch: int, n_tokens: int) -> int:
    b = C.c_size_t(0)
    _check(_lib.moe().moe_latent_attention_workspace_bytes(cache.ref(), heads, batch, n_tokens, C.byref(b)))
    return b.value


def latent_attention(cache: LatentCache, q, q_rope, out, q_start, kv_len, table, mask, scale: float, ws, stream=None):
    """Latent attention in absorbed form (include/moe.h, moe_latent_attention): q, out bf16 [tokens, heads, latent_dim],
    q_rope bf16 [tokens, heads, rope_dim]; the others as for tree_attention."""
    rt = _runtime()
    if q.dim() != 3 or out.shape != q.shape:
        raise ValueError("q must be [tokens, heads, latent_dim] and out have its shape")
    n, heads = q.shape[:2]
    if q_rope.shape[0] != n:
        raise ValueError("q and q_rope must have the same number of tokens")
    batch = kv_len.numel()
    if mask is not None and mask.dtype not in rt.bits:
        raise ValueError(f"mask must be int64, not {mask.dtype}")
    _distinct(out, "out")
    tp, ts = _matrix(table, "table", rt.i32, batch, table.shape[-1])
    d = q.get_device()
    on, here = _here(rt, stream, d)
    args = (cache.ref(), *_rows3(q, "q", rt.rows, heads, cache.latent_dim),
            *_rows3(q_rope, "q_rope", rt.rows, heads, cache.rope_dim), *_rows3(out, "out", rt.rows, heads, cache.latent_dim),
            heads, _dev(q_start, "q_start", rt.i32, batch + 1), _dev(kv_len, "kv_len", rt.i32, batch), tp, ts,
            table.shape[1], None if mask is None else _dev(mask, "mask", mask.dtype, n), batch, n, scale,
            *_bytes(ws), on)
    if not (here and cache.pages.get_device() == d and q_rope.get_device() == d and out.get_device() == d and
            q_start.get_device() == d and kv_len.get_device() == d and table.get_device() == d and ws.get_device() == d and
            (mask is None or mask.get_device() == d)):
        _on_gpu(pages=cache.pages, q=q, q_rope=q_rope, out=out, q_start=q_start, kv_len=kv_len, table=table,
                mask=mask, ws=ws)
    rc = rt.lib.moe_latent_attention(*args)
    if rc:
        _check(rc)


def latent_prompt_attention(q, k, k_rope, v, out, q_start, kv_start, causal: bool, scale: float, status=None, stream=None):
    """Latent attention in expanded form, for prompts (include/moe.h, moe_latent_prompt_attention): q bf16 [q tokens,
    heads, nope + rope], k, v [kv tokens, heads, nope], k_rope [kv tokens, rope], out [q tokens, heads, nope], any token
    and head strides; q_start, kv_start int32 [batch + 1]."""
    rt = _runtime()
    if q.dim() != 3 or k.dim() != 3 or k_rope.dim() != 2:
        raise ValueError("q and k must be [tokens, heads, dims], k_rope [tokens, dims]")
    n, heads, t, nope, rope_dim = q.shape[0], q.shape[1], k.shape[0], k.shape[2], k_rope.shape[1]
    if v.shape != k.shape or k_rope.shape[0] != t:
        raise ValueError("k, v and k_rope must have the same number of tokens, v k's shape")
    if out.shape[0] != n:
        raise ValueError("out must have q's number of tokens")
    batch = q_start.numel() - 1
    _distinct(out, "out")
    d = q.get_device()
    on, here = _here(rt, stream, d)
    args = (*_rows3(q, "q", rt.rows, heads, nope + rope_dim), *_rows3(k, "k", rt.rows, heads, nope),
            *_rows2(k_rope, "k_rope", rt.rows, t, rope_dim), *_rows3(v, "v", rt.rows, heads, nope),
            *_rows3(out, "out", rt.rows, heads, nope), heads, nope, rope_dim,
            _dev(q_start, "q_start", rt.i32, max(batch + 1, 1)), _dev(kv_start, "kv_start", rt.i32, max(batch + 1, 1)),
            max(batch, 0), n, t, int(bool(causal)), scale, _dev(status, "status", rt.i32, 1), on)
    if not (here and k.get_device() == d and k_rope.get_device() == d and v.get_device() == d and out.get_device() == d and
            q_start.get_device() == d and kv_start.get_device() == d and (status is None or status.get_device() == d)):
        _on_gpu(q=q, k=k, k_rope=k_rope, v=v, out=out, q_start=q_start, kv_start=kv_start, status=status)
    rc = rt.lib.moe_latent_prompt_attention(*args)
    if rc:
        _check(rc)


@dataclass
class PagePool:
    """A pool of pages (include/moe.h, moe_page_pool). refs: int32 device tensor, how many table entries hold each page."""
    refs: object
    page_size: int = 64

    def ref(self):
        """The C struct by reference, made again after a field was set or the refs tensor got other memory."""
        refs = self.refs
        if refs.dtype is not _runtime().i32:
            raise ValueError(f"refs must be int32, not {refs.dtype}")
        if not refs.is_contiguous():
            raise ValueError("refs must be contiguous")
        at = (refs.data_ptr(), refs.numel(), self.page_size)
        kept = self.__dict__.get("_kept")
        if kept is None or kept[0] != at:
            kept = self.__dict__["_kept"] = (at, C.byref(_lib.MoePagePool(_ptr(refs), at[1], at[2])))
        return kept[1]


def _pool_table(rt, pool, table, name="table"):
    """The pool; address, row stride, entries a row and rows of a table."""
    if table.dtype is not rt.i32:
        raise ValueError(f"{name} must be int32, not {table.dtype}")
    shape = table.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be [rows, pages], not {list(shape)}")
    sr, se = table.stride()
    if se != 1 and shape[1] > 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    if sr == 0:
        _distinct(table, name)
    return pool.ref(), table.data_ptr(), sr, shape[1], shape[0]


def pages_grow(pool: PagePool, table, lengths, status=None, stream=None):
    """Give each row of the table (int32 [rows, pages], -1: none) the pages that lengths (int32 [rows]) tokens need
    (include/moe.h, moe_pages_grow)."""
    rt = _rt or _runtime()
    head = _pool_table(rt, pool, table)
    d = table.get_device()
    on, here = _here(rt, stream, d)
    args = (*head, _dev(lengths, "lengths", rt.i32, head[4]), _dev(status, "status", rt.i32, 1), on)
    if not (here and pool.refs.get_device() == d and lengths.get_device() == d and
            (status is None or status.get_device() == d)):
        _on_gpu(refs=pool.refs, table=table, lengths=lengths, status=status)
    rc = rt.lib.moe_pages_grow(*args)
    if rc:
        _check(rc)


def pages_fork(pool: PagePool, table, kv_len, source, target, copies, status=None, stream=None):
    """Row target[i] of the table becomes a fork of row source[i] (include/moe.h, moe_pages_fork): full pages shared, a
    part-filled last one to be copied as copies [n, 2] (int32) says (pages_copy). kv_len int32 [rows]."""
    rt = _rt or _runtime()
    n = source.numel()
    head = _pool_table(rt, pool, table)
    d = table.get_device()
    on, here = _here(rt, stream, d)
    args = (*head, _dev(kv_len, "kv_len", rt.i32, head[4]), _dev(source, "source", rt.i32, n),
            _dev(target, "target", rt.i32, n), n, _dev(copies, "copies", rt.i32, 2 * n), _dev(status, "status", rt.i32, 1), on)
    if not (here and pool.refs.get_device() == d and kv_len.get_device() == d and source.get_device() == d and
            target.get_device() == d and copies.get_device() == d and (status is None or status.get_device() == d)):
        _on_gpu(refs=pool.refs, table=table, kv_len=kv_len, source=source, target=target, copies=copies,
                status=status)
    rc = rt.lib.moe_pages_fork(*args)
    if rc:
        _check(rc)


def pages_free(pool: PagePool, table, rows, status=None, stream=None):
    """Give back the pages of the table's rows `rows` (int32); their entries become -1."""
    rt = _rt or _runtime()
    d = table.get_device()
    on, here = _here(rt, stream, d)
    args = (*_pool_table(rt, pool, table), _dev(rows, "rows", rt.i32, 0), rows.numel(), _dev(status, "status", rt.i32, 1), on)
    if not (here and pool.refs.get_device() == d and rows.get_device() == d and (status is None or status.get_device() == d)):
        _on_gpu(refs=pool.refs, table=table, rows=rows, status=status)
    rc = rt.lib.moe_pages_free(*args)
    if rc:
        _check(rc)


def pages_compact(pool: PagePool, table, refs_out, table_out, copies, n_copies, status=None, stream=None):
    """Move the pages held to the pool's front (include/moe.h, moe_pages_compact): counts and table afterwards in
    refs_out and table_out (which may be pool.refs and table), the moves in copies [at least n_pages / 2, 2] and
    n_copies [1] (int32) for pages_copy."""
    rt = _runtime()
    if table_out.shape != table.shape or table_out.stride() != table.stride():
        raise ValueError("table_out must have the table's shape and strides")
    head = _pool_table(rt, pool, table)
    args = (*head, _dev(refs_out, "refs_out", rt.i32, pool.refs.numel()), _pool_table(rt, pool, table_out, "table_out")[1],
            _dev(copies, "copies", rt.i32, 2), copies.numel() // 2, _dev(n_copies, "n_copies", rt.i32, 1),
            _dev(status, "status", rt.i32, 1), _on(rt, stream))
    _on_gpu(refs=pool.refs, table=table, refs_out=refs_out, table_out=table_out, copies=copies, n_copies=n_copies,
            status=status)
    rc = rt.lib.moe_pages_compact(*args)
    if rc:
        _check(rc)


def pages_copy(pages, copies, n_copies=None, status=None, stream=None):
    """Copy pages as copies [n, 2] (int32: from, to) says, n_copies [1] of them where it is given, in every layer of
    pages [layers, n_pages, ...] (each layer contiguous; include/moe.h, moe_pages_copy)."""
    rt = _rt or _runtime()
    shape, strides = pages.shape, pages.stride()
    if len(shape) < 3:
        raise ValueError(f"pages must be [layers, n_pages, ...], not {list(pages.shape)}")
    layers, n_pages = shape[:2]
    per = 1
    for n, st in zip(reversed(shape[2:]), reversed(strides[2:])):
        if n != 1 and st != per:
            raise ValueError("each layer of pages must be contiguous")
        per *= n
    if n_pages > 1 and strides[1] != per:
        raise ValueError("each layer of pages must be contiguous")
    if strides[0] == 0 and layers > 1:
        raise ValueError("pages is an output: its layers must not share memory")
    size, d = pages.element_size(), pages.get_device()
    on, here = _here(rt, stream, d)
    args = (pages.data_ptr(), strides[0] * size, layers, n_pages, per * size, _dev(copies, "copies", rt.i32, 0),
            copies.numel() // 2, _dev(n_copies, "n_copies", rt.i32, 1), _dev(status, "status", rt.i32, 1), on)
    if not (here and copies.get_device() == d and (n_copies is None or n_copies.get_device() == d) and
            (status is None or status.get_device() == d)):
        _on_gpu(pages=pages, copies=copies, n_copies=n_copies, status=status)
    rc = rt.lib.moe_pages_copy(*args)
    if rc:
        _check(rc)

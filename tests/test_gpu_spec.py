"""The quantised cache, tree attention and draft verification on the GPU against plain
64-bit implementations (spec_ref.py).

Tolerances. Codes, scales and the values read back: exact (the definition's f32
operations are deterministic; bf16 output rounds the exact value once). Attention: the
bound spec_ref.attention derives from the documented roundings. Verification: the same
integers, where no decision of the 64-bit run is closer than 1e-5 (f32 exponentials, sums
over the vocabulary)."""
import math
import random

import numpy as np
import pytest
import torch

import moe_decode_quantized_gb300 as moe

import spec_ref

pytestmark = pytest.mark.gpu

FMTS = [moe.MOE_KV_Q8, moe.MOE_KV_Q4]
MARGIN = 1e-5


def make_cache(fmt, dim, heads, page, pages, fill=0xFF):
    per = spec_ref.block_bytes(fmt, dim) * heads * page // 16
    return moe.KvCache(torch.full((pages * per,), fill, dtype=torch.uint8, device="cuda"), dim, heads, page, fmt)


def bf16_rows(rng, shape, spread=True):
    x = rng.standard_normal(shape)
    if spread:  # rows of many magnitudes, a large channel, a row of zeros, one of equal values
        x = x * 10.0 ** rng.uniform(-3, 2, shape[:-1] + (1,))
        x[..., 3] *= 20
        x[shape[0] // 2] = 0.0
        x[-1] = -1.625
    return torch.from_numpy(x.astype(np.float32)).bfloat16()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


# ------------------------------------------------------------------ the cache

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,heads,page,tokens", [(64, 1, 16, 1), (64, 3, 48, 37), (128, 2, 16, 50),
                                                   (128, 8, 64, 16), (256, 2, 32, 33)])
def test_append_writes_the_documented_bytes(fmt, dim, heads, page, tokens):
    rng = np.random.default_rng(dim + tokens)
    k, v = bf16_rows(rng, (tokens, heads, dim)), bf16_rows(rng, (tokens, heads, dim))
    pages = tokens // page + 3
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    if tokens > 4:
        slots[2] = -1
    cache = make_cache(fmt, dim, heads, page, pages)
    want = np.full(cache.pages.numel(), 0xFF, np.uint8)
    for rows, value in ((k, False), (v, True)):
        c, d, m, _ = spec_ref.quantise(f64(rows), fmt)
        for t in range(tokens):
            for h in range(heads):
                if slots[t] >= 0:
                    spec_ref.store_row(want, fmt, heads, page, int(slots[t]), h, value, c[t, h], d[t, h],
                                       None if m is None else m[t, h])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.kv_append(cache, k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), status)
    assert np.array_equal(cache.pages.cpu().numpy(), want)  # and not a byte beside the rows' own
    assert status.item() == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim,heads,page,tokens,layout", [(128, 4, 32, 129, "qkv"), (64, 5, 16, 77, "heads"),
                                                          (128, 2, 64, 40, "odd"), (256, 1, 128, 300, "plain")])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_read_gives_the_quantised_values(fmt, dim, heads, page, tokens, layout, out):
    rng = np.random.default_rng(tokens)
    k, v = bf16_rows(rng, (tokens, heads, dim)), bf16_rows(rng, (tokens, heads, dim))
    want = [spec_ref.quantise(f64(x), fmt)[3] for x in (k, v)]
    pages = tokens // page + 2
    slots = torch.from_numpy(rng.permutation(pages * page)[:tokens].astype(np.int32)).cuda()
    kd, vd = k.cuda(), v.cuda()
    if layout == "qkv":
        qkv = torch.cat([kd, kd, vd], 1).contiguous()
        kd, vd = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
    elif layout == "heads":
        kd, vd = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (kd, vd))
    elif layout == "odd":  # neither 16-byte aligned nor a stride that is a multiple of 8
        big = torch.zeros((tokens, heads, dim + 3), dtype=torch.bfloat16, device="cuda")
        big[:, :, 3:] = kd
        kd = big[:, :, 3:]
    cache = make_cache(fmt, dim, heads, page, pages)
    moe.kv_append(cache, kd, vd, slots)
    read = slots.clone()
    read[tokens // 2] = -1
    ko, vo = (torch.full((tokens, heads, dim), 7.0, dtype=out, device="cuda") for _ in range(2))
    moe.kv_read(cache, read, ko, vo)
    for got, ref in zip((ko, vo), want):
        ref = ref.copy()
        ref[tokens // 2] = 0.0
        ref = ref.astype(np.float32).astype(np.float64)
        assert np.array_equal(f64(got), spec_ref.bf16(ref) if out == torch.bfloat16 else ref)


@pytest.mark.parametrize("fmt", FMTS)
def test_append_of_extreme_values(fmt):
    """Values beyond the range, NaN and infinities: held at the limit or as 0, flagged; tiny ones to the nearest step."""
    x = torch.randn((6, 1, 64)).bfloat16()
    x[0, 0, 5] = float("nan")
    x[1, 0, 7] = float("inf")
    x[2, 0, 9] = -float("inf")
    x[3] = 3.0e38
    x[3, 0, ::2] = -3.0e38
    x[4] = x[4] * 1e-9
    x[5] = x[5] * 1e-38
    for rows, bits in ((x, moe.MOE_WS_NONFINITE), (x[3:], 0)):
        n = rows.shape[0]
        cache = make_cache(fmt, 64, 1, 16, 1)
        slots = torch.arange(n, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        moe.kv_append(cache, rows.cuda(), rows.cuda(), slots, status)
        ko, vo = (torch.empty((n, 1, 64), dtype=torch.float32, device="cuda") for _ in range(2))
        moe.kv_read(cache, slots, ko, vo)
        want = spec_ref.quantise(f64(rows), fmt)[3].astype(np.float32).astype(np.float64)
        assert np.array_equal(f64(ko), want) and np.array_equal(f64(vo), want)
        assert status.item() == bits


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_append_rounds_as_the_quotient(fmt, dim):
    """Numbers of few bits, whose quotients often lie halfway between two codes, at many magnitudes and odd scales."""
    rng = np.random.default_rng(dim)
    x = rng.integers(-255, 256, (512, 2, dim)) * 2.0 ** rng.integers(-20, 8, (512, 2, 1))
    x[::3] = np.round(x[::3] / 2) * 2 + 1  # odd multiples of half a step
    x[::4, :, ::32] = 31.75 * 2.0 ** rng.integers(-6, 6, (128, 2, 1))
    rows = torch.from_numpy(x.astype(np.float32)).bfloat16()
    cache = make_cache(fmt, dim, 2, 16, 33)
    slots = torch.arange(512, dtype=torch.int32, device="cuda") + 16
    moe.kv_append(cache, rows.cuda(), rows.cuda(), slots)
    ko, vo = (torch.empty((512, 2, dim), dtype=torch.float32, device="cuda") for _ in range(2))
    moe.kv_read(cache, slots, ko, vo)
    want = spec_ref.quantise(f64(rows), fmt)[3].astype(np.float32).astype(np.float64)
    assert np.array_equal(f64(ko), want) and np.array_equal(f64(vo), want)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("off", [16, 8, 1])
def test_append_of_rows_at_any_boundary(fmt, dim, off):
    """Rows on 32-byte, 16-byte and 2-byte boundaries give the same bytes."""
    rng = np.random.default_rng(off)
    k, v = bf16_rows(rng, (45, 3, dim)).cuda(), bf16_rows(rng, (45, 3, dim)).cuda()
    slots = torch.from_numpy(rng.permutation(96)[:45].astype(np.int32)).cuda()
    want, got = make_cache(fmt, dim, 3, 48, 2), make_cache(fmt, dim, 3, 48, 2)
    moe.kv_append(want, k, v, slots)
    wide = torch.zeros((45, 3, dim + off), dtype=torch.bfloat16, device="cuda")
    wide[:, :, off:] = k
    moe.kv_append(got, wide[:, :, off:], v, slots)
    assert torch.equal(want.pages, got.pages)


def test_slots_outside_the_cache():
    cache = make_cache(moe.MOE_KV_Q8, 64, 2, 16, 2)
    x = torch.randn((4, 2, 64), device="cuda").bfloat16()
    slots = torch.tensor([32, 0, -2, 1 << 30], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    moe.kv_append(cache, x, x, slots, status)
    assert status.item() == moe.MOE_WS_INDEX
    ko, vo = (torch.empty((4, 2, 64), dtype=torch.float32, device="cuda") for _ in range(2))
    moe.kv_read(cache, slots, ko, vo, status)
    assert (ko[[0, 2, 3]] == 0).all() and (vo[[0, 2, 3]] == 0).all()
    want = spec_ref.quantise(f64(x[1]), moe.MOE_KV_Q8)[3]
    assert np.array_equal(f64(ko[1]), want.astype(np.float32).astype(np.float64))
    before = cache.pages.clone()
    moe.kv_append(cache, x, x, torch.full((4,), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(cache.pages, before)


# ------------------------------------------------------------------ attention

class Sequences:
    """Sequences of given context lengths and query rows in one cache, pages in any order."""

    def __init__(self, fmt, dim, heads, group, page, ctx, rows, seed, kind="tree", pool_pages=None, k_scale=1.0):
        rng = np.random.default_rng(seed)
        pick = random.Random(seed)
        self.group, self.heads, self.scale = group, heads, 1.0 / math.sqrt(dim)
        lens = [c + n for c, n in zip(ctx, rows)]
        self.lens, self.rows = lens, rows
        counts = [-(-t // page) for t in lens]
        pool = pool_pages or sum(counts) + 1
        order = rng.permutation(min(pool, 4096))[:sum(counts)] + max(0, pool - 4096)
        if pool > 4096:  # spread over the whole pool, its ends included
            order[:min(2, len(order))] = [0, pool - 1][:len(order)]
        self.cache = make_cache(fmt, dim, heads, page, pool)
        table = np.full((len(ctx), max(counts + [1]) + 2), -7, np.int32)  # entries past a sequence are not read
        at, self.k, self.v, slots, ks, vs, self.masks = 0, [], [], [], [], [], []
        for b, t in enumerate(lens):
            table[b, :counts[b]] = order[at:at + counts[b]]
            at += counts[b]
            k = rng.standard_normal((t, heads, dim)) * k_scale
            k[..., 5] += 4.0
            v = rng.standard_normal((t, heads, dim)) + 0.25
            k, v = (torch.from_numpy(x.astype(np.float32)).bfloat16() for x in (k, v))
            slots += [int(table[b, j // page]) * page + j % page for j in range(t)]
            ks.append(k)
            vs.append(v)
            self.k.append(spec_ref.quantise(f64(k), fmt)[3])
            self.v.append(spec_ref.quantise(f64(v), fmt)[3])
            n, masks = rows[b], []
            for i in range(n):
                parent = pick.randint(max(0, i - 3), i - 1) if i else -1
                masks.append((masks[parent] if i else 0) | 1 << i)
            if kind == "any":  # not a tree's: any bits, among them none
                masks = [pick.getrandbits(64) & pick.getrandbits(64) for _ in range(n)]
                if n:
                    masks[n // 2] = 0
            self.masks += masks
        self.kind = kind
        if slots:
            moe.kv_append(self.cache, torch.cat(ks).cuda(), torch.cat(vs).cuda(),
                          torch.tensor(slots, dtype=torch.int32, device="cuda"))
        self.table = torch.from_numpy(table).cuda()
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
        signed = [m - (1 << 64) if m >> 63 else m for m in self.masks]
        self.mask = torch.tensor(signed, dtype=torch.int64, device="cuda") if kind != "chain" else None
        q = rng.standard_normal((sum(rows), heads * group, dim)) * 1.5
        self.q = torch.from_numpy(q.astype(np.float32)).bfloat16().cuda()

    def workspace(self):
        ws = torch.empty(moe.tree_attention_workspace_bytes(self.cache, self.heads * self.group, len(self.rows),
                                                            self.q.shape[0]), dtype=torch.uint8, device="cuda")
        moe.workspace_init(ws)
        return ws

    def run(self, ws=None, q=None, out=None):
        ws = self.workspace() if ws is None else ws
        q = self.q if q is None else q
        out = torch.full_like(self.q, 77.0) if out is None else out
        moe.tree_attention(self.cache, q, out, self.q_start, self.kv_len, self.table, self.mask, self.scale, ws)
        assert moe.read_status(ws) == 0
        return out

    def check(self, out, sequences=None):
        at = 0
        for b, n in enumerate(self.rows):
            if sequences is None or b in sequences:
                ref, bound = spec_ref.attention(f64(self.q[at:at + n]), self.k[b], self.v[b], n, self.group, self.scale,
                                                None if self.mask is None else self.masks[at:at + n])
                got = f64(out[at:at + n])
                assert np.isfinite(got).all(), b
                assert (np.abs(got - ref) <= bound).all(), (b, np.abs(got - ref).max(), (np.abs(got - ref) / bound).max())
            at += n


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,heads", [(1, 2), (4, 2), (5, 1), (16, 1)])
def test_single_tokens(fmt, dim, group, heads):
    s = Sequences(fmt, dim, heads, group, 32, [0, 1, 14, 15, 16, 31, 32, 127, 128, 300], [1] * 10, dim + group, "chain")
    s.check(s.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,rows", [(1, [1, 2, 64, 0, 3]), (4, [8, 1, 7, 8, 5]), (8, [64, 0, 2, 61, 33]),
                                        (3, [17, 64, 11, 1, 5])])
@pytest.mark.parametrize("kind", ["tree", "chain", "any"])
def test_trees(fmt, dim, group, rows, kind):
    s = Sequences(fmt, dim, 2, group, 16, [0, 40, 0, 129, 77], rows, dim * 31 + group, kind)
    out = s.run()
    s.check(out)
    if kind == "any":  # the sequences without a context: rows whose mask leaves nothing are zero
        at = 0
        for c, n in zip([0, 40, 0, 129, 77], rows):
            for i in range(n):
                if c == 0 and not s.masks[at + i] & ((1 << n) - 1):
                    assert (out[at + i] == 0).all()
            at += n


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("page", [16, 48, 64, 1024])
def test_pages_and_long_contexts(fmt, page):
    s = Sequences(fmt, 128, 1, 4, page, [5000, 17, 2047], [2, 3, 1], page, "tree")
    s.check(s.run())


def test_many_sequences():
    rng = np.random.default_rng(8)
    ctx = [int(c) for c in rng.integers(0, 400, 200)]
    s = Sequences(moe.MOE_KV_Q8, 64, 2, 2, 16, ctx, [int(n) for n in rng.integers(0, 4, 200)], 9, "tree")
    s.check(s.run())


@pytest.mark.parametrize("fmt,dim,group,nodes", [(moe.MOE_KV_Q8, 128, 4, 1), (moe.MOE_KV_Q8, 64, 2, 12),
                                                 (moe.MOE_KV_Q4, 128, 8, 20), (moe.MOE_KV_Q8, 256, 1, 3)])
@pytest.mark.parametrize("order", ["short first", "long first", "among"])
def test_short_items_beside_long_ones(fmt, dim, group, nodes, order):
    """Runs that begin and end in the part of an item's cost that is no unit, empty runs, items of one unit."""
    ctx = [0, 1, 3, 20, 0, 7] * 12
    ctx = {"short first": ctx + [9000], "long first": [9000] + ctx, "among": ctx[:30] + [9000, 0, 5000] + ctx[30:]}[order]
    s = Sequences(fmt, dim, 2, group, 64, ctx, [nodes if i % 5 else 0 for i in range(len(ctx))], dim + nodes, "tree")
    out = s.run()
    s.check(out)
    assert torch.equal(out, s.run())


@pytest.mark.parametrize("fmt,dim,group,nodes", [(moe.MOE_KV_Q8, 128, 2, 1), (moe.MOE_KV_Q8, 128, 64, 2),
                                                 (moe.MOE_KV_Q4, 128, 16, 4), (moe.MOE_KV_Q4, 256, 1, 2),
                                                 (moe.MOE_KV_Q8, 64, 16, 3)])
def test_the_largest_batch(fmt, dim, group, nodes):
    rng = np.random.default_rng(nodes)
    s = Sequences(fmt, dim, 1, group, 16, [int(c) for c in rng.integers(0, 60, 1024)], [nodes] * 1024, dim + nodes, "tree")
    s.check(s.run(), set(rng.integers(0, 1024, 40).tolist()) | {0, 1023})


@pytest.mark.parametrize("k_scale", [0.0, 40.0, 3000.0])
def test_large_and_equal_scores(k_scale):
    """Weights that are all alike, and scores of hundreds and thousands, where one token takes the whole weight."""
    s = Sequences(moe.MOE_KV_Q8, 128, 1, 4, 64, [700, 33], [8, 1], 3, "tree", k_scale=k_scale)
    s.check(s.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("group,rows", [(4, 1), (8, 8), (8, 40)])
def test_one_long_sequence(fmt, group, rows):
    """One head of one sequence over all CTAs: more partials than are weighed at once."""
    s = Sequences(fmt, 128, 1, group, 128, [40011], [rows], rows, "tree")
    s.check(s.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_large_groups(dim):
    s = Sequences(moe.MOE_KV_Q8, dim, 1, 64, 32, [300, 5, 77], [5, 1, 2], dim, "tree")
    s.check(s.run())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch,ctx,rows", [(300, 20, 9), (40, 500, 30), (3, 3000, 64)])
def test_many_and_few_items_of_many_rows(fmt, batch, ctx, rows):
    """Row blocks of one and of two M tiles, in runs that cut few items and in runs of many whole ones, mixed."""
    rng = np.random.default_rng(batch)
    s = Sequences(fmt, 128, 2, 8, 16, [int(c) for c in rng.integers(0, ctx, batch)],
                  [int(n) for n in rng.integers(0, rows + 1, batch)], batch, "tree")
    out = s.run()
    s.check(out, set(rng.integers(0, batch, 12).tolist()) | {0, batch - 1})
    assert torch.isfinite(out).all()


def test_strides_of_many_rows():
    s = Sequences(moe.MOE_KV_Q8, 128, 2, 4, 32, [900, 5, 64], [64, 33, 40], 17, "tree")
    ws = s.workspace()
    want = s.run(ws)
    s.check(want)
    n, heads, dim = s.q.shape
    odd = torch.zeros((n, heads, dim + 1), dtype=torch.bfloat16, device="cuda")
    odd[:, :, 1:] = s.q
    got = torch.zeros((heads, n, dim + 3), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    s.run(ws, odd[:, :, 1:], got[:, :, 3:])
    assert torch.equal(got[:, :, 3:], want) and (got[:, :, :3] == 0).all()


def test_strides_streams_and_repeats():
    """q and out as views (a fused projection's output; heads first), another stream, and the same bits each time on a
    workspace that other calls used."""
    s = Sequences(moe.MOE_KV_Q8, 128, 2, 4, 32, [900, 5, 64], [8, 1, 3], 12, "tree")
    ws = s.workspace()
    want = s.run(ws)
    s.check(want)
    n, heads, dim = s.q.shape
    fused = torch.zeros((n, heads + 4, dim), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:2 + heads] = s.q
    out = torch.zeros((heads, n, dim), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    s.run(ws, fused[:, 2:2 + heads], out)
    assert torch.equal(out, want)
    odd = torch.zeros((n, heads, dim + 1), dtype=torch.bfloat16, device="cuda")  # rows off the 4-byte boundaries
    odd[:, :, 1:] = s.q
    got = torch.zeros((n, heads, dim + 3), dtype=torch.bfloat16, device="cuda")
    s.run(ws, odd[:, :, 1:], got[:, :, 3:])
    assert torch.equal(got[:, :, 3:], want) and (got[:, :, :3] == 0).all()
    big = Sequences(moe.MOE_KV_Q8, 128, 2, 4, 32, [3000, 2000], [1, 1], 13, "chain")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(5):
            assert torch.equal(s.run(ws), want)
            moe.tree_attention(big.cache, big.q, torch.empty_like(big.q), big.q_start, big.kv_len, big.table, None,
                               big.scale, big.workspace())
    torch.cuda.synchronize()


def test_captured_in_a_graph():
    """Lengths, tables and masks are read on the device: a captured call follows them."""
    s = Sequences(moe.MOE_KV_Q8, 128, 2, 4, 32, [700, 90], [4, 2], 21, "tree")
    ws, out = s.workspace(), torch.empty_like(s.q)
    want = s.run(ws).clone()
    short = s.kv_len.clone()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        moe.tree_attention(s.cache, s.q, out, s.q_start, s.kv_len, s.table, s.mask, s.scale, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    s.kv_len.copy_(torch.tensor([300, 40], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    assert torch.equal(got, s.run(ws)) and not torch.equal(got, want)
    s.kv_len.copy_(short)


def test_offsets_beyond_32_bits():
    """A pool of more than 4 GiB, with pages at its ends."""
    page_bytes = spec_ref.block_bytes(moe.MOE_KV_Q8, 128) * 8 * 4
    pool = (9 << 30) // page_bytes
    s = Sequences(moe.MOE_KV_Q8, 128, 8, 1, 64, [200, 65], [2, 1], 4, "tree", pool_pages=pool)
    assert int(s.table.max()) == pool - 1 and (pool - 1) * page_bytes > 1 << 33
    s.check(s.run())


def test_stale_bytes_and_masked_values_do_not_reach_a_row():
    """Slots past a sequence's length hold any bytes (the pool is filled with 0xFF: scales of NaN), and a masked token's
    key and value may be as large as the cache holds."""
    s = Sequences(moe.MOE_KV_Q8, 128, 1, 4, 64, [37], [4], 6, "any")
    s.masks = [0b0001, 0b0000, 0b0101, 0b0001]
    s.mask.copy_(torch.tensor(s.masks, dtype=torch.int64))
    want = s.run()
    s.check(want)
    big = torch.full((1, 1, 128), 6.0e4, device="cuda").bfloat16()
    slot = int(s.table[0, 0]) * 64 + 38  # query row 1: seen by none
    moe.kv_append(s.cache, big, -big, torch.tensor([slot], dtype=torch.int32, device="cuda"))
    assert torch.equal(s.run(), want)


def test_a_row_of_nan_stays_alone():
    s = Sequences(moe.MOE_KV_Q8, 64, 2, 2, 32, [50, 9], [3, 2], 14, "tree")
    want = s.run()
    s.q[1, 1, 7] = float("nan")
    s.q[3, 0, 2] = float("inf")
    got = s.run()
    assert torch.isnan(got[1, 1]).all() and torch.isnan(got[3, 0]).all()
    got[1, 1], got[3, 0] = want[1, 1], want[3, 0]
    assert torch.equal(got, want)


def test_lengths_and_pages_outside():
    s = Sequences(moe.MOE_KV_Q8, 64, 1, 2, 16, [40, 20, 30], [2, 2, 2], 15, "tree")
    want = s.run()
    ws = s.workspace()

    def status():
        out = torch.full_like(s.q, 5.0)
        moe.tree_attention(s.cache, s.q, out, s.q_start, s.kv_len, s.table, s.mask, s.scale, ws)
        st = moe.read_status(ws)
        moe.workspace_init(ws)
        return st, out

    keep = s.kv_len.clone()
    for bad in (1, -3, 10 ** 6):  # fewer tokens than query rows; negative; more than the table has pages for
        s.kv_len[1] = bad
        st, out = status()
        assert st == moe.MOE_WS_INDEX
        assert torch.equal(out[:2], want[:2]) and torch.equal(out[4:], want[4:]) and (out[2:4] == 0).all()
    s.kv_len.copy_(keep)
    for bad in (-1, s.cache.n_pages, 1 << 30):
        old = int(s.table[0, 0])
        s.table[0, 0] = bad  # its sixteen tokens are not seen
        st, out = status()
        assert st == moe.MOE_WS_INDEX and torch.equal(out[2:], want[2:])
        ref, bound = spec_ref.attention(f64(s.q[:2]), s.k[0][16:], s.v[0][16:], 2, 2, s.scale, s.masks[:2])
        assert (np.abs(f64(out[:2]) - ref) <= bound).all()
        s.table[0, 0] = old
    starts = s.q_start.clone()
    s.q_start.copy_(torch.tensor([0, 2, 70, 6], dtype=torch.int32))
    st, out = status()
    assert st == moe.MOE_WS_INDEX and torch.equal(out[:2], want[:2])
    s.q_start.copy_(starts)
    assert torch.equal(s.run(ws), want)


# ------------------------------------------------------------------ verification

def verify(case, stream=None, ws=None):
    starts = np.concatenate([[0], np.cumsum([len(t) for t in case["tokens"]])]).astype(np.int32)
    batch, rows = len(case["tokens"]), int(starts[-1])

    def dev(x, kind):
        return None if x is None else torch.from_numpy(np.ascontiguousarray(np.concatenate(x), dtype=kind)).cuda()

    n_acc, nxt = (torch.full((batch,), 99, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.full((max(rows, 1),), 99, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.spec_verify_workspace_bytes(batch, rows), dtype=torch.uint8, device="cuda") if ws is None else ws
    moe.workspace_init(ws)
    logits = case["logits"]
    temp = None if case["temp"] is None else torch.tensor(case["temp"], dtype=torch.float32, device="cuda")
    noise = None if case["noise"] is None else torch.from_numpy(np.asarray(case["noise"], np.float32)).cuda()
    moe.spec_verify(logits, torch.from_numpy(starts).cuda(), dev(case["tokens"], np.int32), dev(case["parents"], np.int32),
                    case["draft"], temp, dev(case["u"], np.float32), noise, n_acc, path, nxt, ws)
    return n_acc.tolist(), path.tolist(), nxt.tolist(), moe.read_status(ws), starts


def verify_case(batch, nodes, vocab, kind, shape, drafts, seed, temps=(0.7, 1.0, 0.0), near=0.5):
    rng = np.random.default_rng(seed)
    pick = random.Random(seed)
    sizes = [pick.randint(1, nodes) for _ in range(batch)]
    rows = sum(sizes)
    logits = torch.from_numpy((rng.standard_normal((rows, vocab)) * 2.5).astype(np.float32))
    logits = logits.bfloat16() if kind == "bf16" else logits
    case = {"tokens": [], "parents": [] if shape == "tree" else None, "u": [], "logits": logits.cuda(),
            "temp": [temps[b % len(temps)] for b in range(batch)], "noise": rng.exponential(size=(batch, vocab)) + 1e-12}
    l, at, draft = f64(logits), 0, np.zeros((rows, vocab), np.float32)
    for b, n in enumerate(sizes):
        parents = [-1] + [pick.randint(0, j - 1) if shape == "tree" else j - 1 for j in range(1, n)]
        tokens = [0]
        t = case["temp"][b] or 0.5
        for j in range(1, n):
            z = l[at + parents[j]] / t + rng.standard_normal(vocab) * near
            p = np.exp(z - z.max())
            draft[at + j] = p / p.sum()
            tokens.append(int(rng.choice(vocab, p=p / p.sum())))
        case["tokens"].append(np.array(tokens))
        case["u"].append(rng.random(n))
        if shape == "tree":
            case["parents"].append(np.array(parents))
        at += n
    case["draft"] = torch.from_numpy(draft).cuda() if drafts else None
    return case


def check_verify(case):
    n_acc, path, nxt, status, starts = verify(case)
    l = f64(case["logits"])
    draft = None if case["draft"] is None else case["draft"].cpu().numpy()
    sure = 0
    for b, tokens in enumerate(case["tokens"]):
        at, n = starts[b], len(tokens)
        want, last, margin = spec_ref.verify(
            l[at:at + n], tokens, None if case["parents"] is None else case["parents"][b],
            None if draft is None else draft[at:at + n], 1.0 if case["temp"] is None else case["temp"][b],
            None if case["u"] is None else np.float32(case["u"][b]).astype(np.float64),
            None if case["noise"] is None else np.float32(case["noise"][b]).astype(np.float64))
        if margin > MARGIN:
            sure += 1
            assert n_acc[b] == len(want) and nxt[b] == last, (b, margin)
            assert path[at:at + n] == want + [-1] * (n - len(want))
    assert sure >= 0.95 * len(case["tokens"]) - 1
    return status, n_acc


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", ["chain", "tree"])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("batch,nodes,vocab", [(1, 4, 32000), (40, 6, 1009), (17, 24, 257), (3, 64, 50001)])
def test_verify(kind, shape, drafts, batch, nodes, vocab):
    status, n_acc = check_verify(verify_case(batch, nodes, vocab, kind, shape, drafts, batch + vocab))
    assert status == 0


@pytest.mark.parametrize("kind,batch,vocab", [("f32", 20, 100003), ("bf16", 24, 131072), ("f32", 1, 1 << 22)])
@pytest.mark.parametrize("drafts", [True, False])
def test_verify_large_trees(kind, batch, vocab, drafts):
    """More logits than are gone through ahead: rows as the walk reaches them."""
    status, _ = check_verify(verify_case(batch, 24 if batch > 1 else 6, vocab, kind, "tree", drafts, vocab % 97))
    assert status == 0


@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 31, 1023, 8193, 131072])
def test_verify_vocabularies(vocab):
    for drafts in (True, False):
        status, _ = check_verify(verify_case(6, 3, vocab, "f32", "chain", drafts, vocab))
        assert status == 0


def test_verify_accepts_equal_distributions():
    """Drafts from the target's own distribution are all accepted: u Z q < r wherever u < 1 (a small slack: q in f32)."""
    case = verify_case(32, 8, 500, "f32", "chain", True, 3, temps=(1.0,), near=0.0)
    case["u"] = [np.minimum(u, 0.999) for u in case["u"]]
    status, n_acc = check_verify(case)
    assert status == 0 and n_acc == [len(t) - 1 for t in case["tokens"]]


def test_verify_greedy():
    """Without random numbers: the longest path of arg-max tokens; equal logits go to the lowest index."""
    case = verify_case(20, 8, 300, "bf16", "tree", False, 5, near=0.01)
    case["u"] = case["noise"] = None
    case["logits"][:, 7] = case["logits"][:, 250] = 30.0  # two largest
    for tokens in case["tokens"]:
        tokens[1:] = np.where(np.arange(1, len(tokens)) % 3 == 0, 250, 7)
    status, n_acc = check_verify(case)
    _, _, nxt, _, _ = verify(case)
    assert status == 0 and nxt == [7] * 20 and max(n_acc) >= 2
    case["temp"] = None
    assert verify(case)[2] == [7] * 20


def test_verify_masked_and_strange_logits():
    """-inf and the type's lowest value have no probability; NaN and +inf count as -inf and are flagged; a row without a
    finite logit gives -1."""
    case = verify_case(6, 3, 400, "f32", "chain", True, 6, temps=(1.0,))
    starts = np.concatenate([[0], np.cumsum([len(t) for t in case["tokens"]])])
    case["logits"][:, ::2] = -math.inf
    case["logits"][:, 1::4] = torch.finfo(torch.float32).min
    status, _ = check_verify(case)
    assert status == 0
    assert all(t % 4 == 3 for t in verify(case)[2])
    case["logits"][starts[1], 3] = float("nan")
    case["logits"][starts[2]:starts[3], 7] = float("inf")
    status, _ = check_verify(case)
    assert status == moe.MOE_WS_NONFINITE
    case["logits"][starts[4]:starts[5]] = -math.inf
    n_acc, path, nxt, _, _ = verify(case)
    assert n_acc[4] == 0 and nxt[4] == -1
    case["logits"][:] = torch.finfo(torch.float32).min  # all alike: a uniform distribution
    case["logits"][starts[3]] = 0.0
    status, _ = check_verify(case)
    assert status == 0


def test_verify_temperatures():
    """Very small, very large and infinite temperatures, and those that mean greedy."""
    case = verify_case(8, 4, 333, "f32", "chain", False, 7, temps=(1e-30, 1e30, math.inf, -1.0, 1e-3, 100.0, 5.0, 0.0))
    status, _ = check_verify(case)
    assert status == 0


def test_verify_tokens_and_rows_outside():
    case = verify_case(4, 5, 100, "f32", "tree", True, 8)
    case["tokens"] = [t.copy() for t in case["tokens"]]
    for t in case["tokens"]:
        t[1::2] = np.where(np.arange(len(t[1::2])) % 2 == 0, 100, -1)
    status, _ = check_verify(case)
    assert status == moe.MOE_WS_INDEX


def test_verify_strided_rows():
    """Rows of a wider tensor (a padded vocabulary)."""
    case = verify_case(9, 5, 777, "bf16", "tree", True, 10)
    want = verify(case)[:3]
    wide = torch.full((case["logits"].shape[0], 801), 50.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:780] = case["logits"]
    draft = torch.full((case["logits"].shape[0], 779), 1.0, device="cuda")
    draft[:, :777] = case["draft"]
    case["logits"], case["draft"] = wide[:, 3:780], draft[:, :777]
    assert verify(case)[:3] == want


def test_verify_follows_the_targets_distribution():
    """The first token out of a sequence (its accepted draft, or the next token) is distributed as the target's
    softmax, whatever the draft's distribution: chi-square over 20000 sequences, 11 degrees of freedom, limit at
    probability 1e-6."""
    rng = np.random.default_rng(2)
    batch, vocab = 20000, 12
    l = rng.standard_normal(vocab) * 1.2
    p = np.exp(l - l.max())
    p /= p.sum()
    for shape, n in (("chain", 2), ("tree", 4)):  # the tree: three drafts of the same parent
        q = rng.dirichlet(np.ones(vocab))
        q32 = q.astype(np.float32)
        tokens = rng.choice(vocab, size=(batch, n), p=q32.astype(np.float64) / q32.astype(np.float64).sum())
        case = {"tokens": list(tokens), "parents": [np.array([-1] + [0] * (n - 1))] * batch,
                "u": list(rng.random((batch, n))), "temp": None, "noise": rng.exponential(size=(batch, vocab)) + 1e-12,
                "logits": torch.from_numpy(np.broadcast_to(l.astype(np.float32), (batch * n, vocab)).copy()).cuda(),
                "draft": torch.from_numpy(np.broadcast_to(q32, (batch * n, vocab)).copy()).cuda()}
        n_acc, path, nxt, status, starts = verify(case)
        assert status == 0
        first = [tokens[b, path[starts[b]]] if n_acc[b] else nxt[b] for b in range(batch)]
        seen = np.bincount(first, minlength=vocab)
        assert ((seen - batch * p) ** 2 / (batch * p)).sum() < 51.0
        assert 0.2 * batch < sum(c > 0 for c in n_acc) < batch


# ------------------------------------------------------------------ together

def _example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decode.py")
    spec = importlib.util.spec_from_file_location("speculative_decode", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("fmt", FMTS)
def test_example_decodes_what_single_tokens_decode(fmt):
    """Greedy decoding with drafted trees: every token is the largest logit of the plain decode of the tokens before it
    (one token a step, another model object and cache), up to the rounding of the logits."""
    ex = _example()
    prompt, count = [3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5], 40
    out, rounds = ex.generate(ex.Model(seed=4, kv_format=fmt), prompt, count)
    assert rounds < len(out)  # some drafts were accepted
    plain = ex.Model(seed=4, kv_format=fmt)
    tokens = prompt + out
    for i, t in enumerate(tokens[:-1]):
        logits = plain.rows(torch.tensor([t], dtype=torch.int32, device="cuda"), i, None)[0]
        if i >= len(prompt) - 1:
            # bf16 activations: a few roundings of 2^-8 of logits of unit size times 4
            assert logits[tokens[i + 1]] >= logits.max() - 0.15, i


def test_example_samples():
    ex = _example()
    out, rounds = ex.generate(ex.Model(seed=5), [7, 7], 24, temperature=1.0)
    assert len(out) >= 24 and all(0 <= t < 512 for t in out)
    again, _ = ex.generate(ex.Model(seed=5), [7, 7], 24, temperature=1.0)
    assert out == again

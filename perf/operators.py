"""The cases at which the speculative-decoding operators are measured.

Four operators: a quantised paged cache written (kv_append) and read back
(kv_read), attention of one token, a chain or a tree of drafted tokens over it
(tree_attention), and the verification of drafted tokens against the target's
logits (spec_verify). `run` computes them in plain torch operations in 32 bits,
or, where `own` is set, by the calls of this package. The cache's byte layout,
which both read, is the one documented in include/moe.h (moe_kv_cfg).
"""
import math
import random

import numpy as np
import torch

own = False

GROUP = 32          # values with one scale
LIMIT = 60000.0     # largest magnitude the cache holds
Q8, Q4 = "q8", "q4"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 8 tokens (the largest small batch): latency
        {"name": "kv_decode_8", "op": "kv", "fmt": Q8, "tokens": 8, "heads": 8, "dim": 128, "page": 64,
         "pages": 64, "layout": "qkv", "out": "bf16"},
        # a prompt of 8192 tokens written from a fused QKV product
        {"name": "kv_prompt_8192", "op": "kv", "fmt": Q8, "tokens": 8192, "heads": 8, "dim": 128, "page": 64,
         "pages": 512, "layout": "qkv", "out": "bf16"},
        # an odd prompt at 4 bits, small heads, head-major source
        {"name": "kv_prompt_q4_4099", "op": "kv", "fmt": Q4, "tokens": 4099, "heads": 4, "dim": 64, "page": 16,
         "pages": 700, "layout": "heads", "out": "f32"},
        # a short sequence's rows read back (moving it to another pool)
        {"name": "read_q4_333", "op": "read", "fmt": Q4, "tokens": 333, "heads": 8, "dim": 128, "page": 32,
         "pages": 64, "out": "f32"},
        # a long context read back for a dense prefill pass
        {"name": "read_q8_65536", "op": "read", "fmt": Q8, "tokens": 65536, "heads": 8, "dim": 128, "page": 64,
         "pages": 1100, "out": "bf16"},
        # one token of one sequence, short context: latency
        {"name": "attn_one_b1_511", "op": "attn", "fmt": Q8, "dim": 128, "kv_heads": 8, "group": 4, "batch": 1,
         "nodes": 1, "ctx_lo": 511, "ctx_hi": 511, "page": 64, "shape": "one"},
        # a serving batch of ragged long contexts, one token each
        {"name": "attn_one_b64_24k", "op": "attn", "fmt": Q8, "dim": 128, "kv_heads": 8, "group": 4, "batch": 64,
         "nodes": 1, "ctx_lo": 4000, "ctx_hi": 24000, "page": 64, "shape": "one"},
        # trees of up to 8 drafted tokens (the small batch's size), 4-bit cache
        {"name": "attn_tree_q4_b16_16k", "op": "attn", "fmt": Q4, "dim": 128, "kv_heads": 8, "group": 4, "batch": 16,
         "nodes": 8, "ctx_lo": 1000, "ctx_hi": 16000, "page": 32, "shape": "tree"},
        # one sequence, a long context and a wide tree: many rows a kv head
        {"name": "attn_tree_b1_100k", "op": "attn", "fmt": Q8, "dim": 128, "kv_heads": 4, "group": 8, "batch": 1,
         "nodes": 61, "ctx_lo": 100003, "ctx_hi": 100003, "page": 64, "shape": "tree"},
        # a chain of 3 drafts of one sequence: latency
        {"name": "verify_chain_b1", "op": "verify", "batch": 1, "nodes": 4, "vocab": 32000, "type": "bf16",
         "shape": "chain", "drafts": "probs", "agree": 0.3, "greedy": False},
        # a serving batch of chains of 7 drafts, large vocabulary
        {"name": "verify_chain_b48", "op": "verify", "batch": 48, "nodes": 8, "vocab": 131072, "type": "bf16",
         "shape": "chain", "drafts": "probs", "agree": 0.3, "greedy": False},
        # trees drafted without probabilities, odd vocabulary, some greedy sequences
        {"name": "verify_tree_b16", "op": "verify", "batch": 16, "nodes": 24, "vocab": 100003, "type": "f32",
         "shape": "tree", "drafts": "tokens", "agree": 0.3, "greedy": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["kv", "read", "attn", "attn", "attn", "verify", "verify"])
        fmt = rng.choice([Q8, Q4])
        dim = rng.choice([64, 128, 128, 256])
        page = rng.choice([16, 32, 64, 128])
        if op in ("kv", "read"):
            n = _log(rng, 1, 8192 if op == "kv" else 65536)
            c = {"op": op, "fmt": fmt, "tokens": n, "heads": rng.choice([1, 2, 4, 8]), "dim": dim, "page": page,
                 "pages": n // page + 2 + rng.randint(0, 64), "out": rng.choice(["bf16", "f32"])}
            if op == "kv":
                c["layout"] = rng.choice(["qkv", "heads", "plain"])
        elif op == "attn":
            shape = rng.choice(["one", "chain", "tree"])
            hi = _log(rng, 1, 100003)
            c = {"op": op, "fmt": fmt, "dim": dim, "kv_heads": rng.choice([1, 2, 4, 8]),
                 "group": rng.choice([1, 2, 4, 5, 8, 16]), "batch": _log(rng, 1, 64),
                 "nodes": 1 if shape == "one" else _log(rng, 2, 64), "ctx_lo": rng.randint(0, hi), "ctx_hi": hi,
                 "page": page, "shape": shape}
        else:
            c = {"op": op, "batch": _log(rng, 1, 48), "nodes": _log(rng, 2, 24), "vocab": _log(rng, 1000, 131072),
                 "type": rng.choice(["bf16", "f32"]), "shape": rng.choice(["chain", "tree"]),
                 "drafts": rng.choice(["probs", "tokens"]), "agree": rng.choice([0.1, 0.3, 1.0]),
                 "greedy": rng.random() < 0.3}
        w, tops = work(c), [work(d) for d in listed() if d["op"] == c["op"]]
        room = max(_elements(d) for d in listed() if d["op"] == c["op"])
        if (w["bytes"] <= max(t["bytes"] for t in tops) and w["flops"] <= max(t["flops"] for t in tops)
                and _elements(c) <= room):
            return c


def _elements(c):
    """Values that a case's inputs stand for (bounds the plain form's memory)."""
    if c["op"] == "attn":
        return c["batch"] * (c["ctx_hi"] + c["nodes"]) * c["kv_heads"] * c["dim"]
    if c["op"] == "verify":
        return c["batch"] * c["nodes"] * c["vocab"] * (2 if c["drafts"] == "probs" else 1)
    return c["tokens"] * c["heads"] * c["dim"]


def _row_bytes(fmt, dim):
    """Cache bytes of one row (K or V of one token and head), scales included."""
    return dim + dim // GROUP * 2 if fmt == Q8 else dim // 2 + dim // GROUP * 4


def _tree_sizes(case):
    """Rows (last accepted token and drafts) of each sequence: the case's own, whatever the seed."""
    rng = random.Random(case["nodes"])
    if case["shape"] == "tree":
        return [rng.randint(max(1, case["nodes"] // 2), case["nodes"]) if case["batch"] > 1 else case["nodes"]
                for _ in range(case["batch"])]
    return [case["nodes"]] * case["batch"]


def _contexts(case):
    """Tokens before those rows: the case's own too."""
    rng = random.Random(case["ctx_hi"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    if case["shape"] == "tree" and case["batch"] > 2:
        ctx[1] = 0  # a sequence without a context
    return ctx


def work(case):
    if case["op"] in ("kv", "read"):
        n = 2 * case["tokens"] * case["heads"]
        cache, out = _row_bytes(case["fmt"], case["dim"]), case["dim"] * (2 if case["out"] == "bf16" else 4)
        if case["op"] == "read":
            return {"bytes": n * (cache + out), "flops": 2 * n * case["dim"]}
        return {"bytes": n * (2 * case["dim"] + 2 * cache + out), "flops": 5 * n * case["dim"]}
    if case["op"] == "attn":
        sizes, heads = _tree_sizes(case), case["kv_heads"] * case["group"]
        lens = [c + n for c, n in zip(_contexts(case), sizes)]
        cache = 2 * case["kv_heads"] * sum(lens) * _row_bytes(case["fmt"], case["dim"])
        return {"bytes": cache + 4 * sum(sizes) * heads * case["dim"],
                "flops": 4 * heads * case["dim"] * sum(n * t for n, t in zip(sizes, lens))}
    # the accepted path's rows of logits (about two; which ones depends on the outcome), the noise, one draft row
    size, path = 2 if case["type"] == "bf16" else 4, min(case["nodes"], 2)
    per = path * size + 4 + (4 if case["drafts"] == "probs" else 0)
    return {"bytes": case["batch"] * case["vocab"] * per, "flops": case["batch"] * case["vocab"] * (3 * path + 2)}


# ------------------------------------------------------------------ the cache's layout (plain)

def _half_up(x):
    """f32 >= 0 to f16, rounded up."""
    h = x.half()
    return torch.where(h.float() < x, (h.view(torch.int16) + 1).view(torch.float16), h)


def _half_down(x):
    """f32 to f16, rounded towards minus infinity."""
    h = x.half()
    b = h.view(torch.int16)
    low = torch.where(h > 0, b - 1, torch.where(h == 0, torch.full_like(b, -32767), b + 1))
    return torch.where(h.float() > x, low.view(torch.float16), h)


def _over(x, n):
    """x / n to f16, rounded up (a quotient of tensors: by a number torch would multiply by 1 / n)."""
    return _half_up(x / torch.full_like(x, n))


def _quantise(x, fmt):
    """rows [..., D] -> (codes uint8 [..., D], d f16 [..., D / 32], m f16 or None). Q8 codes are c + 128."""
    g = torch.nan_to_num(x.float(), nan=0.0, posinf=LIMIT, neginf=-LIMIT).clamp(-LIMIT, LIMIT)
    g = g.unflatten(-1, (-1, GROUP))
    if fmt == Q8:
        d = _over(g.abs().amax(-1), 127.0)
        f = d.float().unsqueeze(-1)
        c = torch.where(f > 0, torch.round(g / f), torch.zeros_like(g)).clamp(-127, 127) + 128
        return c.to(torch.uint8).flatten(-2), d, None
    m = _half_down(g.amin(-1))
    g = g - m.float().unsqueeze(-1)
    d = _over(g.amax(-1), 15.0)
    f = d.float().unsqueeze(-1)
    c = torch.where(f > 0, torch.round(g / f), torch.zeros_like(g)).clamp(0, 15)
    return c.to(torch.uint8).flatten(-2), d, m


def _pack4(c):
    """4-bit codes [..., D] -> bytes [..., D / 2]: a 32-bit word holds 8, code i at bit 4 (i / 2) + 16 (i % 2)."""
    e = c.unflatten(-1, (-1, 8))
    return torch.stack([e[..., 0] | e[..., 2] << 4, e[..., 4] | e[..., 6] << 4, e[..., 1] | e[..., 3] << 4,
                        e[..., 5] | e[..., 7] << 4], -1).flatten(-2)


def _unpack4(b):
    w = b.unflatten(-1, (-1, 4))
    lo, hi = w & 15, w >> 4
    return torch.stack([lo[..., 0], lo[..., 2], hi[..., 0], hi[..., 2], lo[..., 1], lo[..., 3], hi[..., 1],
                        hi[..., 3]], -1).flatten(-2)


def _block_bytes(fmt, dim):
    return 32 * _row_bytes(fmt, dim)


def _pack_blocks(k, v, fmt):
    """K and V rows [..., 16, D] of 16 tokens -> the block's bytes [..., block_bytes]."""
    parts = []
    for rows, value in ((k, False), (v, True)):
        c, d, m = _quantise(rows, fmt)
        c = _pack4(c) if fmt == Q4 else c
        if value:  # lane = (eighth of the row, pair of tokens), its bytes: token (2 x 2), piece
            c = c.unflatten(-1, (8, -1)).unflatten(-3, (2, 4, 2))        # th tid tl g x
            c = c.movedim((-2, -4, -5, -3), (-5, -4, -3, -2))            # g tid th tl x
        else:      # lane = (token of eight, quarter of the row), its bytes: eight, piece
            c = c.unflatten(-1, (4, -1)).unflatten(-3, (2, 8))           # nb g tid x
            c = c.movedim(-4, -2)                                        # g tid nb x
            c = c.unflatten(-2, (2, 1))
        c = c.flatten(-3).flatten(-3, -2).unflatten(-1, (-1, 16)).transpose(-3, -2).flatten(-3)
        s = [d] if m is None else [d, m]
        s = torch.stack(s, -1).flatten(-3) if not value else torch.stack(s, -3).transpose(-1, -2).flatten(-3)
        parts += [c, s.contiguous().view(torch.uint8)]
    return torch.cat(parts, -1)


def _codes_of(part, fmt, dim, value):
    """Bytes of a block's K or V codes [..., 16 RB] -> codes uint8 [..., 16, D]."""
    c = part.unflatten(-1, (-1, 32, 16)).transpose(-3, -2).flatten(-2)   # lane, its bytes
    if value:
        c = c.unflatten(-1, (2, 2, -1)).unflatten(-4, (8, 4))            # g tid th tl x
        c = c.movedim((-5, -4, -3, -2), (-2, -4, -5, -3)).flatten(-2).flatten(-4, -2)
    else:
        c = c.unflatten(-1, (2, -1)).unflatten(-3, (8, 4))               # g tid nb x
        c = c.movedim(-2, -4).flatten(-2).flatten(-3, -2)
    return _unpack4(c) if fmt == Q4 else c


def _unpack_blocks(b, fmt, dim):
    """Block bytes [..., block_bytes] -> K, V f32 [..., 16, D]."""
    rb, gr, out, at = (dim if fmt == Q8 else dim // 2), dim // GROUP, [], 0
    for value in (False, True):
        c = _codes_of(b[..., at:at + 16 * rb], fmt, dim, value).unflatten(-1, (gr, GROUP)).float()
        at += 16 * rb
        size = 32 * gr * (1 if fmt == Q8 else 2)
        s = b[..., at:at + size].contiguous().view(torch.float16).float()
        at += size
        if fmt == Q8:
            s = s.unflatten(-1, (gr, 16)).transpose(-1, -2) if value else s.unflatten(-1, (16, gr))
            r = (c - 128.0) * s.unsqueeze(-1)
        else:
            s = s.unflatten(-1, (2, gr, 16)).movedim((-3, -1), (-1, -3)) if value else s.unflatten(-1, (16, gr, 2))
            r = c * s[..., :1] + s[..., 1:]
        out.append(r.flatten(-2))
    return out


def _byte_places(case, slots, value):
    """Byte addresses in the pool of the rows of `slots` [T] -> codes [T, H, RB], scales [T, H, groups, 1 or 2] (of
    f16 words)."""
    heads, dim, page, fmt = case["heads"], case["dim"], case["page"], case["fmt"]
    rb, gr, dev = (dim if fmt == Q8 else dim // 2), dim // GROUP, slots.device
    bb, per = _block_bytes(fmt, dim), 1 if fmt == Q8 else 2
    slots = slots.long()
    head = torch.arange(heads, device=dev)
    base = ((slots // page)[:, None] * heads + head) * (page // 16) + (slots % page // 16)[:, None]
    base = base * bb + (16 * rb + 32 * gr * per if value else 0)
    t = (slots % 16)[:, None]
    i = torch.arange(rb, device=dev)
    if value:
        piece = rb // 8
        lane, x = i // piece * 4 + t % 8 // 2, (t // 8 * 2 + t % 2) * piece + i % piece
    else:
        piece = rb // 4
        lane, x = t % 8 * 4 + i // piece, t // 8 * piece + i % piece
    codes = base[..., None] + (x // 16 * 512 + lane * 16 + x % 16)[:, None, :]
    g, p = torch.arange(gr, device=dev)[:, None], torch.arange(per, device=dev)
    word = (p * gr + g) * 16 + t[..., None] if value else (t[..., None] * gr + g) * per + p
    return codes, (base + 16 * rb)[..., None, None] // 2 + word[:, None]


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _kv_rows(shape, g):
    """K and V rows as a model makes them: a few large K channels with an offset, V of unit size."""
    dim = shape[-1]
    k = torch.randn(shape, device="cuda", generator=g)
    big = torch.arange(dim, device="cuda") % 37 == 5
    k = torch.where(big, k * 2.0 + 5.0, k)
    return k.bfloat16(), torch.randn(shape, device="cuda", generator=g).bfloat16()


def _slots(tokens, page, pages, rng):
    """Consecutive tokens over pages in any order, the first page begun in its middle; some rows skipped (-1)."""
    first = rng.randint(0, page - 1)
    order = list(range(pages))
    rng.shuffle(order)
    t = torch.arange(tokens) + min(first, pages * page - tokens)
    s = torch.tensor(order)[t // page] * page + t % page
    if tokens > 4:
        s[rng.randint(0, tokens - 1)] = -1
    return s.int().cuda()


def _tree(n, shape, rng):
    """Parents (-1 for row 0) and ancestor masks of n rows."""
    parent = [-1]
    for j in range(1, n):
        parent.append(j - 1 if shape != "tree" else rng.randint(max(0, (j - 1) // 3 - 1), max(0, (j - 1) // 2)))
    mask = []
    for j in range(n):
        mask.append((mask[parent[j]] if j else 0) | 1 << j)
    return parent, [m - (1 << 64) if m >> 63 else m for m in mask]


def prepare(case, seed):
    rng, g = random.Random(seed), _gen(seed)
    st = {"case": case}
    if case["op"] in ("kv", "read"):
        tokens, heads, dim = case["tokens"], case["heads"], case["dim"]
        bb = _block_bytes(case["fmt"], dim)
        blocks = case["pages"] * heads * case["page"] // 16
        if case["op"] == "read":
            st["pages"] = _pack_blocks(*_kv_rows((blocks, 16, dim), g), case["fmt"]).flatten()
        else:
            st["pages"] = torch.zeros(blocks * bb, dtype=torch.uint8, device="cuda")
            k, v = _kv_rows((tokens, heads, dim), g)
            if case["layout"] == "qkv":  # views of one fused product's output
                qkv = torch.cat([torch.zeros_like(k), k, v], 1).contiguous()
                st["k"], st["v"] = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]
            elif case["layout"] == "heads":
                st["k"], st["v"] = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (k, v))
            else:
                st["k"], st["v"] = k, v
        st["slots"] = _slots(tokens, case["page"], case["pages"], rng)
        kind = torch.bfloat16 if case["out"] == "bf16" else torch.float32
        st["ko"], st["vo"] = (torch.empty((tokens, heads, dim), dtype=kind, device="cuda") for _ in range(2))
        return st
    if case["op"] == "attn":
        sizes, ctx = _tree_sizes(case), _contexts(case)
        lens = [c + n for c, n in zip(ctx, sizes)]
        page, heads, dim = case["page"], case["kv_heads"], case["dim"]
        counts = [-(-n // page) for n in lens]
        order = list(range(sum(counts)))
        rng.shuffle(order)
        table = torch.zeros((case["batch"], max(counts)), dtype=torch.int32)
        at, masks = 0, []
        for b, n in enumerate(counts):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
            masks += _tree(sizes[b], case["shape"], rng)[1]
        if case["shape"] == "tree" and case["batch"] > 2:
            masks[sizes[0]] = 0  # a row that sees nothing
        parts, left = [], at * heads * page // 16
        while left > 0:  # in parts: the rows before quantisation are several times the cache's size
            n = min(left, 1 << 18)
            parts.append(_pack_blocks(*_kv_rows((n, 16, dim), g), case["fmt"]))
            left -= n
        st["pages"], parts = torch.cat(parts).flatten(), None
        st["table"] = table.cuda()
        st["kv_len"] = torch.tensor(lens, dtype=torch.int32).cuda()
        st["q_start"] = torch.tensor([0] + sizes).cumsum(0).int().cuda()
        st["mask"] = torch.tensor(masks, dtype=torch.int64).cuda() if case["shape"] == "tree" else None
        st["scale"] = 1.0 / math.sqrt(dim)
        heads_q = heads * case["group"]
        q = torch.randn((sum(sizes), heads_q, dim), device="cuda", generator=g) * 1.5
        st["q"] = q.bfloat16()
        st["out"] = torch.empty_like(st["q"])
        st["n_max"] = max(sizes)
        return st
    batch, vocab = case["batch"], case["vocab"]
    sizes = _tree_sizes(case)
    starts = [0]
    for n in sizes:
        starts.append(starts[-1] + n)
    total = starts[-1]
    logits = torch.randn((total, vocab), device="cuda", generator=g) * 2.0
    hot = torch.randint(0, vocab, (total, 6), device="cuda", generator=g)
    logits.scatter_add_(1, hot, torch.rand((total, 6), device="cuda", generator=g) * 9.0)  # the likely tokens
    temp = torch.tensor([0.0 if case["greedy"] and b % 4 == 1 else 0.6 + 0.1 * (b % 5) for b in range(batch)]).cuda()
    parent = [p for n in sizes for p in _tree(n, case["shape"], rng)[0]]
    seq = torch.tensor([b for b, n in enumerate(sizes) for _ in range(n)]).cuda()
    st["parent"] = torch.tensor(parent, dtype=torch.int32).cuda() if case["shape"] == "tree" else None
    up = torch.tensor([starts[b] + max(0, parent[starts[b] + j]) for b, n in enumerate(sizes) for j in range(n)]).cuda()
    # the draft's distribution of a row: its parent's with an error, at the sequence's temperature
    near = torch.randn((total, vocab), device="cuda", generator=g).mul_(case["agree"]).add_(logits[up])
    near.div_(temp[seq].clamp(min=0.5)[:, None])
    draft = torch.softmax(near, -1)
    del near
    race = torch.empty_like(draft).exponential_(generator=g).clamp_(min=1e-30)
    st["tokens"] = (draft / race).argmax(-1).int()
    del race
    st["draft"] = draft if case["drafts"] == "probs" else None
    st["logits"] = logits.bfloat16() if case["type"] == "bf16" else logits
    st["q_start"], st["temp"] = torch.tensor(starts, dtype=torch.int32).cuda(), temp
    st["u"] = torch.rand(total, device="cuda", generator=g)
    st["noise"] = torch.empty((batch, vocab), device="cuda").exponential_(generator=g)
    st["n_acc"], st["next"] = (torch.empty(batch, dtype=torch.int32, device="cuda") for _ in range(2))
    st["path"] = torch.empty(total, dtype=torch.int32, device="cuda")
    st["n_max"] = max(sizes)
    return st


# ------------------------------------------------------------------ plain forms

def _plain_read(case, st):
    slots, kind = st["slots"], st["ko"].dtype
    out = []
    for value in (False, True):
        codes, scales = _byte_places(case, slots.clamp(min=0), value)
        c = st["pages"][codes]
        c = (_unpack4(c) if case["fmt"] == Q4 else c).float().unflatten(-1, (-1, GROUP))
        s = st["pages"].view(torch.float16)[scales].float()
        r = (c - 128.0) * s if case["fmt"] == Q8 else c * s[..., :1] + s[..., 1:]
        out.append(torch.where((slots >= 0)[:, None, None], r.flatten(-2), torch.zeros((), device="cuda")).to(kind))
    return out


def _plain_append(case, st):
    keep = st["slots"] >= 0
    slots = st["slots"][keep]
    for rows, value in ((st["k"], False), (st["v"], True)):
        c, d, m = _quantise(rows[keep], case["fmt"])
        codes, scales = _byte_places(case, slots, value)
        st["pages"][codes] = _pack4(c) if case["fmt"] == Q4 else c
        st["pages"].view(torch.float16)[scales] = torch.stack([d] if m is None else [d, m], -1)


def _plain_attn(case, st):
    heads, group, dim, page = case["kv_heads"], case["group"], case["dim"], case["page"]
    q_start, kv_len, n = st["q_start"].long(), st["kv_len"].long(), st["n_max"]
    blocks = st["pages"].view(-1, heads, page // 16, _block_bytes(case["fmt"], dim))[st["table"].long()]
    k, v = (x.movedim(2, 1).flatten(2, 4) for x in _unpack_blocks(blocks, case["fmt"], dim))  # [B, H, tokens, D]
    size = q_start[1:] - q_start[:-1]
    i = torch.arange(n, device="cuda")
    rows = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"].float()[rows].unflatten(2, (heads, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, H, n G, D]
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    j = torch.arange(k.shape[2], device="cuda") - (kv_len - size)[:, None]  # place after the context
    j = j[:, None, :]
    if st["mask"] is None:
        sees = j <= i[:, None]
    else:
        sees = (j < 0) | ((st["mask"][rows][..., None] >> j.clamp(0, 63)) & 1 > 0) & (j < 64)
    sees = (sees & (j < size[:, None, None])).repeat_interleave(group, 1)[:, None]
    s = s.masked_fill(~sees, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    o = torch.matmul(e, v) / e.sum(-1, keepdim=True).clamp(min=1e-38)
    o = o.unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return o[i < size[:, None]].bfloat16()


def _plain_verify(case, st):
    n, vocab = st["n_max"], case["vocab"]
    q_start = st["q_start"].long()
    size = q_start[1:] - q_start[:-1]
    i = torch.arange(n, device="cuda")
    rows = (q_start[:-1, None] + i).clamp(max=q_start[-1] - 1)
    l = st["logits"][rows].float()
    temp = st["temp"][:, None, None]
    top, at = l.max(-1, keepdim=True)
    e = torch.exp((l - top) / torch.where(temp > 0, temp, torch.ones_like(temp)))
    one = torch.arange(vocab, device="cuda") == at
    p = torch.where(temp > 0, e / e.sum(-1, keepdim=True), one.float())
    parent = st["parent"][rows].long() if st["parent"] is not None else (i - 1).expand(rows.shape)
    token, u = st["tokens"][rows].long(), st["u"][rows]
    b = torch.arange(rows.shape[0], device="cuda")
    cur, r, z = torch.zeros_like(b), p[:, 0], torch.ones(b.shape, device="cuda")
    path = torch.full(rows.shape, -1, dtype=torch.int32, device="cuda")
    count = torch.zeros_like(b)
    for j in range(1, n):  # children come after their parent, siblings in order
        x = token[:, j, None]
        q = st["draft"][rows[:, j]] if st["draft"] is not None else None
        qx = q.gather(1, x)[:, 0] if q is not None else torch.ones_like(z)
        asked = (j < size) & (parent[:, j] == cur)
        yes = asked & (u[:, j] * z * qx < r.gather(1, x)[:, 0])
        no = asked & ~yes
        less = (r - z[:, None] * q).clamp(min=0) if q is not None else r.scatter(1, x, 0.0)
        r = torch.where(yes[:, None], p[:, j], torch.where(no[:, None], less, r))
        z = torch.where(yes, torch.ones_like(z), torch.where(no, less.sum(-1), z))
        cur = torch.where(yes, torch.full_like(cur, j), cur)
        path[b, torch.where(yes, count, torch.full_like(count, n - 1))] = torch.where(
            yes, torch.full_like(cur, j).int(), path[:, n - 1])
        count = count + yes.long()
    r = torch.where((z > 0)[:, None], r, p[b, cur])
    nxt = (r / st["noise"]).argmax(-1)
    return count.int(), path[i < size[:, None]], nxt.int()


# ------------------------------------------------------------------ one pass

def _cache(moe, case, st):
    heads = case["heads"] if "heads" in case else case["kv_heads"]
    return moe.KvCache(st["pages"], head_dim=case["dim"], n_kv_heads=heads, page_size=case["page"],
                       format=moe.MOE_KV_Q8 if case["fmt"] == Q8 else moe.MOE_KV_Q4)


def run(state):
    st, case = state, state["case"]
    if not own:
        if case["op"] == "kv":
            _plain_append(case, st)
        if case["op"] in ("kv", "read"):
            return _plain_read(case, st)
        return _plain_attn(case, st) if case["op"] == "attn" else _plain_verify(case, st)
    import moe_decode_quantized_gb300 as moe
    if "kept" not in st:  # what a program keeps for its life: the cache's description, a workspace
        if case["op"] == "verify":
            st["kept"] = torch.empty(moe.spec_verify_workspace_bytes(case["batch"], st["tokens"].numel()),
                                     dtype=torch.uint8, device="cuda")
            moe.workspace_init(st["kept"])
        else:
            st["kept"] = _cache(moe, case, st)
        if case["op"] == "attn":
            st["ws"] = torch.empty(moe.tree_attention_workspace_bytes(
                st["kept"], case["kv_heads"] * case["group"], case["batch"], st["q"].shape[0]), dtype=torch.uint8,
                device="cuda")
            moe.workspace_init(st["ws"])
    if case["op"] == "verify":
        moe.spec_verify(st["logits"], st["q_start"], st["tokens"], st["parent"], st["draft"], st["temp"], st["u"],
                        st["noise"], st["n_acc"], st["path"], st["next"], st["kept"])
        return st["n_acc"], st["path"], st["next"]
    if case["op"] == "attn":
        moe.tree_attention(st["kept"], st["q"], st["out"], st["q_start"], st["kv_len"], st["table"], st["mask"],
                           st["scale"], st["ws"])
        return st["out"]
    if case["op"] == "kv":
        moe.kv_append(st["kept"], st["k"], st["v"], st["slots"])
    moe.kv_read(st["kept"], st["slots"], st["ko"], st["vo"])
    return [st["ko"], st["vo"]]


# ------------------------------------------------------------------ the definition in 64 bits

def _f16_towards(x, up):
    """float64 array to the f16 neighbour above (or below), as float64."""
    h = x.astype(np.float16)
    step = np.nextafter(h, np.float16(np.inf if up else -np.inf))
    off = h.astype(np.float64) < x if up else h.astype(np.float64) > x
    return np.where(off, step, h).astype(np.float64)


def _exact_values(x, fmt):
    """What the cache holds of float64 rows [..., D]."""
    g = np.clip(np.nan_to_num(x, nan=0.0, posinf=LIMIT, neginf=-LIMIT), -LIMIT, LIMIT)
    g = g.reshape(g.shape[:-1] + (-1, GROUP))
    if fmt == Q8:
        d = _f16_towards(np.abs(g).max(-1, keepdims=True) / 127.0, True)
        c = np.clip(np.rint(g / np.where(d > 0, d, 1.0)), -127, 127)
        return (c * d).reshape(x.shape)
    m = _f16_towards(g.min(-1, keepdims=True), False)
    d = _f16_towards((g - m).max(-1, keepdims=True) / 15.0, True)
    c = np.clip(np.rint((g - m) / np.where(d > 0, d, 1.0)), 0, 15)
    return (np.where(d > 0, c, 0.0) * d + m).reshape(x.shape)


def _exact_rows(pages, case, heads, page, token, value):
    """Values of a cache's rows: int64 arrays page, token (place in the page) [N] -> float64 [N, heads, D]. By bytes."""
    dim, fmt = case["dim"], case["fmt"]
    q8, groups = fmt == Q8, dim // 32
    n16, s16 = (16 * dim if q8 else 8 * dim), groups * (32 if q8 else 64)
    block = (page[:, None] * heads + torch.arange(heads, device="cuda")) * (case["page"] // 16) + (token // 16)[:, None]
    first = (block * 2 + (1 if value else 0)) * (n16 + s16)
    t, d = (token % 16)[:, None], torch.arange(dim, device="cuda")
    if value:
        lane, k = (d // (dim // 8)) * 4 + (t % 8) // 2, ((t // 8) * 2 + t % 2) * (dim // 8) + d % (dim // 8)
    else:
        lane, k = (t % 8) * 4 + d // (dim // 4), (t // 8) * (dim // 4) + d % (dim // 4)
    if q8:
        at, shift = k, torch.zeros_like(k)
    else:  # the k-th code of the lane: word k / 8, bit 4 (i / 2) + 16 (i % 2)
        bit = (k % 8) // 2 * 4 + (k % 2) * 16
        at, shift = k // 8 * 4 + bit // 8, bit % 8
    at = at // 16 * 512 + lane * 16 + at % 16
    code = pages[first[:, :, None] + at[:, None, :]].long()
    code = code - 128 if q8 else code >> shift[:, None, :] & 15
    g = d // 32
    if value:
        place = [(z * groups + g) * 16 + t for z in range(1 if q8 else 2)]
    else:
        place = [(t * groups + g) * (1 if q8 else 2) + z for z in range(1 if q8 else 2)]
    words = pages.view(torch.float16)
    s = [words[(first[:, :, None] + n16) // 2 + p[:, None, :]].double() for p in place]
    return code.double() * s[0] + (0 if q8 else s[1])


def _exact_verify(case, st):
    counts, nexts, paths = [], [], []
    starts = st["q_start"].tolist()
    for b in range(case["batch"]):
        lo, n, t = starts[b], starts[b + 1] - starts[b], float(st["temp"][b])

        def row(j):
            l = st["logits"][lo + j].double()
            if t > 0:
                return torch.softmax(l / t, 0)
            return (torch.arange(l.numel(), device="cuda") == int((l == l.max()).nonzero()[0])).double()

        cur, r, z, path = 0, row(0), 1.0, []
        for j in range(1, n):
            if (int(st["parent"][lo + j]) if st["parent"] is not None else j - 1) != cur:
                continue
            x = int(st["tokens"][lo + j])
            q = torch.zeros_like(r)
            q[x] = 1.0
            q = st["draft"][lo + j].double() if st["draft"] is not None else q
            if float(st["u"][lo + j]) * z * float(q[x]) < float(r[x]):
                cur, r, z = j, row(j), 1.0
                path.append(j)
            else:
                r = (r - z * q).clamp(min=0)
                z = float(r.sum())
        s = (r if z > 0 else row(cur)) / st["noise"][b].double()
        nexts.append(int((s == s.max()).nonzero()[0]))
        counts.append(len(path))
        paths += path + [-1] * (n - len(path))
    return tuple(torch.tensor(x, dtype=torch.int32) for x in (counts, paths, nexts))


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(case, st)
    if case["op"] == "kv":
        skip = (st["slots"] < 0).cpu().numpy()[:, None, None]
        return [torch.from_numpy(np.where(skip, 0.0, _exact_values(x.double().cpu().numpy(), case["fmt"])))
                for x in (st["k"], st["v"])]
    if case["op"] == "read":
        out = []
        for value in (False, True):
            part = []
            for s in st["slots"].long().split(4096):
                r = _exact_rows(st["pages"], case, case["heads"], s.clamp(min=0) // case["page"],
                                s.clamp(min=0) % case["page"], value)
                part.append(torch.where(s[:, None, None] < 0, torch.zeros_like(r), r))
            out.append(torch.cat(part))
        return out
    starts, out = st["q_start"].tolist(), []
    heads, group = case["kv_heads"], case["group"]
    for b in range(case["batch"]):
        n, length = starts[b + 1] - starts[b], int(st["kv_len"][b])
        q = st["q"][starts[b]:starts[b + 1]].double()
        place = torch.arange(length, device="cuda")
        page = st["table"][b].long()[place // case["page"]]
        k, v = [], []
        for p, t in zip(page.split(8192), (place % case["page"]).split(8192)):
            k.append(_exact_rows(st["pages"], case, heads, p, t, False))
            v.append(_exact_rows(st["pages"], case, heads, p, t, True))
        k, v = torch.cat(k), torch.cat(v)
        sees = torch.zeros((n, length), dtype=torch.bool)
        sees[:, :length - n] = True
        for i in range(n):
            m = (2 << i) - 1 if st["mask"] is None else int(st["mask"][starts[b] + i]) % (1 << 64)
            sees[i, length - n:] = torch.tensor([bool(m >> j & 1) for j in range(n)])
        s = torch.einsum("nhgd,thd->hgnt", q.unflatten(1, (heads, group)), k) * st["scale"]
        s = torch.where(sees.cuda(), s, torch.full_like(s, -math.inf))
        w = torch.softmax(s, -1).nan_to_num(nan=0.0)
        out.append(torch.einsum("hgnt,thd->nhgd", w, v).flatten(1, 2))
    return torch.cat(out)

"""The cases at which rotary positions, latent attention and the care of pages are measured.

Five operators: rotary positions (rope), the paged cache of latent vectors written
and read back (latent), attention over it in absorbed form (absorbed) and, for
prompts, in expanded form (expanded), and the bookkeeping of pages: freeing,
forking, growing, compacting and copying them (pages). `run` computes them in
plain torch operations in 32 bits, or, where `own` is set, by the calls of this
package.

A table of rotary frequencies holds one 64-bit whole number a pair of
dimensions: the part of a turn that one position adds, times 2^64.
"""
import math
import random

import torch

own = False

HALF, INTER = "half", "interleaved"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 8 tokens: queries and keys of a fused projection's output, whole heads
        {"name": "rope_decode_8", "op": "rope", "tokens": 8, "heads": 40, "dim": 128, "rope": 128, "offset": 0,
         "layout": HALF, "type": "bf16", "transposed": False, "scaling": "plain", "far": 32768, "source": "fused"},
        # a prompt's queries of latent attention: the last 64 of 192 dimensions turn, frequencies scaled for 131072
        {"name": "rope_prompt_16384", "op": "rope", "tokens": 16384, "heads": 32, "dim": 192, "rope": 64, "offset": 128,
         "layout": INTER, "type": "bf16", "transposed": False, "scaling": "parts", "far": 131072, "source": "plain"},
        # the gradient's way back in 32 bits, odd sizes, strided rows
        {"name": "rope_back_4099_f32", "op": "rope", "tokens": 4099, "heads": 12, "dim": 96, "rope": 90, "offset": 6,
         "layout": HALF, "type": "f32", "transposed": True, "scaling": "linear", "far": 4099, "source": "fused"},
        # one decode step's latent vectors into the cache and back
        {"name": "latent_decode_8", "op": "latent", "tokens": 8, "latent": 512, "rope": 64, "page": 64, "pages": 64,
         "layout": INTER, "far": 32768, "turn": True},
        # a long prompt's
        {"name": "latent_prompt_65536", "op": "latent", "tokens": 65536, "latent": 512, "rope": 64, "page": 64,
         "pages": 1100, "layout": INTER, "far": 65536, "turn": True},
        # one token of one sequence, short context: latency
        {"name": "absorbed_one_b1_511", "op": "absorbed", "latent": 512, "rope": 64, "heads": 16, "batch": 1, "nodes": 1,
         "ctx_lo": 511, "ctx_hi": 511, "page": 64, "shape": "one"},
        # a serving batch of ragged long contexts, one token each, many heads
        {"name": "absorbed_one_b64_24k", "op": "absorbed", "latent": 512, "rope": 64, "heads": 128, "batch": 64, "nodes": 1,
         "ctx_lo": 4000, "ctx_hi": 24000, "page": 64, "shape": "one"},
        # trees of up to 8 drafted tokens (the small batch's size), small pages
        {"name": "absorbed_tree_b16_16k", "op": "absorbed", "latent": 512, "rope": 64, "heads": 32, "batch": 16, "nodes": 8,
         "ctx_lo": 1000, "ctx_hi": 16000, "page": 16, "shape": "tree"},
        # short prompts with parts of them in the cache already, ragged
        {"name": "expanded_b6_ragged", "op": "expanded", "nope": 128, "rope": 64, "heads": 16, "batch": 6, "q_lo": 1,
         "q_hi": 700, "ctx_lo": 0, "ctx_hi": 900, "causal": True},
        # one long prompt
        {"name": "expanded_b1_8192", "op": "expanded", "nope": 128, "rope": 64, "heads": 32, "batch": 1, "q_lo": 8192,
         "q_hi": 8192, "ctx_lo": 0, "ctx_hi": 0, "causal": True},
        # samples started anew from common prompts each step: their pages freed, forked, grown, part-filled ones copied
        {"name": "pages_fork_24", "op": "fork", "parents": 8, "children": 24, "len_lo": 1000, "len_hi": 4000, "grow": 70,
         "page": 64, "pages": 2048, "layers": 4, "page_bytes": 64 * 1152},
        # a half-empty pool of long contexts moved to its front
        {"name": "pages_compact_4096", "op": "compact", "rows": 48, "len_lo": 500, "len_hi": 5000, "page": 64,
         "pages": 4096, "layers": 2, "page_bytes": 64 * 1152},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "rope", "latent", "absorbed", "absorbed", "absorbed", "expanded", "expanded", "fork",
                         "compact"])
        c = {"op": op}
        if op == "rope":
            dim = rng.choice([64, 96, 128, 192, 256])
            part = rng.choice([dim, dim, 64, 32, 2 * rng.randint(1, dim // 2)])
            c.update(tokens=_log(rng, 1, 16384), heads=_log(rng, 1, 64), dim=dim, rope=part,
                     offset=rng.choice([0, dim - part]), layout=rng.choice([HALF, INTER]),
                     type=rng.choice(["bf16", "f32"]), transposed=rng.random() < 0.4,
                     scaling=rng.choice(["plain", "linear", "base", "parts"]), far=_log(rng, 1, 1 << 30),
                     source=rng.choice(["fused", "plain", "heads"]))
        elif op == "latent":
            n, page = _log(rng, 1, 65536), rng.choice([16, 32, 64, 128])
            c.update(tokens=n, latent=rng.choice([128, 256, 512, 512]), rope=rng.choice([16, 32, 64, 64]), page=page,
                     pages=n // page + 2 + rng.randint(0, 64), layout=rng.choice([HALF, INTER]), far=_log(rng, 1, 1 << 20),
                     turn=rng.random() < 0.8)
        elif op == "absorbed":
            shape = rng.choice(["one", "one", "chain", "tree"])
            hi = _log(rng, 1, 100003)
            c.update(latent=rng.choice([128, 256, 512, 512]), rope=rng.choice([16, 32, 64, 64]), heads=_log(rng, 1, 128),
                     batch=_log(rng, 1, 64), nodes=1 if shape == "one" else _log(rng, 2, 64), ctx_lo=rng.randint(0, hi),
                     ctx_hi=hi, page=rng.choice([16, 32, 48, 64, 128]), shape=shape)
        elif op == "expanded":
            q, ctx = _log(rng, 1, 8192), rng.choice([0, _log(rng, 1, 4096)])
            c.update(nope=rng.choice([64, 128, 128]), rope=rng.choice([16, 32, 64, 64]), heads=_log(rng, 1, 64),
                     batch=_log(rng, 1, 8), q_lo=rng.randint(1, q), q_hi=q, ctx_lo=0, ctx_hi=ctx,
                     causal=rng.random() < 0.8)
        elif op == "fork":
            page, hi = rng.choice([16, 32, 64, 128]), _log(rng, 1, 4000)
            c.update(parents=rng.randint(1, 16), children=rng.randint(1, 48), len_lo=rng.randint(1, hi), len_hi=hi,
                     grow=rng.randint(0, 200), page=page, layers=rng.randint(1, 4), page_bytes=page * rng.choice([160, 640, 1152]))
            c["pages"] = (c["parents"] + c["children"]) * ((hi + c["grow"]) // page + 1) + rng.randint(1, 300)
        else:
            page, hi = rng.choice([16, 32, 64, 128]), _log(rng, 1, 8000)
            c.update(rows=_log(rng, 2, 200), len_lo=rng.randint(0, hi), len_hi=hi, page=page, layers=rng.randint(1, 4),
                     page_bytes=page * rng.choice([160, 640, 1152]))
            c["pages"] = int(c["rows"] * (hi // page + 1) * rng.uniform(1.2, 2.5)) + 2
        w, tops = work(c), [work(d) for d in listed() if d["op"] == op]
        room = max(_elements(d) for d in listed() if d["op"] == op)
        if (w["bytes"] <= max(t["bytes"] for t in tops) and w["flops"] <= max(t["flops"] for t in tops)
                and _elements(c) <= room):
            return c


def _elements(c):
    """Values that a case's inputs, and the plain form's scores, stand for (bounds the plain form's memory)."""
    if c["op"] == "rope":
        return c["tokens"] * c["heads"] * c["dim"]
    if c["op"] == "latent":
        return c["tokens"] * (c["latent"] + c["rope"])
    if c["op"] == "absorbed":
        top = c["ctx_hi"] + c["nodes"]
        return c["batch"] * top * (c["latent"] + c["rope"] + c["nodes"] * c["heads"])
    if c["op"] == "expanded":
        return c["batch"] * c["heads"] * (c["q_hi"] + c["ctx_hi"]) * (c["q_hi"] + 2 * c["nope"] + c["rope"])
    return c["pages"] * c["layers"] * c["page_bytes"]


def _rows_of(case):
    """Rows (last token and drafts) of each sequence: the case's own, whatever the seed."""
    rng = random.Random(case["nodes"])
    if case["shape"] == "tree" and case["batch"] > 1:
        return [rng.randint(max(1, case["nodes"] // 2), case["nodes"]) for _ in range(case["batch"])]
    return [case["nodes"]] * case["batch"]


def _contexts(case):
    """Tokens before them: the case's own too."""
    rng = random.Random(case["ctx_hi"])
    ctx = [rng.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    if case["shape"] == "tree" and case["batch"] > 2:
        ctx[1] = 0  # a sequence without a context
    return ctx


def _prompts(case):
    """(query rows, tokens) of each sequence of an expanded case."""
    rng = random.Random(case["q_hi"] * 7 + case["ctx_hi"])
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    q[0] = case["q_hi"]
    if case["batch"] > 3:
        q[2] = 0  # a sequence without a row in this step
    return q, [n + rng.randint(case["ctx_lo"], case["ctx_hi"]) for n in q]


def _lengths(case, rows, tag):
    """Tokens of each row of a table: the case's own."""
    rng = random.Random(case["len_hi"] + tag)
    return [rng.randint(case["len_lo"], case["len_hi"]) for _ in range(rows)]


def work(case):
    op = case["op"]
    if op == "rope":
        size = 2 if case["type"] == "bf16" else 4
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["dim"] * size + 4 * case["tokens"] + 4 * case["rope"], "flops": 3 * n * case["rope"]}
    if op == "latent":  # rows into the pages, and out of them
        row = 2 * (case["latent"] + case["rope"])
        return {"bytes": case["tokens"] * (4 * row + 12), "flops": 3 * case["tokens"] * case["rope"]}
    if op == "absorbed":
        sizes = _rows_of(case)
        lens = [c + n for c, n in zip(_contexts(case), sizes)]
        wide, heads = case["latent"] + case["rope"], case["heads"]
        return {"bytes": 2 * sum(lens) * wide + 2 * sum(sizes) * heads * (wide + case["latent"]),
                "flops": 2 * heads * (wide + case["latent"]) * sum(n * t for n, t in zip(sizes, lens))}
    if op == "expanded":
        q, lens = _prompts(case)
        heads, wide = case["heads"], case["nope"] + case["rope"]
        pairs = sum(n * t - (n * (n - 1) // 2 if case["causal"] else 0) for n, t in zip(q, lens))
        return {"bytes": 2 * sum(q) * heads * (wide + case["nope"]) + 2 * sum(lens) * (2 * heads * case["nope"] + case["rope"]),
                "flops": 2 * heads * (wide + case["nope"]) * pairs}
    if op == "fork":
        lens, kids = _lengths(case, case["parents"], 0), [i % case["parents"] for i in range(case["children"])]
        copied = sum(1 for i in kids if lens[i] % case["page"])
        held = sum(-(-(lens[i] + case["grow"]) // case["page"]) for i in kids)
        return {"bytes": 2 * copied * case["layers"] * case["page_bytes"] + 12 * held, "flops": held}
    counts = [-(-n // case["page"]) for n in _lengths(case, case["rows"], 0)]
    live = sum(counts)
    moved = int(live * max(0.0, 1 - live / case["pages"]))  # about: pages in any places
    return {"bytes": 2 * moved * case["layers"] * case["page_bytes"] + 8 * case["pages"] + 8 * live, "flops": case["pages"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _frequencies(dim, scaling):
    """Radians a position of each pair, and the magnitude that scaling gives."""
    f = [10000.0 ** (-2 * i / dim) for i in range(dim // 2)]
    if scaling == "linear":
        return [x / 8 for x in f], 1.0
    if scaling == "base":
        return [(10000.0 * 8.0 ** (dim / max(dim - 2, 1))) ** (-2 * i / dim) for i in range(dim // 2)], 1.0
    if scaling == "parts":  # few turns in the first 4096 positions: stretched 32 times; many: as they are
        keep = [min(max((4096 * x / (2 * math.pi) - 1) / 31, 0.0), 1.0) for x in f]
        return [x * k + x / 32 * (1 - k) for x, k in zip(f, keep)], 0.1 * math.log(32.0) + 1
    return f, 1.0


def _table(dim, scaling):
    f, magnitude = _frequencies(dim, scaling)
    turns = [int(round(x / (2 * math.pi) * 2.0 ** 64)) for x in f]
    return torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64).cuda(), magnitude


def _positions(tokens, far, rng):
    """Consecutive ones of a prompt, or single tokens of many sequences."""
    if tokens > 64:
        first = rng.randint(0, max(0, far - tokens))
        return torch.arange(first, first + tokens, dtype=torch.int32).cuda()
    return torch.tensor([rng.randint(0, far) for _ in range(tokens)], dtype=torch.int32).cuda()


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
    """Ancestor masks of n rows."""
    mask = []
    for j in range(n):
        up = j - 1 if shape != "tree" else rng.randint(max(0, (j - 1) // 3 - 1), max(0, (j - 1) // 2)) if j else 0
        mask.append((mask[up] if j else 0) | 1 << j)
    return [m - (1 << 64) if m >> 63 else m for m in mask]


def _randn(shape, g, scale=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * scale).bfloat16()


def prepare(case, seed):
    rng, g, op = random.Random(seed), _gen(seed), case["op"]
    st = {"case": case}
    if op == "rope":
        shape, kind = (case["tokens"], case["heads"], case["dim"]), torch.bfloat16 if case["type"] == "bf16" else torch.float32
        if case["source"] == "heads":
            x = torch.randn((shape[1], shape[0], shape[2]), device="cuda", generator=g).to(kind).transpose(0, 1)
        elif case["source"] == "fused":  # heads of a wider projection's output
            x = torch.randn((shape[0], shape[1] + 3, shape[2]), device="cuda", generator=g).to(kind)[:, :shape[1]]
        else:
            x = torch.randn(shape, device="cuda", generator=g).to(kind)
        st["x"], st["out"] = x, torch.empty(shape, dtype=kind, device="cuda")
        st["pos"] = _positions(case["tokens"], case["far"], rng)
        st["table"], st["magnitude"] = _table(case["rope"], case["scaling"])
        return st
    if op == "latent":
        n, latent, rope = case["tokens"], case["latent"], case["rope"]
        x = _randn((n, latent + rope), g)  # one projection's output: the latent vector and the key's turning part
        st["c"], st["kr"] = x[:, :latent], x[:, latent:]
        st["pages"] = torch.zeros((case["pages"], case["page"], latent + rope), dtype=torch.bfloat16, device="cuda")
        st["slots"] = _slots(n, case["page"], case["pages"], rng)
        st["pos"] = _positions(n, case["far"], rng)
        st["table"], st["magnitude"] = _table(rope, "plain")
        st["c_out"] = torch.empty((n, latent), dtype=torch.bfloat16, device="cuda")
        st["kr_out"] = torch.empty((n, rope), dtype=torch.bfloat16, device="cuda")
        return st
    if op == "absorbed":
        sizes, page, wide, heads = _rows_of(case), case["page"], case["latent"] + case["rope"], case["heads"]
        lens = [c + n for c, n in zip(_contexts(case), sizes)]
        counts = [-(-n // page) for n in lens]
        order = list(range(sum(counts)))
        rng.shuffle(order)
        table = torch.zeros((case["batch"], max(counts)), dtype=torch.int32)
        at, masks = 0, []
        for b, n in enumerate(counts):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
            masks += _tree(sizes[b], case["shape"], rng)
        if case["shape"] == "tree" and case["batch"] > 2:
            masks[sizes[0]] = 0  # a row that sees nothing
        # latent vectors behind a norm: unit size and a few large channels
        pages = torch.randn((at, page, wide), device="cuda", generator=g)
        pages[..., 5::97] *= 3.0
        st["pages"], st["table"] = pages.bfloat16(), table.cuda()
        st["kv_len"] = torch.tensor(lens, dtype=torch.int32).cuda()
        st["q_start"] = torch.tensor([0] + sizes).cumsum(0).int().cuda()
        st["mask"] = torch.tensor(masks, dtype=torch.int64).cuda() if case["shape"] == "tree" else None
        st["scale"] = 1.0 / math.sqrt(192)
        st["q"] = _randn((heads, sum(sizes), case["latent"]), g).transpose(0, 1)  # a product a head: head-major
        st["qr"] = _randn((sum(sizes), heads, 128 + case["rope"]), g)[..., 128:]
        st["out"] = torch.empty((sum(sizes), heads, case["latent"]), dtype=torch.bfloat16, device="cuda")
        st["n_max"] = max(sizes)
        return st
    if op == "expanded":
        q, lens = _prompts(case)
        heads, nope, rope = case["heads"], case["nope"], case["rope"]
        st["q"] = _randn((sum(q), heads, nope + rope), g, 1.3)
        kv = _randn((sum(lens), heads, 2 * nope), g)  # one up-projection's output
        st["k"], st["v"] = kv[..., :nope], kv[..., nope:]
        st["kr"] = _randn((sum(lens), rope), g)
        st["q_start"] = torch.tensor([0] + q).cumsum(0).int().cuda()
        st["kv_start"] = torch.tensor([0] + lens).cumsum(0).int().cuda()
        st["scale"] = 1.0 / math.sqrt(nope + rope)
        st["out"] = torch.empty((sum(q), heads, nope), dtype=torch.bfloat16, device="cuda")
        st["q_max"], st["kv_max"] = max(q), max(lens)
        return st
    page, pages, layers = case["page"], case["pages"], case["layers"]
    order = list(range(pages))
    rng.shuffle(order)
    rows = case["rows"] if op == "compact" else case["parents"] + case["children"]
    lens = _lengths(case, rows, 0)
    held = case["rows"] if op == "compact" else case["parents"]
    grown = [n + case.get("grow", 0) for n in lens]
    table = torch.full((rows, max(-(-n // page) for n in grown) + 1), -1, dtype=torch.int32)
    refs, at = torch.zeros(pages, dtype=torch.int32), 0
    for r in range(held):
        n = -(-grown[r] // page)
        table[r, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        refs[table[r, :n].long()] += 1
        at += n
        if op == "compact" and r % 3 == 1:  # shares its beginning with the row before
            n = min(-(-lens[r - 1] // page), n) // 2
            refs[table[r, :n].long()] -= 1
            table[r, :n] = table[r - 1, :n]
            refs[table[r, :n].long()] += 1
    st["refs"], st["table"] = refs.cuda(), table.cuda()
    st["pages"] = torch.randint(0, 256, (layers, pages, case["page_bytes"]), dtype=torch.uint8, device="cuda", generator=g)
    if op == "fork":
        st["source"] = torch.tensor([i % held for i in range(case["children"])], dtype=torch.int32).cuda()
        st["target"] = torch.arange(held, rows, dtype=torch.int32).cuda()
        for i in range(held, rows):
            lens[i] = lens[(i - held) % held]
        st["new_len"] = torch.tensor([n + case["grow"] for n in lens], dtype=torch.int32).cuda()
        st["copies"] = torch.empty((case["children"], 2), dtype=torch.int32, device="cuda")
    else:
        st["refs_out"], st["table_out"] = torch.empty_like(st["refs"]), torch.empty_like(st["table"])
        st["copies"] = torch.empty((pages, 2), dtype=torch.int32, device="cuda")
        st["count"] = torch.empty(1, dtype=torch.int32, device="cuda")
    st["kv_len"] = torch.tensor(lens, dtype=torch.int32).cuda()
    return st


# ------------------------------------------------------------------ plain forms

def _plain_turned(x, pos, table, layout, magnitude, transposed):
    """x f32 [tokens, heads, dims] with every dimension turned; angles in 64 bits."""
    turns = table.double()
    turns = torch.where(table < 0, turns + 2.0 ** 64, turns) / 2.0 ** 64
    angle = torch.remainder(pos.double()[:, None] * turns, 1.0) * (2 * math.pi)
    cos, sin = (torch.cos(angle) * magnitude).float()[:, None], (torch.sin(angle) * magnitude).float()[:, None]
    sin = -sin if transposed else sin
    if layout == HALF:
        a, b = x[..., :x.shape[-1] // 2], x[..., x.shape[-1] // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _plain_rope(case, st):
    lo, hi = case["offset"], case["offset"] + case["rope"]
    x = st["x"].float()
    y = _plain_turned(x[..., lo:hi], st["pos"], st["table"], case["layout"], st["magnitude"], case["transposed"])
    return torch.cat([x[..., :lo], y, x[..., hi:]], -1).to(st["x"].dtype)


def _plain_latent(case, st):
    kr = st["kr"].float()[:, None]
    if case["turn"]:
        kr = _plain_turned(kr, st["pos"], st["table"], case["layout"], st["magnitude"], False)
    rows = torch.cat([st["c"], kr[:, 0].bfloat16()], -1)
    keep = st["slots"] >= 0
    flat = st["pages"].view(-1, rows.shape[-1])
    flat[st["slots"][keep].long()] = rows[keep]
    back = torch.where(keep[:, None], flat[st["slots"].clamp(min=0).long()], torch.zeros_like(rows))
    return [back[:, :case["latent"]], back[:, case["latent"]:], st["pages"]]


def _plain_softmax(s, sees):
    s = s.masked_fill(~sees, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    return e, e.sum(-1, keepdim=True).clamp(min=1e-38)


def _plain_absorbed(case, st):
    heads, n, latent = case["heads"], st["n_max"], case["latent"]
    q_start, kv_len = st["q_start"].long(), st["kv_len"].long()
    k = st["pages"][st["table"].long()].flatten(1, 2).float()  # [B, tokens, latent + rope]
    size = q_start[1:] - q_start[:-1]
    i = torch.arange(n, device="cuda")
    rows = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = torch.cat([st["q"], st["qr"]], -1).float()[rows].flatten(1, 2)  # [B, n heads, latent + rope]
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    j = (torch.arange(k.shape[1], device="cuda") - (kv_len - size)[:, None])[:, None, :]  # place after the context
    if st["mask"] is None:
        sees = j <= i[:, None]
    else:
        sees = (j < 0) | ((st["mask"][rows][..., None] >> j.clamp(0, 63)) & 1 > 0) & (j < 64)
    sees = (sees & (j < size[:, None, None])).repeat_interleave(heads, 1)
    e, total = _plain_softmax(s, sees)
    o = torch.matmul(e, k[..., :latent]) / total
    return o.unflatten(1, (n, heads))[i < size[:, None]].bfloat16()


def _plain_expanded(case, st):
    q_start, kv_start = st["q_start"].long(), st["kv_start"].long()
    n, t = q_start[1:] - q_start[:-1], kv_start[1:] - kv_start[:-1]
    i, j = torch.arange(st["q_max"], device="cuda"), torch.arange(st["kv_max"], device="cuda")
    rows = (q_start[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    cols = (kv_start[:-1, None] + j).clamp(max=st["k"].shape[0] - 1)
    q = st["q"].float()[rows].transpose(1, 2)  # [B, heads, n, dims]
    k = torch.cat([st["k"], st["kr"][:, None].expand(-1, case["heads"], -1)], -1).float()[cols].transpose(1, 2)
    v = st["v"].float()[cols].transpose(1, 2)
    sees = (j < t[:, None])[:, None, :].expand(-1, i.numel(), -1)
    if case["causal"]:
        sees = sees & (j <= i[:, None] + (t - n)[:, None, None])
    e, total = _plain_softmax(torch.matmul(q, k.transpose(-1, -2)) * st["scale"], sees[:, None])
    o = torch.matmul(e, v) / total
    return o.transpose(1, 2)[i < n[:, None]].bfloat16()


def _plain_fork(case, st):
    refs, table, page = st["refs"], st["table"], case["page"]
    kids, src = st["target"].long(), st["source"].long()
    # the children's pages are given back
    had = table[kids].flatten().long()
    refs.index_add_(0, had.clamp(min=0), -(had >= 0).int())
    table[kids] = -1
    # whole pages shared, a part-filled last one copied to the lowest free page
    j = torch.arange(table.shape[1], device="cuda")
    whole, part = (st["kv_len"][src] // page)[:, None], st["kv_len"][src] % page > 0
    new = torch.where(j < whole, table[src], -1)
    refs.index_add_(0, new.flatten().clamp(min=0).long(), (new >= 0).flatten().int())
    free = torch.nonzero(refs == 0)[:, 0].int()
    rank = torch.cumsum(part.int(), 0) - 1
    got = torch.where(part, free[rank.clamp(min=0)], -1)
    last = table[src].gather(1, whole.long().clamp(max=table.shape[1] - 1))[:, 0]
    table[kids] = torch.where((j == whole) & part[:, None], got[:, None], new)
    refs[got[part].long()] = 1
    st["copies"].copy_(torch.stack([torch.where(part, last, -1), got], 1))
    # every row grown to its new length, lowest free pages first
    need = (j * page < st["new_len"][:, None]) & (table < 0)
    free = torch.nonzero(refs == 0)[:, 0].int()
    rank = (torch.cumsum(need.flatten().int(), 0) - 1).view(need.shape)
    table.copy_(torch.where(need, free[rank.clamp(min=0, max=free.numel() - 1)], table))
    refs[table[need].long()] = 1
    at = st["copies"][part].long()
    st["pages"][:, at[:, 1]] = st["pages"][:, at[:, 0]]
    return [refs, table, st["copies"], st["pages"]]


def _plain_compact(case, st):
    refs, table = st["refs"], st["table"]
    live = refs > 0
    n = int(live.sum())
    at = torch.arange(refs.numel(), device="cuda")
    src, dst = torch.nonzero(live & (at >= n))[:, 0], torch.nonzero(~live & (at < n))[:, 0]
    to = at.clone()
    to[src] = dst
    st["refs_out"].zero_()
    st["refs_out"][to[live]] = refs[live]
    st["table_out"].copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    st["copies"].fill_(-1)
    st["copies"][:src.numel()] = torch.stack([src, dst], 1).int()
    st["count"].fill_(src.numel())
    st["pages"][:, dst] = st["pages"][:, src]
    return [st["refs_out"], st["table_out"], st["copies"], st["count"], st["pages"]]


# ------------------------------------------------------------------ one pass

PLAIN = {"rope": _plain_rope, "latent": _plain_latent, "absorbed": _plain_absorbed, "expanded": _plain_expanded,
         "fork": _plain_fork, "compact": _plain_compact}


def run(state):
    st, case = state, state["case"]
    if not own:
        return PLAIN[case["op"]](case, st)
    import moe_decode_quantized_gb300 as moe
    op = case["op"]
    layout = moe.MOE_ROPE_HALF if case.get("layout") == HALF else moe.MOE_ROPE_INTERLEAVED
    if op == "rope":
        moe.rope(st["x"], st["out"], st["pos"], st["table"], offset=case["offset"], layout=layout,
                 magnitude=st["magnitude"], transposed=case["transposed"])
        return st["out"]
    if op in ("latent", "absorbed") and "kept" not in st:  # what a program keeps for its life: the cache's description
        st["kept"] = moe.LatentCache(st["pages"], case["latent"], case["rope"], case["page"])
    if op == "latent":
        turn = case["turn"]
        moe.latent_append(st["kept"], st["c"], st["kr"], st["slots"], positions=st["pos"] if turn else None,
                          table=st["table"] if turn else None, layout=layout, magnitude=st["magnitude"])
        moe.latent_read(st["kept"], st["slots"], st["c_out"], st["kr_out"])
        return [st["c_out"], st["kr_out"], st["pages"]]
    if op == "absorbed":
        if "ws" not in st:  # and a workspace
            st["ws"] = torch.empty(moe.latent_attention_workspace_bytes(st["kept"], case["heads"], case["batch"],
                                                                        st["q"].shape[0]), dtype=torch.uint8, device="cuda")
            moe.workspace_init(st["ws"])
        moe.latent_attention(st["kept"], st["q"], st["qr"], st["out"], st["q_start"], st["kv_len"], st["table"],
                             st["mask"], st["scale"], st["ws"])
        return st["out"]
    if op == "expanded":
        moe.latent_prompt_attention(st["q"], st["k"], st["kr"], st["v"], st["out"], st["q_start"], st["kv_start"],
                                    case["causal"], st["scale"])
        return st["out"]
    pool = moe.PagePool(st["refs"], case["page"])
    if op == "fork":
        moe.pages_free(pool, st["table"], st["target"])
        moe.pages_fork(pool, st["table"], st["kv_len"], st["source"], st["target"], st["copies"])
        moe.pages_grow(pool, st["table"], st["new_len"])
        moe.pages_copy(st["pages"], st["copies"])
        return [st["refs"], st["table"], st["copies"], st["pages"]]
    moe.pages_compact(pool, st["table"], st["refs_out"], st["table_out"], st["copies"], st["count"])
    moe.pages_copy(st["pages"], st["copies"], st["count"])
    return [st["refs_out"], st["table_out"], st["copies"], st["count"], st["pages"]]


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_turned(x, pos, dim, scaling, layout, transposed):
    """x float64 [..., dim] of one row a position (its first axis), by complex multiplication."""
    f, magnitude = _frequencies(dim, scaling)
    angle = pos.double().reshape((-1,) + (1,) * (x.dim() - 1)) * torch.tensor(f, dtype=torch.float64, device="cuda")
    by = torch.polar(torch.full_like(angle, magnitude), -angle if transposed else angle)
    if layout == HALF:
        z = torch.complex(x[..., :dim // 2].contiguous(), x[..., dim // 2:].contiguous()) * by
        return torch.cat([z.real, z.imag], -1)
    z = torch.view_as_complex(x.reshape(x.shape[:-1] + (dim // 2, 2)).contiguous()) * by
    return torch.view_as_real(z).flatten(-2)


def _exact_attention(q, k, v, sees, scale):
    """q [heads, n, dims], k [heads or 1, tokens, dims], v alike, sees [n, tokens] -> float64 [n, heads, dims of v]."""
    out = []
    for h in range(q.shape[0]):
        s = q[h] @ k[h % k.shape[0]].T * scale
        s[~sees] = -math.inf
        out.append(torch.softmax(s, -1).nan_to_num(nan=0.0) @ v[h % v.shape[0]])
    return torch.stack(out, 1)


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "rope":
        y, lo, hi = st["x"].double(), case["offset"], case["offset"] + case["rope"]
        y[..., lo:hi] = _exact_turned(y[..., lo:hi].clone(), st["pos"], case["rope"], case["scaling"], case["layout"],
                                      case["transposed"])
        return y
    if op == "latent":
        c, kr, pages = st["c"].double(), st["kr"].double(), st["pages"].double()
        if case["turn"]:
            kr = _exact_turned(kr, st["pos"], case["rope"], "plain", case["layout"], False)
        for t, s in zip((st["slots"] >= 0).nonzero()[:, 0].split(8192), st["slots"][st["slots"] >= 0].long().split(8192)):
            pages[s // case["page"], s % case["page"]] = torch.cat([c[t], kr[t]], 1)
        there = (st["slots"] >= 0).double()[:, None]
        return [c * there, kr * there, pages]
    out = []
    if op == "absorbed":
        starts = st["q_start"].tolist()
        for b in range(case["batch"]):
            n, length = starts[b + 1] - starts[b], int(st["kv_len"][b])
            place = torch.arange(length, device="cuda")
            k = st["pages"][st["table"][b].long()[place // case["page"]], place % case["page"]].double()
            sees = torch.ones((n, length), dtype=torch.bool)
            for i in range(n):
                m = (2 << i) - 1 if st["mask"] is None else int(st["mask"][starts[b] + i]) % (1 << 64)
                sees[i, length - n:] = torch.tensor([bool(m >> j & 1) for j in range(n)])
            q = torch.cat([st["q"][starts[b]:starts[b + 1]], st["qr"][starts[b]:starts[b + 1]]], -1).double()
            rows = q.flatten(0, 1)[None]  # all rows of all heads share the keys
            o = _exact_attention(rows, k[None], k[None, :, :case["latent"]],
                                 sees.cuda().repeat_interleave(case["heads"], 0), st["scale"])
            out.append(o[:, 0].unflatten(0, (n, case["heads"])))
        return torch.cat(out)
    if op == "expanded":
        qs, ks = st["q_start"].tolist(), st["kv_start"].tolist()
        for b in range(case["batch"]):
            n, t = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
            sees = torch.ones((n, t), dtype=torch.bool, device="cuda")
            sees = sees.tril(t - n) if case["causal"] else sees
            kr = st["kr"][ks[b]:ks[b + 1]].double()[:, None].expand(-1, case["heads"], -1)
            k = torch.cat([st["k"][ks[b]:ks[b + 1]].double(), kr], -1).transpose(0, 1)
            v = st["v"][ks[b]:ks[b + 1]].double().transpose(0, 1)
            out.append(_exact_attention(st["q"][qs[b]:qs[b + 1]].double().transpose(0, 1), k, v, sees, st["scale"]))
        return torch.cat(out)
    return None  # whole numbers and bytes

"""Rotary positions, the latent cache and latent attention on the GPU against plain 64-bit
implementations (latent_ref.py), with the bounds derived there from the documented roundings."""
import math
import random

import numpy as np
import pytest
import torch

import moe_decode_quantized_gb300 as moe

import latent_ref as ref

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def table_of(dim, **kw):
    t, magnitude = moe.rope_table(dim, **kw)
    return torch.from_numpy(t.view(np.int64)).cuda(), [int(x) for x in t], magnitude


def near(got, want, bound):
    """Every value within its bound; NaN and infinities where the plain form has them."""
    got = got.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine)
    off = ((got - want).abs() - bound)[fine]
    assert off.numel() == 0 or off.max() <= 0, (float(off.max()), int(off.argmax()), int((off > 0).sum()))


# ------------------------------------------------------------------ rotary positions

def rows_of(shape, kind, source, g):
    t, h, d = shape
    if source == "heads":
        return torch.randn((h, t, d), generator=g).to(kind).cuda().transpose(0, 1)
    if source == "odd":  # neither aligned nor strides of whole pieces
        return torch.randn((t, h, d + 3), generator=g).to(kind).cuda()[..., 3:]
    if source == "fused":
        return torch.randn((t, h + 2, d), generator=g).to(kind).cuda()[:, 1:h + 1]
    return torch.randn(shape, generator=g).to(kind).cuda()


@pytest.mark.parametrize("kind", [BF, F32])
@pytest.mark.parametrize("layout", [moe.MOE_ROPE_HALF, moe.MOE_ROPE_INTERLEAVED])
@pytest.mark.parametrize("tokens,heads,dim,rope,offset,source", [
    (1, 1, 2, 2, 0, "plain"), (8, 40, 128, 128, 0, "fused"), (5, 3, 192, 64, 128, "plain"), (33, 7, 96, 90, 6, "odd"),
    (700, 2, 64, 32, 0, "heads"), (1301, 5, 64, 64, 0, "fused"), (3, 129, 80, 16, 40, "plain"), (2, 1, 1024, 1024, 0, "plain"),
    (9, 4, 7, 4, 3, "odd")])
@pytest.mark.parametrize("place", ["out", "in"])
def test_rope(kind, layout, tokens, heads, dim, rope, offset, source, place):
    g = torch.Generator().manual_seed(tokens * 7 + dim)
    x = rows_of((tokens, heads, dim), kind, source, g)
    table, ints, _ = table_of(rope)
    positions = [random.Random(t).choice([t, -t, 2 ** 31 - 1 - t, -2 ** 31 + t, 100003 * t % 2 ** 31]) for t in range(tokens)]
    magnitude, transposed = 1.25, tokens % 2 == 0
    want = x.double().cpu()
    part = want[..., offset:offset + rope].clone()
    bound = torch.zeros_like(want)
    bound[..., offset:offset + rope] = ref.turned_bound(part, layout, magnitude, kind == BF)
    want[..., offset:offset + rope] = ref.turned(part, positions, ints, layout, magnitude, transposed)
    before = x.clone()
    out = x if place == "in" else rows_of((tokens, heads, dim), kind, "odd" if source == "heads" else "fused", g)
    moe.rope(x, out, i32(positions), table, offset=offset, layout=layout, magnitude=magnitude, transposed=transposed)
    near(out, want, bound)
    if place == "out":
        assert torch.equal(x, before)


def test_rope_moves_other_dimensions_bit_for_bit():
    x = torch.randint(-2 ** 15, 2 ** 15, (4, 3, 48), dtype=torch.int16).cuda().view(BF)  # NaNs among them
    for rows in (x, torch.zeros((4, 3, 49), dtype=BF, device="cuda")[..., 1:].copy_(x)):
        out = torch.zeros_like(x)
        moe.rope(rows, out, i32([1, 2, 3, 4]), table_of(16)[0], offset=16)
        for part in (slice(0, 16), slice(32, 48)):
            assert torch.equal(out[..., part].view(torch.int16), x[..., part].view(torch.int16))


@pytest.mark.parametrize("layout", [moe.MOE_ROPE_HALF, moe.MOE_ROPE_INTERLEAVED])
def test_rope_transposed_is_the_gradient(layout):
    """<rope(x), y> = <x, rope_transposed(y)>, and the quotient of differences along y's direction (the map is linear)."""
    g = torch.Generator().manual_seed(3)
    x, y = (torch.randn((50, 6, 64), generator=g).cuda() for _ in range(2))
    table, _, magnitude = table_of(64, scaling=moe.MOE_ROPE_PARTS, factor=16.0)
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 977
    fx, by = torch.empty_like(x), torch.empty_like(x)
    moe.rope(x, fx, pos, table, layout=layout, magnitude=magnitude)
    moe.rope(y, by, pos, table, layout=layout, magnitude=magnitude, transposed=True)
    lhs, rhs = (fx.double() * y.double()).sum(), (x.double() * by.double()).sum()
    size = (x.double().abs() * by.double().abs()).sum()
    assert abs(lhs - rhs) <= 2e-6 * magnitude * size
    step = 2.0 ** -6
    moved = torch.empty_like(x)
    d = torch.randn((50, 6, 64), generator=g).cuda()
    moe.rope(x + step * d, moved, pos, table, layout=layout, magnitude=magnitude)
    quotient = ((moved.double() - fx.double()) * y.double()).sum() / step
    along = (by.double() * d.double()).sum()
    assert abs(quotient - along) <= 5e-7 * magnitude * 4 / step * (x.double().abs() + d.double().abs()).mean() * y.double().abs().sum()


# ------------------------------------------------------------------ the cache

def make_cache(latent, rope, page, pages, fill=float("nan")):
    t = torch.full((pages, page, latent + rope), fill, dtype=BF, device="cuda")
    return moe.LatentCache(t, latent, rope, page)


@pytest.mark.parametrize("latent,rope,page,tokens,source", [(512, 64, 64, 130, "fused"), (128, 8, 16, 1, "fused"),
                                                            (256, 24, 48, 77, "odd"), (512, 32, 32, 40, "plain")])
@pytest.mark.parametrize("turn", [None, moe.MOE_ROPE_HALF, moe.MOE_ROPE_INTERLEAVED])
def test_append_and_read(latent, rope, page, tokens, source, turn):
    g = torch.Generator().manual_seed(latent + tokens)
    wide = torch.randn((tokens, latent + rope + 3), generator=g).bfloat16().cuda()
    c, kr = (wide[:, 3:latent + 3], wide[:, latent + 3:]) if source == "odd" else (wide[:, :latent], wide[:, latent:latent + rope])
    if source == "plain":
        c, kr = c.contiguous(), kr.contiguous()
    pages = tokens // page + 3
    cache = make_cache(latent, rope, page, pages, 7.0)
    rng = np.random.default_rng(tokens)
    slots = rng.permutation(pages * page)[:tokens].astype(np.int32)
    bad = []
    if tokens > 20:
        slots[[3, 9, 11]] = [-1, pages * page, -5]
        bad = [3, 9, 11]
    status = i32([0])
    table, ints, _ = table_of(rope)
    positions = [t * 1009 for t in range(tokens)]
    kw = {} if turn is None else dict(positions=i32(positions), table=table, layout=turn, magnitude=0.75)
    moe.latent_append(cache, c, kr, torch.from_numpy(slots).cuda(), status=status, **kw)
    assert status.item() == (moe.MOE_WS_INDEX if bad else 0)
    wc, wk = c.double().cpu(), kr.double().cpu()
    bound = torch.zeros_like(wk)
    if turn is not None:
        bound = ref.turned_bound(wk, turn, 0.75, True)
        wk = ref.turned(wk[:, None], positions, ints, turn, 0.75)[:, 0]
    flat = cache.pages.double().cpu().view(-1, latent + rope)
    untouched = torch.ones(flat.shape[0], dtype=torch.bool)
    for t in range(tokens):
        if t in bad:
            continue
        untouched[slots[t]] = False
        assert torch.equal(flat[slots[t], :latent], wc[t])
        assert ((flat[slots[t], latent:] - wk[t]).abs() <= bound[t]).all()
    assert (flat[untouched] == 7.0).all()
    co, ko = (torch.full((tokens, d + 5), 3.0, dtype=BF, device="cuda") for d in (latent, rope))
    status.zero_()
    moe.latent_read(cache, torch.from_numpy(slots).cuda(), co[:, :latent], ko[:, 5:], status=status)
    assert status.item() == (moe.MOE_WS_INDEX if bad else 0)
    for t in range(tokens):
        row = flat[slots[t]] if t not in bad else torch.zeros(latent + rope, dtype=torch.float64)
        assert torch.equal(torch.cat([co[t, :latent], ko[t, 5:]]).double().cpu(), row)
    assert (co[:, latent:] == 3).all() and (ko[:, :5] == 3).all()


def test_rows_past_4_gigabytes():
    cache = make_cache(512, 64, 64, 90000)  # 6.6 GB
    n = 90000 * 64
    slots = i32([0, n - 1, n // 2, 4 * 10 ** 6])
    c, kr = torch.randn((4, 512), device="cuda").bfloat16(), torch.randn((4, 64), device="cuda").bfloat16()
    moe.latent_append(cache, c, kr, slots)
    flat = cache.pages.view(-1, 576)
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(flat[s], torch.cat([c[t], kr[t]]))
    # and read by attention through the last pages of the pool
    q, qr = torch.randn((1, 2, 512), device="cuda").bfloat16(), torch.randn((1, 2, 64), device="cuda").bfloat16()
    out, ws = torch.empty_like(q), workspace(cache, 2, 1, 1)
    flat[n - 64:] = 0.5
    flat[n - 1, :512] = c[1]
    moe.latent_attention(cache, q, qr, out, i32([0, 1]), i32([64]), i32([[89999]]), None, 0.1, ws)
    k = flat[n - 64:].double().cpu()[:, None]
    want, bound = ref.attention(torch.cat([q, qr], -1).double().cpu(), k, k[..., :512], torch.ones((1, 64), dtype=torch.bool), 0.1)
    near(out, want, bound)


# ------------------------------------------------------------------ absorbed form

def workspace(cache, heads, batch, tokens):
    ws = torch.empty(moe.latent_attention_workspace_bytes(cache, heads, batch, tokens), dtype=torch.uint8, device="cuda")
    moe.workspace_init(ws)
    return ws


class Case:
    """Sequences of n rows over `lens` tokens, their rows in shuffled pages whose other rows are NaN."""

    def __init__(self, latent, rope, heads, page, sizes, lens, masks=None, seed=0, source="fused", size=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = random.Random(seed)
        self.heads, self.sizes, self.lens, self.latent, self.rope = heads, sizes, lens, latent, rope
        counts = [-(-n // page) for n in lens]
        order = list(range(sum(counts) + 2))
        rng.shuffle(order)
        self.cache = make_cache(latent, rope, page, len(order))
        self.table = torch.full((len(lens), max(max(counts), 1) + 1), 10 ** 6, dtype=torch.int32)
        self.rows = [torch.randn((n, latent + rope), generator=g).bfloat16() * size for n in lens]
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table = self.table.cuda()
        self.write()
        total = sum(sizes)
        self.q, self.qr = self.queries(total, heads, latent, source, g), self.queries(total, heads, rope, source, g)
        self.out = self.queries(total, heads, latent, source, g)
        self.q_start = i32(np.cumsum([0] + sizes).tolist())
        self.kv_len = i32(lens)
        self.masks = masks
        self.mask = None if masks is None else torch.tensor([m - 2 ** 64 if m >> 63 else m for m in masks], dtype=torch.int64).cuda()
        self.ws = workspace(self.cache, heads, len(lens), total)

    def write(self):
        flat = self.cache.pages.view(-1, self.latent + self.rope)
        page = self.cache.page_size
        for b, r in enumerate(self.rows):
            place = torch.arange(r.shape[0], device="cuda")
            flat[self.table[b].long()[place // page] * page + place % page] = r.cuda()

    @staticmethod
    def queries(total, heads, dim, source, g):
        if source == "heads":
            return torch.randn((heads, total, dim), generator=g).bfloat16().cuda().transpose(0, 1)
        if source == "odd":
            return torch.randn((total, heads, dim + 1), generator=g).bfloat16().cuda()[..., 1:]
        return torch.randn((total, heads + 1, dim), generator=g).bfloat16().cuda()[:, :heads]

    def sees(self, b):
        n, t, first = self.sizes[b], self.lens[b], sum(self.sizes[:b])
        s = torch.ones((n, t), dtype=torch.bool)
        for i in range(n):
            m = (2 << i) - 1 if self.masks is None else self.masks[first + i]
            for j in range(n):
                s[i, t - n + j] = bool(m >> j & 1)
        return s

    def run(self, scale, **kw):
        moe.latent_attention(self.cache, self.q, self.qr, self.out, self.q_start, self.kv_len, self.table, self.mask, scale,
                             self.ws, **kw)
        return self.out

    def check(self, scale, got=None, skip=()):
        got = self.out if got is None else got
        first = 0
        for b, n in enumerate(self.sizes):
            if b not in skip and n:
                k = self.rows[b].double()[:, None]
                q = torch.cat([self.q[first:first + n], self.qr[first:first + n]], -1).double().cpu()
                near(got[first:first + n], *ref.attention(q, k, k[..., :self.latent], self.sees(b), scale))
            first += n


@pytest.mark.parametrize("latent,rope", [(512, 64), (512, 40), (256, 64), (128, 8), (256, 32)])
@pytest.mark.parametrize("heads,page,lens", [
    (16, 64, [511]), (1, 16, [1]), (128, 64, [300, 1, 77]), (3, 48, [64, 65, 127, 128, 129, 191, 192]), (64, 1024, [1000]),
    (33, 16, [15, 16, 17, 640])])
def test_single_tokens(latent, rope, heads, page, lens):
    c = Case(latent, rope, heads, page, [1] * len(lens), lens, seed=latent + heads, source=["fused", "heads", "odd"][heads % 3])
    c.run(0.07)
    c.check(0.07)
    assert moe.read_status(c.ws) == 0


@pytest.mark.parametrize("latent,rope,heads,page,sizes,lens", [
    (512, 64, 32, 16, [8, 5, 8], [700, 5, 129]), (512, 64, 5, 64, [64], [64]), (512, 64, 128, 32, [3, 2], [200, 131]),
    (256, 16, 7, 48, [20, 1, 40], [333, 1, 40]), (128, 64, 16, 64, [8] * 9, [130 + 17 * i for i in range(9)]),
    (512, 64, 16, 64, [17, 63], [17, 2000])])
@pytest.mark.parametrize("shape", ["chain", "tree", "any"])
def test_drafted_rows(latent, rope, heads, page, sizes, lens, shape):
    rng = random.Random(sum(lens))
    masks = None
    if shape == "tree":
        masks = []
        for n in sizes:
            own = []
            for j in range(n):
                own.append((own[rng.randint(max(0, j // 2 - 1), j - 1)] if j else 0) | 1 << j)
            masks += own
    elif shape == "any":  # any bits, past the rows too; rows that see no drafted token
        masks = [rng.choice([rng.getrandbits(64), 0, 1 << 63, rng.getrandbits(64) & rng.getrandbits(64)]) for n in sizes for _ in range(n)]
    c = Case(latent, rope, heads, page, sizes, lens, masks, seed=len(sizes))
    c.run(0.05)
    c.check(0.05)
    assert moe.read_status(c.ws) == 0


def test_rows_that_see_nothing_and_sequences_without_rows():
    c = Case(512, 64, 4, 16, [2, 0, 3, 1], [2, 50, 3, 20], [0, 1, 0, 7, 5, 0], seed=4)
    c.out.fill_(9.0)
    c.run(0.1)
    c.check(0.1)
    assert (c.out[0] == 0).all() and (c.out[2] == 0).all()


def test_rows_behind_the_last_sequence_are_left():
    c = Case(256, 64, 4, 16, [2, 3], [20, 3], seed=6)
    c.q_start, c.kv_len, c.table = c.q_start[:2], c.kv_len[:1], c.table[:1]
    c.out.fill_(9.0)
    c.run(0.1)
    c.check(0.1, skip=(1,))
    assert (c.out[2:] == 9).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_values_of_tokens_that_a_row_does_not_see(what):
    """Of siblings in a tree, and of drafted tokens that no row sees: no trace in the rows that do not see them."""
    masks = [1, 3, 5, 9, 11]  # node 3 is seen by rows 3 and 4 (bit 3), node 4 by none
    c = Case(512, 64, 20, 16, [5, 2], [150, 40], masks + [1, 3], seed=8)
    for part in (slice(0, 512), slice(512, 576), slice(100, 101)):
        keep = [r.clone() for r in c.rows]
        for node in (3, 4):
            c.rows[0][150 - 5 + node, part] = what
        c.write()
        c.run(0.05)
        blind = torch.cat([c.out[:3], c.out[5:]])
        c.rows = keep
        first = 0
        for b, (rows, n) in enumerate(zip(c.rows, c.sizes)):
            k = rows.double()[:, None]
            q = torch.cat([c.q[first:first + n], c.qr[first:first + n]], -1).double().cpu()
            want, bound = ref.attention(q, k, k[..., :512], c.sees(b), 0.05)
            near(blind[:3] if b == 0 else blind[3:], want[:3] if b == 0 else want, bound[:3] if b == 0 else bound)
            first += n
        if math.isnan(what):
            assert torch.isnan(c.out[3:5]).any(-1).all()
        c.write()


def test_a_token_seen_that_is_not_a_number():
    c = Case(512, 64, 3, 16, [1, 1], [150, 300], seed=8)
    c.rows[0][70, 7] = float("nan")
    c.write()
    c.run(0.05)
    assert torch.isnan(c.out[0]).all()
    c.check(0.05, skip=(0,))
    c.q[1, 1, 9] = float("nan")  # a query's NaN stays in its row
    c.rows[0][70, 7] = 1.0
    c.write()
    c.run(0.05)
    assert torch.isnan(c.out[1, 1]).all() and torch.isfinite(c.out[1, 0]).all() and torch.isfinite(c.out[0]).all()


@pytest.mark.parametrize("scale", [1.0, -0.3, 0.0, 30.0, 1e-8])
def test_scales(scale):
    c = Case(512, 64, 9, 32, [1, 4], [517, 200], seed=12)
    c.run(scale)
    c.check(scale)


def test_scores_of_any_size():
    """Queries of 1e18 against unit rows: the largest score takes all, without infinities."""
    c = Case(512, 64, 6, 32, [1, 2], [517, 200], seed=13)
    c.q.mul_(1e18)
    c.qr.mul_(1e18)
    c.run(1.0)
    first = 0
    for b, n in enumerate(c.sizes):
        q = torch.cat([c.q[first:first + n], c.qr[first:first + n]], -1).double().cpu()
        s = torch.einsum("nhd,td->nht", q, c.rows[b].double()).masked_fill(~c.sees(b)[:, None], -math.inf)
        top = s.topk(2, -1)
        assert (top.values[..., 0] - top.values[..., 1] > 1e13).all()
        want = c.rows[b][:, :512][top.indices[..., 0]]
        assert torch.equal(c.out[first:first + n].cpu(), want)
        first += n


def test_pages_and_lengths_outside():
    c = Case(512, 64, 8, 16, [2, 1, 2, 1], [100, 90, 60, 40], seed=14)
    c.table[0, 2] = c.cache.n_pages  # tokens 32 .. 47 are not seen
    c.table[1, 0] = -1
    c.kv_len[2] = 1                  # fewer than its rows
    c.out.fill_(9.0)
    c.run(0.06)
    assert moe.read_status(c.ws) == moe.MOE_WS_INDEX
    assert (c.out[3:5] == 0).all()
    first = 0
    for b, gone in ((0, slice(32, 48)), (1, slice(0, 16)), (3, slice(0, 0))):
        first = sum(c.sizes[:b])
        n = c.sizes[b]
        sees = c.sees(b)
        sees[:, gone] = False
        k = c.rows[b].double()[:, None]
        q = torch.cat([c.q[first:first + n], c.qr[first:first + n]], -1).double().cpu()
        near(c.out[first:first + n], *ref.attention(q, k, k[..., :512], sees, 0.06))
    moe.workspace_init(c.ws)
    for lens in ([-1, 90, 60, 40], [100, 10 ** 9, 60, 40]):
        c.table[0, 2], c.table[1, 0] = c.table[0, 1], c.table[1, 1]
        c.kv_len.copy_(i32(lens))
        c.run(0.06)
        assert moe.read_status(c.ws) == moe.MOE_WS_INDEX
        c.check(0.06, skip=(0, 1, 2))


def test_query_starts_outside():
    c = Case(512, 64, 8, 16, [2, 1, 2], [100, 90, 60], seed=15)
    c.q_start.copy_(i32([0, 2, 3, 70]))
    c.out.fill_(9.0)
    c.run(0.06)
    assert moe.read_status(c.ws) == moe.MOE_WS_INDEX
    c.check(0.06, skip=(2,))
    assert (c.out[3:] == 9).all()


def test_every_token_of_a_long_sequence_counts():
    """Rows of equal scores: the mean of all tokens' values; each token's value shows in a dimension of its own sum."""
    n = 40011
    pages = -(-n // 64)
    cache = make_cache(512, 64, 64, pages)
    flat = cache.pages.view(-1, 576)
    flat.zero_()
    place = torch.arange(n, device="cuda")
    table = torch.randperm(pages, device="cuda").int()[None]
    slot = table[0].long()[place // 64] * 64 + place % 64
    flat[slot, place % 512] = 1.0
    flat[table[0].long()[-1] * 64 + n % 64:(table[0].long()[-1] + 1) * 64] = float("nan")
    q, qr = torch.zeros((2, 128, 512), dtype=BF, device="cuda"), torch.zeros((2, 128, 64), dtype=BF, device="cuda")
    out, ws = torch.empty_like(q), workspace(cache, 128, 1, 2)
    moe.latent_attention(cache, q, qr, out, i32([0, 2]), i32([n]), table, None, 1.0, ws)
    for i in range(2):
        seen = n - 1 + i
        want = torch.bincount(place[:seen] % 512, minlength=512).double() / seen
        assert ((out[i].double() - want).abs() <= ref.BF16 * want + 1e-7).all()


def test_a_winning_token_anywhere():
    """One token of a large score, at each place of a length that is cut into runs: it is found, once."""
    n = 5000
    cache = make_cache(512, 64, 64, -(-n // 64), 0.0)
    flat = cache.pages.view(-1, 576)
    flat[:, 0] = torch.randn(flat.shape[0], device="cuda").bfloat16()
    table = torch.arange(-(-n // 64), dtype=torch.int32, device="cuda")[None]
    q, qr = torch.zeros((1, 16, 512), dtype=BF, device="cuda"), torch.zeros((1, 16, 64), dtype=BF, device="cuda")
    qr[:] = 1.0
    out, ws = torch.empty_like(q), workspace(cache, 16, 1, 1)
    for j in list(range(0, n, 61)) + [n - 1, 63, 64, 127, 128]:
        flat[j, 512:] = 2.0
        flat[j, 300] = 3.0
        moe.latent_attention(cache, q, qr, out, i32([0, 1]), i32([n]), table, None, 1.0, ws)
        assert (out[0, :, 300] == 3.0).all() and torch.equal(out[0, :, 0], flat[j, 0].expand(16))
        flat[j, 300:] = 0.0


def test_graphs_streams_and_one_workspace():
    """Two captured calls that share a workspace, replayed in turn on another stream, with lengths changed between."""
    a = Case(512, 64, 32, 32, [1, 1, 1], [900, 40, 333], seed=21)
    b = Case(512, 64, 16, 32, [8, 4], [600, 50], seed=22)
    b.ws = a.ws
    stream = torch.cuda.Stream()
    graphs = []
    for c in (a, b):
        c.run(0.07)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            c.run(0.07)
        graphs.append(g)
    for lens in ([900, 40, 333], [17, 40, 1], [64, 1, 128]):
        a.lens = lens
        a.rows = [r[:n] for r, n in zip(Case(512, 64, 32, 32, [1, 1, 1], [900, 40, 333], seed=21).rows, lens)]
        a.kv_len.copy_(i32(lens))
        a.out.fill_(5.0)
        b.out.fill_(5.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(3):
                graphs[0].replay()
                graphs[1].replay()
        stream.synchronize()
        a.check(0.07)
        b.check(0.07)
    first = a.out.clone()
    a.run(0.07)
    assert torch.equal(a.out, first)  # the same whatever the timing


def test_a_run_on_a_stream_given():
    c = Case(256, 64, 8, 16, [1], [77], seed=23)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.run(0.05, stream=s)
    s.synchronize()
    c.check(0.05)


def test_large_batch():
    n = 1024
    lens = [1 + 7 * b % 50 for b in range(n)]
    c = Case(128, 16, 2, 16, [1] * n, lens, seed=24)
    c.run(0.1)
    c.check(0.1)


# ------------------------------------------------------------------ expanded form

class Prompt:
    def __init__(self, nope, rope, heads, q, kv, causal=True, seed=0, size=1.0):
        g = torch.Generator().manual_seed(seed)

        def rand(*shape):
            return (torch.randn(shape, generator=g) * size).bfloat16().cuda()

        self.nope, self.heads, self.n, self.t, self.causal = nope, heads, q, kv, causal
        self.q = rand(sum(q), heads, nope + rope)
        kvs = rand(max(sum(kv), 1), heads, 2 * nope)
        self.k, self.v = kvs[:sum(kv), :, :nope], kvs[:sum(kv), :, nope:]
        self.kr = rand(sum(kv), rope + 8)[:, 8:]
        self.out = rand(sum(q), heads, nope + 5)[..., :nope]
        self.q_start, self.kv_start = (i32(np.cumsum([0] + x).tolist()) for x in (q, kv))
        self.status = i32([0])

    def run(self, scale, **kw):
        moe.latent_prompt_attention(self.q, self.k, self.kr, self.v, self.out, self.q_start, self.kv_start, self.causal, scale,
                                    status=self.status, **kw)
        return self.out

    def check(self, scale, skip=()):
        qs, ks = np.cumsum([0] + self.n), np.cumsum([0] + self.t)
        for b, (n, t) in enumerate(zip(self.n, self.t)):
            if b in skip or n == 0:
                continue
            a, z = slice(qs[b], qs[b + 1]), slice(ks[b], ks[b + 1])
            sees = torch.ones((n, t), dtype=torch.bool)
            sees = sees.tril(t - n) if self.causal else sees
            k = torch.cat([self.k[z], self.kr[z][:, None].expand(-1, self.heads, -1)], -1).double().cpu()
            near(self.out[a], *ref.attention(self.q[a].double().cpu(), k, self.v[z].double().cpu(), sees, scale))
        assert self.status.item() == 0 or skip


@pytest.mark.parametrize("nope,rope", [(128, 64), (64, 64), (128, 8), (64, 40)])
@pytest.mark.parametrize("heads,q,kv", [(1, [1], [1]), (2, [300], [300]), (3, [1, 130, 0, 64], [40, 200, 30, 64]),
                                        (2, [128, 129, 255], [128, 400, 255]), (1, [257, 2], [513, 700]), (5, [7] * 20, [7] * 20)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(nope, rope, heads, q, kv, causal):
    p = Prompt(nope, rope, heads, q, kv, causal, seed=sum(q) + heads)
    p.run(0.09)
    p.check(0.09)


def test_prompt_with_fewer_tokens_than_rows():
    p = Prompt(128, 64, 2, [200, 5, 3], [70, 0, 3], seed=1)
    p.out.fill_(9.0)
    p.run(0.09)
    p.check(0.09)
    assert (p.out[:130] == 0).all() and (p.out[200:205] == 0).all()


def test_prompt_without_tokens_or_rows():
    p = Prompt(128, 64, 2, [3], [0], seed=1)
    p.out.fill_(9.0)
    p.run(0.09)
    assert (p.out == 0).all()
    p = Prompt(128, 64, 2, [0, 0], [3, 0], seed=1)
    p.run(0.09)


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_prompt_later_tokens_leave_no_trace(what):
    """Of the row's own sequence, and of the sequence that follows in memory."""
    p = Prompt(128, 64, 2, [150, 40], [150, 60], seed=2)
    keep = [x.clone() for x in (p.k, p.kr, p.v)]
    for j, t in ((100, p.k), (120, p.kr), (131, p.v), (150, p.k), (151, p.v)):
        t[j] = what
    p.run(0.09)
    got = p.out[:100].clone()
    for x, y in zip((p.k, p.kr, p.v), keep):
        x.copy_(y)
    p.run(0.09)
    p.check(0.09)
    near(got, p.out[:100].double().cpu(), torch.zeros((100, 2, 128), dtype=torch.float64))


@pytest.mark.parametrize("scale", [-0.2, 0.0, 5.0, 1e-9])
def test_prompt_scales(scale):
    p = Prompt(128, 64, 2, [140, 3], [300, 300], seed=3)
    p.run(scale)
    p.check(scale)


def test_prompt_starts_outside():
    p = Prompt(128, 64, 2, [20, 30, 10], [20, 40, 10], seed=4)
    p.kv_start.copy_(i32([0, 20, 60, 71]))
    p.out.fill_(9.0)
    p.run(0.1)
    p.check(0.1, skip=(2,))
    assert p.status.item() == moe.MOE_WS_INDEX and (p.out[50:] == 0).all()


def test_prompt_rows_that_no_sequence_has_are_left():
    p = Prompt(128, 64, 2, [20, 30], [20, 40], seed=5)
    p.q_start, p.kv_start = p.q_start[:2], p.kv_start[:2]
    p.out.fill_(9.0)
    p.run(0.1)
    p.check(0.1, skip=(1,))
    assert (p.out[20:] == 9).all()


def test_prompt_graphs():
    p = Prompt(128, 64, 4, [200, 80], [300, 80], seed=6)
    p.run(0.1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run(0.1)
    p.q.neg_()
    p.n, p.t = [100, 180], [180, 200]
    p.q_start.copy_(i32([0, 100, 280]))
    p.kv_start.copy_(i32([0, 180, 380]))
    for _ in range(3):
        p.out.fill_(5.0)
        g.replay()
        p.check(0.1)


def test_both_forms_agree():
    """A sequence's last rows through the expanded form over its whole prompt and the absorbed form over the cache."""
    g = torch.Generator().manual_seed(31)
    n, rows, heads, latent, rope, nope = 300, 8, 16, 512, 64, 128
    c = torch.randn((n, latent), generator=g).bfloat16().cuda()
    kr = torch.randn((n, rope), generator=g).bfloat16().cuda()
    uk, uv = (torch.randn((heads, nope, latent), generator=g).cuda() * latent ** -0.5 for _ in range(2))
    q = torch.randn((rows, heads, nope + rope), generator=g).bfloat16().cuda()
    cache = make_cache(latent, rope, 64, 5)
    slots = torch.randperm(5, generator=g).int().repeat_interleave(64).cuda() * 64 + torch.arange(320, device="cuda").int() % 64
    moe.latent_append(cache, c, kr, slots[:n].contiguous())
    scale = (nope + rope) ** -0.5
    k, v = (torch.einsum("tl,hdl->thd", c.float(), w).bfloat16() for w in (uk, uv))
    full = torch.empty((rows, heads, nope), dtype=BF, device="cuda")
    moe.latent_prompt_attention(q, k, kr, v, full, i32([0, rows]), i32([0, n]), True, scale)
    ql = torch.einsum("nhd,hdl->nhl", q[..., :nope].float(), uk).bfloat16()
    ol = torch.empty((rows, heads, latent), dtype=BF, device="cuda")
    table = (slots[::64] // 64)[None].contiguous()
    moe.latent_attention(cache, ql, q[..., nope:], ol, i32([0, rows]), i32([n]), table, None, scale, workspace(cache, heads, 1, rows))
    short = torch.einsum("nhl,hdl->nhd", ol.float(), uv)
    # five roundings to bf16 on the way (k, v, the folded query, the latent output, the results), each 2^-8 of its value at
    # most: a score of about 1 moves by a few 2^-8, and so does a weight; values of unit size, averaged
    assert (short - full.float()).abs().max() <= 8 * ref.BF16 * 1.5
    assert (short - full.float()).square().mean().sqrt() <= ref.BF16


# ------------------------------------------------------------------ more of what a caller can do

def test_batch_that_leaves_three_stages():
    n = 300
    lens = [1 + 37 * b % 400 for b in range(n)]
    c = Case(512, 64, 3, 16, [1] * n, lens, seed=41)
    c.run(0.06)
    c.check(0.06)


def test_most_rows_a_sequence():
    c = Case(512, 64, 128, 64, [64], [200], seed=42)
    c.run(0.06)
    got = c.out[:, ::17]
    k = c.rows[0].double()[:, None]
    q = torch.cat([c.q, c.qr], -1)[:, ::17].double().cpu()
    near(got, *ref.attention(q, k, k[..., :512], c.sees(0), 0.06))


def test_an_item_of_many_runs_beside_short_ones():
    lens = [30000] + [3] * 20
    c = Case(256, 64, 16, 64, [1] * 21, lens, seed=43)
    c.run(0.02)
    c.check(0.02)
    assert moe.read_status(c.ws) == 0


@pytest.mark.parametrize("layout", ["heads", "shared", "odd"])
def test_prompts_of_other_layouts(layout):
    """Head-major tensors; keys and values that all heads share (expanded); queries that TMA does not take."""
    p = Prompt(128, 64, 3, [130, 40], [200, 40], seed=44)
    if layout == "heads":
        p.q, p.k, p.v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (p.q, p.k, p.v))
        p.out = torch.empty((3, 170, 128), dtype=BF, device="cuda").transpose(0, 1)
    elif layout == "shared":
        p.k, p.v = (x[:, :1].contiguous().expand(-1, 3, -1) for x in (p.k, p.v))
    else:
        big = torch.zeros((170, 3, 193), dtype=BF, device="cuda")
        big[..., 1:] = p.q
        p.q = big[..., 1:]
    p.run(0.09)
    p.check(0.09)


def test_values_of_seen_tokens_that_are_not_finite():
    """In the tiles that are looked through and in those that are not: in their own dimensions, of the rows that see them."""
    p = Prompt(128, 64, 1, [300], [300], seed=45)
    p.v[10, 0, 5] = float("inf")
    p.v[150, 0, 7] = float("nan")
    p.v[290, 0, 9] = -float("inf")
    p.run(0.05)
    out = p.out[:, 0].double().cpu()
    assert (out[10:, 5] == math.inf).all() and torch.isfinite(out[:10]).all()
    assert torch.isnan(out[150:, 7]).all() and torch.isfinite(out[:150, 7]).all()
    assert (out[290:, 9] == -math.inf).all() and torch.isfinite(out[:290, 9]).all()
    assert torch.isfinite(out[:, [0, 1, 2, 3, 4, 6, 8] + list(range(10, 128))]).all()


@pytest.mark.parametrize("nope,rope", [(128, 64), (64, 24)])
@pytest.mark.parametrize("heads,q,kv", [(31, [300, 2, 255], [300, 700, 400]), (31, [513], [640]), (52, [129, 131], [130, 128])])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_of_many_heads(nope, rope, heads, q, kv, causal):
    """Too many for a CTA to every 128 rows: one to 256."""
    p = Prompt(nope, rope, heads, q, kv, causal, seed=sum(kv) + heads)
    p.out.fill_(9.0)
    p.run(0.09)
    p.check(0.09)


def test_values_that_are_not_finite_in_prompts_of_many_heads():
    p = Prompt(128, 64, 52, [300], [300], seed=47)
    p.v[10, :, 5] = float("inf")
    p.v[150, :, 7] = float("nan")
    p.v[290, :, 9] = -float("inf")
    p.run(0.05)
    out = p.out.double().cpu()
    assert (out[10:, :, 5] == math.inf).all() and torch.isfinite(out[:10]).all()
    assert torch.isnan(out[150:, :, 7]).all() and torch.isfinite(out[:150, :, 7]).all()
    assert (out[290:, :, 9] == -math.inf).all() and torch.isfinite(out[:290, :, 9]).all()
    assert torch.isfinite(out[..., [0, 1, 2, 3, 4, 6, 8] + list(range(10, 128))]).all()


@pytest.mark.parametrize("nope,rope", [(128, 64), (64, 40)])
@pytest.mark.parametrize("heads,q,kv", [(1, [40], [5000]), (2, [1, 300, 0], [3000, 2001, 600]), (9, [513], [4097]),
                                        (1, [3200], [3200]), (3, [128, 90], [1030, 60])])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_whose_tokens_are_shared_out(nope, rope, heads, q, kv, causal):
    """Few blocks of rows: several CTAs to each, a part of its tokens each (none, for rows that see few)."""
    p = Prompt(nope, rope, heads, q, kv, causal, seed=sum(kv) + heads)
    p.out.fill_(9.0)
    p.run(0.09)
    p.check(0.09)


def test_shared_out_tokens_that_are_not_finite():
    p = Prompt(128, 64, 1, [300], [4000], seed=48)
    p.v[10, 0, 5] = float("inf")
    p.v[3850, 0, 7] = float("nan")
    p.v[3990, 0, 9] = -float("inf")
    p.run(0.05)
    out = p.out[:, 0].double().cpu()  # row i sees tokens 0 .. 3700 + i
    assert (out[:, 5] == math.inf).all()
    assert torch.isnan(out[150:, 7]).all() and torch.isfinite(out[:150, 7]).all()
    assert (out[290:, 9] == -math.inf).all() and torch.isfinite(out[:290, 9]).all()
    assert torch.isfinite(out[:, [0, 1, 2, 3, 4, 6, 8] + list(range(10, 128))]).all()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 30.0])
def test_shared_out_scales(scale):
    """Scores far apart, so that parts weigh nothing beside others."""
    p = Prompt(64, 64, 2, [140, 3], [2000, 3000], seed=49)
    p.run(scale)
    p.check(scale)


def test_shared_out_tokens_in_a_graph():
    p = Prompt(128, 64, 2, [200, 80], [3000, 1080], seed=50)
    p.run(0.1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):
            p.run(0.1)
    p.q.neg_()
    p.n, p.t = [100, 180], [180, 3900]
    p.q_start.copy_(i32([0, 100, 280]))
    p.kv_start.copy_(i32([0, 180, 4080]))
    for _ in range(3):
        p.out.fill_(5.0)
        g.replay()
        p.check(0.1)


@pytest.mark.parametrize("heads,q,kv", [(2, [200, 80], [3000, 1080]), (16, [300, 700, 5], [301, 900, 2000])])
def test_prompts_give_the_same_bits_again(heads, q, kv):
    p = Prompt(128, 64, heads, q, kv, seed=51)
    p.run(0.1)
    once = p.out.clone()
    for _ in range(20):
        p.out.fill_(5.0)
        p.run(0.1)
        assert torch.equal(p.out[: sum(q)], once[: sum(q)])


def test_rope_and_rows_in_a_graph():
    g = torch.Generator().manual_seed(46)
    x, c = torch.randn((9, 4, 64), generator=g).bfloat16().cuda(), torch.randn((9, 144), generator=g).bfloat16().cuda()
    cache, table = make_cache(128, 16, 16, 3, 0.0), table_of(16)
    pos, slots = i32(list(range(9))), i32(list(range(20, 29)))
    out, co, ko = torch.empty_like(x), torch.empty((9, 128), dtype=BF, device="cuda"), torch.empty((9, 16), dtype=BF, device="cuda")

    def step():
        moe.rope(x, out, pos, table[0], offset=48)
        moe.latent_append(cache, c[:, :128], c[:, 128:], slots, pos, table[0])
        moe.latent_read(cache, slots, co, ko)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for first in (100, 70000):
        pos.copy_(i32(list(range(first, first + 9))))
        graph.replay()
        part = x[..., 48:].double().cpu()
        near(out[..., 48:], ref.turned(part, pos.tolist(), table[1], 0), ref.turned_bound(part, 0, 1.0, True))
        part = c[:, None, 128:].double().cpu()
        near(ko[:, None], ref.turned(part, pos.tolist(), table[1], 0), ref.turned_bound(part, 0, 1.0, True))
        assert torch.equal(co, c[:, :128])


def test_example_decodes_samples():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "latent_decode.py")
    spec = importlib.util.spec_from_file_location("latent_decode", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    prompts = [[3, 1, 4, 1, 5, 9, 2, 6] * 5, [2, 7, 1, 8]]
    model = ex.Model()
    out = ex.generate(model, prompts, 3, 20)
    assert [len(o) for o in out] == [20] * 6 and len({tuple(o) for o in out[:3]}) > 1
    # what six forked, grown and compacted rows hold: the prompt's tokens and 19 more
    counts = [-(-(len(p) + 19) // 16) for p in prompts for _ in range(3)]
    assert [(r >= 0).sum().item() for r in model.table[2:8]] == counts
    held = int((model.pool.refs > 0).sum())
    assert held == sum(counts) - 2 * (40 // 16)  # two full pages of the first prompt are shared by its three samples
    assert model.pool.refs.sum().item() == sum(counts)
    # the tokens so far as a prompt, anew: its last logits against those of the step that made the last token
    again = ex.Model()
    for b, p in ((0, 0), (4, 1)):
        fresh = ex.Model()
        logits = fresh.prompts([prompts[p] + out[b][:-1]])
        again.prompts([prompts[p]])
        for j, t in enumerate(out[b][:-1]):
            last = again.step([0], [len(prompts[p]) + j], [t])
        moe.pages_free(again.pool, again.table, i32([0]))
        # both forms round to bf16 some twenty times on the way, 2^-8 each of values of the size of the logits' inputs; the
        # logits are 4 times sums of 256 products
        assert (logits - last).abs().max() <= 20 * ref.BF16 * 4 and torch.corrcoef(torch.stack([logits[0], last[0]]))[0, 1] > 0.99

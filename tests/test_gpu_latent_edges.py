"""Edges of rotary positions and latent attention on the GPU, beside test_gpu_latent.py, against the same plain 64-bit
implementations (latent_ref.py)."""
import math

import numpy as np
import pytest
import torch

import moe_decode_quantized_gb300 as moe

import latent_ref as ref
import test_gpu_latent as base

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
i32 = base.i32


# ------------------------------------------------------------------ expanded form: starts

@pytest.mark.parametrize("heads,kv", [(4, [10, 10, 10]), (1, [4000, 30, 900]), (40, [200, 1, 300])])
@pytest.mark.parametrize("starts,rows", [
    ([0, 2000, 1000, 3000], 3000), ([0, 10 ** 9, 20, 60], 600), ([500, 100, 300, 600], 600), ([0, 300, 600, 771], 700),
    ([-5, 200, 500, 600], 600), ([200, 300, 0, 400], 600), ([0, 100, 100, 90], 300), ([0, 0, 700, 700], 800)])
def test_prompt_query_starts_that_do_not_hold(starts, rows, heads, kv):
    """A sequence that falls, lies outside or begins before an earlier one's start has no results: its rows that no other
    sequence has are 0. The others' are as ever, and rows that no sequence has stay."""
    p = base.Prompt(128, 64, heads, [rows], kv, seed=rows + heads)
    p.q_start, p.kv_start = i32(starts), i32(np.cumsum([0] + kv).tolist())
    p.out.fill_(9.0)
    p.run(0.1)
    held = [0 <= a <= z <= rows and a == max(starts[:b + 1]) for b, (a, z) in enumerate(zip(starts, starts[1:]))]
    assert p.status.item() == (0 if all(held) else moe.MOE_WS_INDEX)
    zero = torch.zeros(rows, dtype=torch.bool)
    for good, (a, z) in sorted(zip(held, zip(starts, starts[1:]))):
        zero[max(a, 0):max(min(z, rows), 0)] = not good
    some = torch.zeros(rows, dtype=torch.bool)
    for b, (a, z) in enumerate(zip(starts, starts[1:])):
        if held[b] and z > a:
            some[a:z] = True
            k0, t = int(p.kv_start[b]), kv[b]
            pick = sorted({a, z - 1, (a + z) // 2, *range(max(a, z - t - 1), min(z, max(a, z - t - 1) + 3))})
            k = torch.cat([p.k[k0:k0 + t], p.kr[k0:k0 + t, None].expand(-1, heads, -1)], -1).double().cpu()
            sees = torch.ones((z - a, t), dtype=torch.bool).tril(t - (z - a))[[r - a for r in pick]]
            cut = slice(0, heads, max(1, heads // 3))
            base.near(p.out[pick][:, cut], *ref.attention(p.q[pick][:, cut].double().cpu(), k[:, cut],
                                                          p.v[k0:k0 + t, cut].double().cpu(), sees, 0.1))
    out = p.out.cpu()
    assert (out[zero] == 0).all() and (out[~zero & ~some] == 9).all()


# ------------------------------------------------------------------ expanded form: layouts in each plan

@pytest.mark.parametrize("nope,rope", [(128, 64), (64, 40)])
@pytest.mark.parametrize("heads,q,kv", [(3, [130, 40], [200, 40]),      # a CTA to every 128 rows
                                        (52, [129, 131], [130, 128]),   # to every 256
                                        (3, [140, 60], [2100, 1100]), (19, [100], [4000]), (37, [90], [3000])])  # clusters
@pytest.mark.parametrize("layout", ["plain", "heads", "shared", "odd", "by 8"])
def test_prompts_of_other_layouts_in_each_plan(nope, rope, heads, q, kv, layout):
    """Results written 32 bytes at a time (plain, head-major), 16 (rows 8 values apart) and value by value (the others);
    keys and values of all heads; queries that TMA does not take."""
    p = base.Prompt(nope, rope, heads, q, kv, seed=heads + nope)
    n = sum(q)
    p.out = torch.full((n, heads, nope + (8 if layout == "by 8" else 5 if layout in ("shared", "odd") else 0)), 9.0, dtype=BF,
                       device="cuda")
    if layout == "heads":
        p.q, p.k, p.v = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (p.q, p.k, p.v))
        p.out = torch.empty((heads, n, nope), dtype=BF, device="cuda").transpose(0, 1)
    elif layout == "shared":
        p.k, p.v = (x[:, :1].contiguous().expand(-1, heads, -1) for x in (p.k, p.v))
    elif layout == "odd":
        big = torch.zeros((n, heads, nope + rope + 1), dtype=BF, device="cuda")
        big[..., 1:] = p.q
        p.q = big[..., 1:]
    whole, p.out = p.out, p.out[..., :nope]
    p.run(0.09)
    if layout not in ("plain", "heads"):
        assert (whole[..., nope:] == 9).all()
    cut = slice(0, heads, max(1, heads // 4))
    p.q, p.k, p.v, p.out = (x[:, cut] for x in (p.q, p.k, p.v, p.out))
    p.heads = p.q.shape[1]
    p.check(0.09)


# ------------------------------------------------------------------ expanded form: infinities that are seen

@pytest.mark.parametrize("heads,q,kv", [(3, 130, 400), (52, 260, 390), (3, 140, 3100)])  # 128 rows a CTA, 256, clusters
@pytest.mark.parametrize("back", [4, 135, 330])  # tokens from the end: of a tile that not all rows see, and not
def test_infinities_of_tokens_that_a_row_sees(heads, q, kv, back):
    """An infinite value whose token's score is -inf (a weight of 0), +inf or NaN: not finite in rows that see it. Rows that
    do not are as without the token."""
    p = base.Prompt(128, 64, heads, [q], [kv], seed=heads + back)
    at = kv - back
    p.kr[at, 7] = math.inf
    p.v[at, :, 5] = -math.inf
    p.run(0.09)
    out, score = p.out.float().cpu(), p.q[:, :, 128 + 7].float().cpu() * math.inf
    low = score == -math.inf
    sees = torch.arange(kv - q, kv) >= at
    assert not torch.isfinite(out[sees][..., 5]).any()
    assert torch.isnan(out[sees][~low[sees]]).all()
    others = [i for i in range(128) if i != 5]
    assert torch.isfinite(out[sees][low[sees]][:, others]).all() and low[sees].any()
    blind = (~sees).nonzero().flatten()[-3:]
    cut = slice(0, heads, max(1, heads // 3))
    if len(blind):
        k = torch.cat([p.k, p.kr[:, None].expand(-1, heads, -1)], -1).double().cpu()
        seen = torch.arange(kv) <= (kv - q + blind)[:, None]
        base.near(p.out[blind.cuda()][:, cut], *ref.attention(p.q[blind.cuda()][:, cut].double().cpu(), k[:, cut],
                                                              p.v[:, cut].double().cpu(), seen, 0.09))


# ------------------------------------------------------------------ absorbed form: scores that are exact in f32

class Exact(base.Case):
    """Queries and rows of multiples of 1/8 in eight dimensions, zeros in the queries' others: every product is a multiple of
    1/64 and every sum is below 2^8, so that scores have no error in f32 in any order."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        g = torch.Generator().manual_seed(1)
        self.rows = [(torch.randint(-24, 25, r.shape, generator=g) / 8).bfloat16() for r in self.rows]
        self.write()
        self.q.zero_()
        self.qr.zero_()
        for x, n in ((self.q, 5), (self.qr, 3)):
            x[..., :n] = (torch.randint(-24, 25, (*x.shape[:2], n), generator=g) / 8).to(x)

    def check_exact(self, scale):
        first = 0
        for b, n in enumerate(self.sizes):
            k = self.rows[b].double()
            q = torch.cat([self.q[first:first + n], self.qr[first:first + n]], -1).double().cpu()
            s = torch.einsum("nhd,td->nht", q, k).mul(math.copysign(1, scale)).masked_fill(~self.sees(b)[:, None], -math.inf)
            p = torch.exp((s - s.amax(-1, keepdim=True)) * abs(scale))
            p /= p.sum(-1, keepdim=True)
            v = k[:, :self.latent]
            o = p @ v
            # exponents and exponentials in f32 2^-14 in all (an exponent that weighs is below 2^5: 2^-18 of it and less),
            # weights rounded to bf16 and added up as rounded, sums 2^-14, one rounding to bf16
            far = torch.einsum("nht,nhtd->nhd", p, (v - o[..., None, :]).abs())
            bound = 1.01 * ref.BF16 * far + 2.0 ** -13 * (p @ v.abs())
            bound = bound * (1 + ref.BF16) + ref.BF16 * o.abs() + 1e-30
            assert (bound.mean() < 0.05 * o.abs().mean()), "a bound that zeros would pass"
            base.near(self.out[first:first + n], o, bound)
            first += n


@pytest.mark.parametrize("scale", [30.0, -30.0, 2.0, 1e4, 1e36, -1e37, 3e38])
@pytest.mark.parametrize("latent,heads,sizes,lens", [(512, 6, [1, 4], [517, 200]), (512, 16, [1], [3001]), (128, 3, [2, 1], [2500, 1]),
                                                     (256, 128, [1], [700])])
def test_scores_far_apart(latent, heads, sizes, lens, scale):
    """Items that are cut into runs and joined, and items that are not: the same whatever the scale, although a score times
    it passes what f32 holds."""
    c = Exact(latent, 64, heads, 32, sizes, lens, seed=sum(lens))
    c.run(scale)
    c.check_exact(scale)
    assert moe.read_status(c.ws) == 0


@pytest.mark.parametrize("scale", [30.0, 1e36, -3e38])
def test_scores_far_apart_of_many_runs(scale):
    """Joined by the kernel that takes items of many parts."""
    c = Exact(512, 64, 16, 64, [1], [40000], seed=3)
    c.run(scale)
    c.check_exact(scale)


# ------------------------------------------------------------------ absorbed form: infinities that are seen

@pytest.mark.parametrize("what", [math.inf, -math.inf])
@pytest.mark.parametrize("latent,heads,lens,scale", [(512, 20, [150, 40], 0.05), (512, 20, [150, 40], -0.05),
                                                     (128, 3, [4000, 40], 0.05), (256, 70, [70, 6], 0.05)])
@pytest.mark.parametrize("dims", [[100], [3, 127], [0, 64], "rope"])
def test_infinities_of_drafted_tokens_that_a_row_sees(latent, heads, lens, scale, dims, what):
    """A score of -inf is a weight of 0, and 0 times an infinity no number: in the token's dimensions that are infinite the
    row is NaN, in the others as without the token. A score of +inf or NaN: all of the row."""
    masks = [1, 3, 5, 9, 11]  # node 3 is seen by rows 3 and 4, node 1 by rows 1 and 4
    c = base.Case(latent, 64, heads, 16, [5, 2], lens, masks + [1, 3], seed=8)
    at = lens[0] - 5 + 3
    place = [latent + 9] if dims == "rope" else dims
    c.rows[0][at, place] = what
    c.write()
    c.run(scale)
    q = torch.cat([c.q, c.qr], -1).double().cpu()
    k, first = c.rows[0].double(), 0
    score = scale * (q[:, :, place] * what).sum(-1)  # what is finite does not matter beside it
    low = 0
    for i in range(5):
        sees = c.sees(0)[i:i + 1]
        for h in range(heads):
            got = c.out[i, h].double().cpu()
            if sees[0, at] and score[i, h] != -math.inf:
                assert torch.isnan(got).all()
                continue
            without = sees.clone()
            without[0, at] = False
            want, bound = ref.attention(q[i:i + 1, h:h + 1], k[:, None], k[:, None, :latent], without, scale)
            want = want[0, 0]
            if sees[0, at]:
                low += 1
                if dims != "rope":
                    want[place] = math.nan
                    assert torch.isnan(got[place]).all()
            base.near(got, want, bound[0, 0])
    assert low > 0 or heads < 20
    q1, k1 = q[5:], c.rows[1].double()[:, None]
    base.near(c.out[5:], *ref.attention(q1, k1, k1[..., :latent], c.sees(1), scale))


# ------------------------------------------------------------------ absorbed form: pages that are not there

@pytest.mark.parametrize("latent,heads,page,sizes,lens", [(128, 20, 16, [1], [20000]), (512, 70, 16, [3, 1], [9000, 700]),
                                                          (256, 128, 16, [1] * 4, [3000, 2000, 64, 16]), (128, 4, 48, [2], [30001])])
def test_pages_that_are_not_there_in_every_tile(latent, heads, page, sizes, lens):
    """Which of a tile's tokens are there differs from tile to tile: every tile takes its own."""
    c = base.Case(latent, 64, heads, page, sizes, lens, seed=17)
    for b, n in enumerate(lens):
        pages = -(-n // page)
        gone = torch.rand(pages, generator=torch.Generator().manual_seed(b)) < 0.4
        c.table[b, :pages][gone.cuda()] = c.cache.n_pages + 5
        c.rows[b] = torch.where(gone[torch.arange(n) // page, None], math.nan, c.rows[b])
    c.run(0.05)
    assert moe.read_status(c.ws) == moe.MOE_WS_INDEX
    once = c.out.clone()
    first = 0
    for b, n in enumerate(sizes):
        k = c.rows[b].double()[:, None]
        sees = c.sees(b) & ~torch.isnan(c.rows[b][:, 0])
        q = torch.cat([c.q[first:first + n], c.qr[first:first + n]], -1)[:, ::5].double().cpu()
        base.near(c.out[first:first + n, ::5], *ref.attention(q, k, k[..., :latent], sees, 0.05))
        first += n
    for _ in range(50):
        c.run(0.05)
        assert torch.equal(c.out, once)


# ------------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("layout", [moe.MOE_ROPE_HALF, moe.MOE_ROPE_INTERLEAVED])
def test_angles_next_to_quarter_turns(layout):
    """Small sines and cosines there are as near as documented: 2^-26 + 2^-33 of a turn for the angle's two roundings, and
    sine and cosine within an ulp, 2^-23, which is doubled for this plain form."""
    table, ints, _ = base.table_of(2)
    f, found = ints[0], []
    for p in range(1, 400000):
        t = p * f % 2 ** 64
        q = (t + 2 ** 61) >> 62
        rest = t - (q << 62)
        if 0 < abs(rest) < 2 ** 58:  # 1/64 of a turn
            found.append((p if p % 3 else -p, q % 4, rest))
    found = found[::7]
    assert {q for _, q, _ in found} == {0, 1, 2, 3} and len(found) > 1000
    x = torch.zeros((len(found), 1, 2), device="cuda")
    x[..., 0] = 1.0
    out = torch.empty_like(x)
    moe.rope(x, out, i32([p for p, _, _ in found]), table, layout=layout)
    for (c, s), (p, q, rest) in zip(out[:, 0].double().cpu().tolist(), found):
        small = math.sin(2 * math.pi * (rest / 2.0 ** 64)) * (-1 if q > 1 else 1)
        value = s if q % 2 == 0 else -c  # sine, -cosine, sine, -cosine from the nearest quarter turn
        small = -small if p < 0 and q % 2 == 0 else small
        assert abs(value - small) <= 2 * math.pi * (2.0 ** -26 + 2.0 ** -33) + abs(small) * 2.0 ** -22, (p, q, rest)


def test_the_most_tokens():
    """2^31 - 1 of one pair, in place: 26 GB with their positions."""
    n = 2 ** 31 - 1
    table, ints, _ = base.table_of(2)
    x = torch.zeros((n, 1, 2), dtype=BF, device="cuda")
    x[..., 0] = 1.0
    positions = torch.arange(n, dtype=torch.int32, device="cuda")
    moe.rope(x, x, positions, table)
    for at in (0, 2047, 2048, n // 2, n - 2049, n - 1):
        want = torch.zeros((1, 1, 2), dtype=torch.float64)
        want[..., 0] = 1.0
        base.near(x[at:at + 1], ref.turned(want, [at], ints, ref.HALF), ref.turned_bound(want, ref.HALF, 1.0, True))
    for at in range(0, n, n // 4):  # everywhere a turn of length 1, by roundings of 2^-8 each
        part = x[at:at + 10 ** 7].float()
        assert (part.square().sum(-1) - 1).abs().max() < 4 * ref.BF16

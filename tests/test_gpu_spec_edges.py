"""Edges of the speculative-decoding operators on the GPU, beside test_gpu_spec.py: what
clusters, waits, extreme scales and values, hidden tokens and empty calls come to. The same
plain 64-bit implementations (spec_ref.py) and, where nothing else is said, the same
tolerances."""
import random

import numpy as np
import pytest
import torch

import moe_decode_quantized_gb300 as moe

import spec_ref
import test_gpu_spec as base

pytestmark = pytest.mark.gpu


def verify_rows(sizes, vocab, kind, shape, drafts, seed, temps=(0.7, 1.0)):
    """A case of base.verify_case's form with the given numbers of rows."""
    rng, pick = np.random.default_rng(seed), random.Random(seed)
    rows, batch = sum(sizes), len(sizes)
    logits = torch.from_numpy((rng.standard_normal((rows, vocab), dtype=np.float32) * 2.5))
    logits = logits.bfloat16() if kind == "bf16" else logits
    case = {"tokens": [], "parents": [] if shape == "tree" else None, "u": [], "logits": logits.cuda(),
            "temp": [temps[b % len(temps)] for b in range(batch)], "noise": rng.exponential(size=(batch, vocab)) + 1e-12}
    l, at, draft = logits.float().numpy(), 0, np.zeros((rows, vocab) if drafts else (1, 1), np.float32)
    for b, n in enumerate(sizes):
        parents = [-1] + [pick.randint(max(0, j - 3), j - 1) if shape == "tree" else j - 1 for j in range(1, n)]
        tokens, t = [0], case["temp"][b] or 0.5
        for j in range(1, n):
            z = l[at + parents[j]] / np.float32(t) + rng.standard_normal(vocab, dtype=np.float32) * np.float32(0.5)
            p = np.exp(z - z.max(), dtype=np.float32)
            p /= p.sum()
            if drafts:
                draft[at + j] = p
            tokens.append(min(int(np.searchsorted(np.cumsum(p, dtype=np.float64), rng.random())), vocab - 1))
        case["tokens"].append(np.array(tokens[:n], dtype=np.int64))
        case["u"].append(rng.random(n))
        if shape == "tree":
            case["parents"].append(np.array(parents[:n], dtype=np.int64))
        at += n
    case["draft"] = torch.from_numpy(draft).cuda() if drafts else None
    return case


@pytest.mark.parametrize("ranks", range(2, 9))
@pytest.mark.parametrize("sizes,shape", [([5, 3, 7], "chain"), ([24] * 56, "tree")])
def test_verify_clusters_of_short_slices(ranks, sizes, shape):
    """Clusters of every size with the shortest slices, whose CTAs exchange their first results soonest after they
    start: rows ahead (the chains) and rows as the walk reaches them (the trees: more than 20 MB of logits)."""
    case = verify_rows(sizes, 2048 * ranks + 3, "f32", shape, shape == "chain", ranks)
    status, _ = base.check_verify(case)
    assert status == 0
    want = base.verify(case)[:3]
    for _ in range(3):
        assert base.verify(case)[:3] == want


def test_verify_of_refused_sequences_is_over_before_the_next_kernel():
    """Sequences of too many rows are refused at once, but the call ends only when its reads of the logits have: what
    the stream writes over them next is not seen (NaN would be flagged)."""
    rows, vocab = 70, 131072
    logits = torch.zeros((2 * rows, vocab), device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    starts, tokens = torch.tensor([0, rows, 2 * rows], **i32), torch.zeros(2 * rows, **i32)
    u, noise = torch.full((2 * rows,), 0.5, device="cuda"), torch.ones((2, vocab), device="cuda")
    n_acc, nxt, path = torch.full((2,), 9, **i32), torch.full((2,), 9, **i32), torch.full((2 * rows,), 9, **i32)
    ws = torch.empty(moe.spec_verify_workspace_bytes(2, 2 * rows), dtype=torch.uint8, device="cuda")
    moe.workspace_init(ws)
    for _ in range(20):
        moe.spec_verify(logits, starts, tokens, None, None, None, u, noise, n_acc, path, nxt, ws)
        logits.fill_(float("nan"))
        assert moe.read_status(ws) == moe.MOE_WS_INDEX
        assert n_acc.tolist() == [0, 0] and nxt.tolist() == [-1, -1]
        logits.zero_()


def refill(s, keys, values, skip=(), fill=0xFF):
    """The cache of a base.Sequences anew: `fill` in every byte, then the rows keys[b], values[b] [tokens, heads, dim]
    (bf16) but those of the places (sequence, token) in `skip`."""
    s.cache.pages.fill_(fill)
    table, page, slots = s.table.cpu().numpy(), s.cache.page_size, []
    for b, n in enumerate(s.lens):
        slots += [-1 if (b, j) in skip else int(table[b, j // page]) * page + j % page for j in range(n)]
    moe.kv_append(s.cache, torch.cat(keys).cuda(), torch.cat(values).cuda(),
                  torch.tensor(slots, dtype=torch.int32, device="cuda"))
    s.k = [spec_ref.quantise(base.f64(x), s.cache.format)[3] for x in keys]
    s.v = [spec_ref.quantise(base.f64(x), s.cache.format)[3] for x in values]


# (format, head size, heads of a kv head, rows of a sequence): the warp kernel's instances, then the tensor-core kernel's
# with one M tile and with two
SHAPES = [(moe.MOE_KV_Q8, 64, 2, 3), (moe.MOE_KV_Q4, 64, 16, 4), (moe.MOE_KV_Q8, 128, 4, 1), (moe.MOE_KV_Q4, 128, 4, 8),
          (moe.MOE_KV_Q8, 256, 1, 3), (moe.MOE_KV_Q4, 128, 8, 12), (moe.MOE_KV_Q8, 128, 8, 40)]


@pytest.mark.parametrize("fmt,dim,group,rows", SHAPES)
@pytest.mark.parametrize("scale", [1.0 / 32, 1.0 / 128, -1.0 / 128, 1e-38])
def test_queries_of_subnormal_numbers(fmt, dim, group, rows, scale):
    """Scores that vanish against 1, times a scale that takes their multiplier below f32: the mean of the seen values,
    and masked tokens stay masked."""
    s = base.Sequences(fmt, dim, 2, group, 16, [300, 20, 0], [rows, rows, rows], 31, "any")
    s.scale = scale
    s.q = (torch.randint(-1, 2, s.q.shape, device="cuda").float() * 2.0 ** -133).bfloat16()
    s.check(s.run())


def check_winners(fmt, dim, group, rows, scale, size):
    """Queries along single dimensions, for each of which two tokens far apart have equal keys four times as large as
    all others: their mean comes back, however large the scores."""
    s = base.Sequences(fmt, dim, 2, group, 16, [700], [rows], 32, "any")
    rng = np.random.default_rng(dim)
    t = s.lens[0]
    k = rng.uniform(-2, 2, (t, 2, dim))
    first, second = rng.integers(0, 300, dim), rng.integers(400, 700, dim)
    k[first, :, np.arange(dim)] = 8.0
    k[second, :, np.arange(dim)] = 8.0
    k[:, :, ::32] = 8.0 * 15 / 16  # the groups' ends, so that both keys have the same scale (and minimum)
    k[:, :, 1::32] = -8.0
    k[:, :, 2::32] = 8.0
    v = rng.standard_normal((t, 2, dim)) + 0.25
    k, v = (torch.from_numpy(x.astype(np.float32)).bfloat16() for x in (k, v))
    refill(s, [k], [v])
    at = rng.choice([d for d in range(dim) if d % 32 > 2], s.q.shape[:2])
    q = torch.zeros(s.q.shape)
    q.scatter_(2, torch.from_numpy(at)[..., None], size if scale > 0 else -size)
    s.q, s.scale = q.bfloat16().cuda(), scale
    got = base.f64(s.run())
    for i in range(rows):
        for h in range(2 * group):
            d = at[i, h]
            pair = s.v[0][[first[d], second[d]], h // group]
            ref = pair.mean(0)
            # V rounded to f16 (2^-11 of each), one rounding to bf16, f32 sums
            bound = (2.0 ** -11 + 2.0 ** -14) * np.abs(pair).mean(0) + 2.0 ** -8 * np.abs(ref) + 1e-6
            assert (np.abs(got[i, h] - ref) <= bound).all(), (i, h, got[i, h, :4], ref[:4])


@pytest.mark.parametrize("fmt,dim,group,rows", SHAPES)
@pytest.mark.parametrize("scale,size", [(3e38, 1.0), (-3e38, 1.0), (0.09, 2.0 ** 127), (3e38, 2.0 ** 127)])
def test_scores_beyond_f32(fmt, dim, group, rows, scale, size):
    check_winners(fmt, dim, group, rows, scale, size)


@pytest.mark.parametrize("fmt,dim,group,rows", SHAPES)
@pytest.mark.parametrize("scale,size", [(1.0, 2.0 ** 16), (0.7, 2.0 ** 20), (1.0, 2.0 ** 24), (-0.7, 2.0 ** 27),
                                        (0.11, 2.0 ** 33), (1.0, 2.0 ** 60)])
def test_scores_of_many_digits(fmt, dim, group, rows, scale, size):
    """A score's multiple of log2(e) has more digits than f32 from some 2^24 on."""
    check_winners(fmt, dim, group, rows, scale, size)


@pytest.mark.parametrize("fmt,dim,group,rows", SHAPES)
def test_near_scores_of_many_digits(fmt, dim, group, rows):
    """Scores of some 2^26 that differ by 4, 8, ..: f32 holds them, and the weights are e^-4, e^-8, .. of the largest."""
    s = base.Sequences(fmt, dim, 2, group, 16, [700], [rows], 34, "any")
    rng = np.random.default_rng(dim)
    t = s.lens[0]
    k = np.zeros((t, 2, dim))
    k[:, :, ::32] = 15.0  # steps of 1 from 0 to 15
    k[:, :, 1::32] = rng.integers(0, 8, (t, 2, dim // 32))
    if fmt == moe.MOE_KV_Q8:
        k[:, :, ::32] = 127.0
    v = rng.standard_normal((t, 2, dim)) + 0.25
    k, v = (torch.from_numpy(x.astype(np.float32)).bfloat16() for x in (k, v))
    refill(s, [k], [v])
    assert np.array_equal(s.k[0], base.f64(k))  # held exactly
    q = torch.zeros(s.q.shape)
    q[:, :, 0] = 2.0 ** (22 if fmt == moe.MOE_KV_Q4 else 19)  # the large part of the score, the same for all
    q[:, :, 1] = 4.0
    s.q, s.scale = q.bfloat16().cuda(), 1.0
    got = base.f64(s.run())
    for i in range(rows):
        seen = [j for j in range(t) if j < 700 or s.masks[i] >> (j - 700) & 1]
        for h in range(2 * group):
            w = np.exp(4.0 * (s.k[0][seen, h // group, 1] - 7.0))
            w /= w.sum()
            ref, size = w @ s.v[0][seen, h // group], w @ np.abs(s.v[0][seen, h // group])
            # V and the weights rounded to f16 (2^-11 each), exponentials and sums in f32 (2^-14), one rounding to bf16
            assert (np.abs(got[i, h] - ref) <= (2.0 ** -10 + 2.0 ** -14) * size + 2.0 ** -8 * np.abs(ref) + 1e-6).all()


@pytest.mark.parametrize("fmt,dim,group,rows", [x for x in SHAPES if x[3] > 1])
@pytest.mark.parametrize("fill", [0xFF, 0x7B])
def test_slots_never_written_that_no_row_sees(fmt, dim, group, rows, fill):
    """Drafted tokens that were left out of the cache (slot -1) and that every mask leaves out: their bytes, scales of
    NaN or too large for f16, reach no row. One lies beside seen tokens, one at the end, one sequence sees none."""
    s = base.Sequences(fmt, dim, 2, group, 16, [300, 13, 0], [rows, rows, rows], 33, "any")
    rng = np.random.default_rng(rows)
    kv = [[torch.from_numpy(rng.standard_normal((t, 2, dim)).astype(np.float32)).bfloat16() for t in s.lens]
          for _ in range(2)]
    hidden = [{rows // 2, rows - 1}, {0}, set(range(rows))]
    s.masks = [m & ~sum(1 << j for j in hidden[i // rows]) for i, m in enumerate(s.masks)]
    s.mask = torch.tensor([m - (1 << 64) if m >> 63 else m for m in s.masks], dtype=torch.int64, device="cuda")
    refill(s, *kv, {(b, s.lens[b] - rows + j) for b in range(3) for j in hidden[b]}, fill)
    out = s.run()
    s.check(out)
    assert (out[2 * rows:] == 0).all()


@pytest.mark.parametrize("fmt,dim,group,rows", SHAPES)
def test_values_at_the_ends_of_the_range(fmt, dim, group, rows):
    """The largest scales (and minima) that the cache's writer makes: values up to 60000 of either sign or of both."""
    s = base.Sequences(fmt, dim, 2, group, 16, [300, 13], [rows, rows], 35, "any")
    rng = np.random.default_rng(rows)
    k = [torch.from_numpy(rng.standard_normal((t, 2, dim)).astype(np.float32)).bfloat16() for t in s.lens]
    v = []
    for t in s.lens:
        x = rng.uniform(-1, 1, (t, 2, dim)) * 6.2e4
        x[::3] = np.abs(x[::3])
        x[1::3] = -np.abs(x[1::3])
        x[::5] = np.sign(x[::5]) * 6.2e4
        v.append(torch.from_numpy(x.astype(np.float32)).bfloat16())
    refill(s, k, v)
    s.check(s.run())


def test_verify_of_no_rows():
    """A step in which no sequence has rows, and sequences without rows among others."""
    i32 = dict(dtype=torch.int32, device="cuda")
    for drafts in (True, False):
        n_acc, nxt = torch.full((3,), 9, **i32), torch.full((3,), 9, **i32)
        empty, ws = torch.empty(0, **i32), torch.empty(moe.spec_verify_workspace_bytes(3, 0), dtype=torch.uint8, device="cuda")
        moe.workspace_init(ws)
        draft = torch.empty((0, 100), device="cuda") if drafts else None
        moe.spec_verify(torch.empty((0, 100), device="cuda"), torch.zeros(4, **i32), empty, empty, draft, None,
                        torch.empty(0, device="cuda"), torch.ones((3, 100), device="cuda"), n_acc, empty, nxt, ws)
        assert moe.read_status(ws) == 0 and n_acc.tolist() == [0, 0, 0] and nxt.tolist() == [-1, -1, -1]
    case = verify_rows([0, 3, 0, 0, 5, 0], 333, "f32", "tree", True, 5)
    n_acc, path, nxt, status, _ = base.verify(case)
    alone = verify_rows([0, 3, 0, 0, 5, 0], 333, "f32", "tree", True, 5)
    for x in ("tokens", "parents", "u"):
        alone[x] = [alone[x][1], alone[x][4]]
    alone["temp"], alone["noise"] = [alone["temp"][1], alone["temp"][4]], alone["noise"][[1, 4]]
    want = base.verify(alone)
    assert status == 0 and [n_acc[1], n_acc[4]] == want[0] and path == want[1] and [nxt[1], nxt[4]] == want[2]
    assert [n_acc[b] for b in (0, 2, 3, 5)] == [0] * 4 and [nxt[b] for b in (0, 2, 3, 5)] == [-1] * 4


def test_one_host_tensor_among_device_ones_is_refused():
    s = base.Sequences(moe.MOE_KV_Q8, 64, 1, 2, 16, [5], [2], 36)
    ws, slots = s.workspace(), torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    good = dict(cache=s.cache, q=s.q, out=torch.empty_like(s.q), q_start=s.q_start, kv_len=s.kv_len, table=s.table,
                mask=s.mask, scale=s.scale, ws=ws)
    for name in ("q", "out", "q_start", "kv_len", "table", "mask", "ws"):
        with pytest.raises(ValueError, match=f"{name} must be on the GPU"):
            moe.tree_attention(**{**good, name: good[name].cpu()})
    moe.tree_attention(**good)
    for name, bad in (("k", (x.cpu(), x, slots)), ("v", (x, x.cpu(), slots)), ("slots", (x, x, slots.cpu()))):
        with pytest.raises(ValueError, match=f"{name} must be on the GPU"):
            moe.kv_append(s.cache, *bad)
    with pytest.raises(ValueError, match="status must be on the GPU"):
        moe.kv_append(s.cache, x, x, slots, torch.zeros(1, dtype=torch.int32))
    case = verify_rows([2], 100, "f32", "chain", True, 1)
    for name in ("logits", "draft"):
        with pytest.raises(ValueError, match=f"{name} must be on the GPU"):
            base.verify({**case, name: case[name].cpu()})


# ------------------------------------------------------------------ every part of a long item

LONG = [(4, 1), (8, 4), (8, 8), (8, 40)]  # heads of a kv head and rows over 40011 tokens: the join of some 300 and 150 parts


@pytest.mark.parametrize("fmt", base.FMTS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,rows", LONG)
def test_every_token_of_a_long_sequence_counts(fmt, dim, group, rows):
    """Equal weights, and a dimension for each stretch of tokens: one that lost (or counted twice) as few as 16 tokens
    would be off by 2 % or more."""
    s = base.Sequences(fmt, dim, 1, group, 128, [40011], [rows], rows, "chain")
    t = s.lens[0]
    stretch = min(-(-t // dim), 700)
    for first in range(0, t, stretch * dim):
        v = torch.zeros((t, 1, dim))
        part = torch.arange(first, min(t, first + stretch * dim))
        v[part, 0, (part - first) // stretch] = 1.0
        refill(s, [torch.zeros((t, 1, dim)).bfloat16()], [v.bfloat16()])
        got = base.f64(s.run())
        for i in range(rows):
            ref = s.v[0][:t - rows + i + 1, 0].mean(0)
            # V and the weights rounded to f16 (2^-11 each), sums in f32 (2^-14), one rounding to bf16
            bound = (2.0 ** -10 + 2.0 ** -14 + 2.0 ** -8) * np.abs(ref)
            assert (np.abs(got[i] - ref) <= bound).all(), (i, np.abs(got[i] - ref).max(), ref.max())
    assert 16 / stretch > 2 * (2.0 ** -10 + 2.0 ** -14 + 2.0 ** -8)  # what the test can see


@pytest.mark.parametrize("fmt", base.FMTS)
@pytest.mark.parametrize("dim,group,rows", [(128, 4, 1), (128, 8, 8), (128, 8, 40), (64, 16, 4), (256, 4, 3)])
def test_a_winning_token_anywhere_in_a_long_sequence(fmt, dim, group, rows):
    """Tokens whose keys are the queries' own random signs, beside and at the places where runs of 128 tokens (and tiles
    of the tensor-core kernel) meet: each query row gets its token's value back, in whichever part it lies."""
    s = base.Sequences(fmt, dim, 1, group, 128, [40011], [rows], rows, "chain")
    t, rng = s.lens[0], np.random.default_rng(rows)
    places = np.unique(np.concatenate([np.arange(0, 40011, 128), np.arange(127, 40011, 128), [40010]]))
    signs = rng.choice([-1.0, 1.0], (len(places), dim))
    k, v = rng.standard_normal((t, 1, dim)) * 0.1, rng.standard_normal((t, 1, dim)) + 0.25
    k[places, 0] = signs
    refill(s, *([torch.from_numpy(x.astype(np.float32)).bfloat16()] for x in (k, v)))
    s.scale = 1.0
    cross = signs @ signs.T - 2 * dim * np.eye(len(places))
    gain = 64.0 / (dim - cross.max())  # the next best token has a weight of e^-60 or less (of the quantised keys)
    ws = s.workspace()
    for first in range(0, len(places), rows * group):
        at = np.resize(np.arange(first, min(len(places), first + rows * group)), (rows, group))
        s.q = torch.from_numpy(signs[at] * gain).to(torch.bfloat16).cuda()
        got, ref = base.f64(s.run(ws)), s.v[0][places[at], 0]
        assert (np.abs(got - ref) <= (2.0 ** -11 + 2.0 ** -14 + 2.0 ** -8) * np.abs(ref) + 1e-6).all(), first


@pytest.mark.parametrize("fmt,dim,group,rows", SHAPES)
@pytest.mark.parametrize("scale,size", [(1.0, 2.0 ** 3), (0.7, 2.0 ** 5), (-1.0, 2.0 ** 7), (1.0, 2.0 ** 10)])
def test_scores_of_hundreds_and_thousands(fmt, dim, group, rows, scale, size):
    check_winners(fmt, dim, group, rows, scale, size)


# ------------------------------------------------------------------ the tensor-core kernel's own paths

# heads of 128: a row block of two M tiles, and of one
MANY = [(moe.MOE_KV_Q8, 8, 61), (moe.MOE_KV_Q4, 8, 61), (moe.MOE_KV_Q8, 4, 16), (moe.MOE_KV_Q4, 4, 16)]


@pytest.mark.parametrize("fmt,group,rows", MANY)
def test_many_rows_in_a_graph(fmt, group, rows):
    """A captured call follows the lengths, and gives the same bits each time."""
    s = base.Sequences(fmt, 128, 2, group, 32, [700, 90, 1500], [rows, rows - 3, rows], 41, "tree")
    ws, out = s.workspace(), torch.empty_like(s.q)
    want = s.run(ws).clone()
    s.check(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        moe.tree_attention(s.cache, s.q, out, s.q_start, s.kv_len, s.table, s.mask, s.scale, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    s.kv_len.copy_(torch.tensor([300, 80, 1001], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    assert torch.equal(got, s.run(ws)) and not torch.equal(got, want)


@pytest.mark.parametrize("fmt,group,rows", MANY)
def test_many_rows_one_of_them_nan(fmt, group, rows):
    """Within one run and across runs and groups: the row is NaN, the others keep their bits."""
    s = base.Sequences(fmt, 128, 2, group, 32, [50, 3000], [rows, rows], 42, "tree")
    want = s.run()
    at = [(1, 1), (rows - 1, 0), (rows, 2 * group - 1), (rows + rows // 2, 3)]
    for n, (i, h) in enumerate(at):
        s.q[i, h, 7 * n] = float("nan") if n % 2 else -float("inf")
    got = s.run()
    for i, h in at:
        assert torch.isnan(got[i, h]).all()
        got[i, h] = want[i, h]
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt,group,rows", MANY)
def test_many_rows_lengths_and_pages_outside(fmt, group, rows):
    s = base.Sequences(fmt, 128, 1, group, 16, [400, 20, 300], [rows] * 3, 43, "tree")
    want, ws = s.run(), s.workspace()

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
        assert torch.equal(out[:rows], want[:rows]) and torch.equal(out[2 * rows:], want[2 * rows:])
        assert (out[rows:2 * rows] == 0).all()
    s.kv_len.copy_(keep)
    # blocks of a tile that are not there: one, two in different tiles, the tile's first and last, a whole tile of eight
    for pages in ([0], [3, 17], [8, 15], list(range(8, 16)), [24]):
        old = s.table[0].clone()
        for n, p in enumerate(pages):
            s.table[0, p] = (-1, s.cache.n_pages, 1 << 30)[n % 3]
        st, out = status()
        s.table[0] = old
        assert st == moe.MOE_WS_INDEX and torch.equal(out[rows:], want[rows:])
        kept = [j for j in range(400 + rows) if j // 16 not in pages]  # pages of the context alone
        ref, bound = spec_ref.attention(base.f64(s.q[:rows]), s.k[0][kept], s.v[0][kept], rows, group, s.scale,
                                        s.masks[:rows])
        assert (np.abs(base.f64(out[:rows]) - ref) <= bound).all(), pages
    assert torch.equal(s.run(ws), want)


@pytest.mark.parametrize("fmt,group,rows", MANY)
def test_many_rows_masked_values_do_not_reach_a_row(fmt, group, rows):
    """A drafted token that no row sees, with a key and value as large as the cache holds; one that only a few see."""
    s = base.Sequences(fmt, 128, 1, group, 64, [137], [rows], 44, "any")
    s.masks = [m & ~(1 << 2) for m in s.masks]
    s.mask = torch.tensor([m - (1 << 64) if m >> 63 else m for m in s.masks], dtype=torch.int64, device="cuda")
    want = s.run()
    s.check(want)
    big = torch.full((1, 1, 128), 6.0e4, device="cuda").bfloat16()

    def put(node):
        j = 137 + node
        slot = int(s.table[0, j // 64]) * 64 + j % 64
        moe.kv_append(s.cache, big, -big, torch.tensor([slot], dtype=torch.int32, device="cuda"))

    put(2)
    assert torch.equal(s.run(), want)
    put(5)
    blind = [i for i in range(rows) if not s.masks[i] >> 5 & 1]
    assert blind and torch.equal(s.run()[blind], want[blind])


# ------------------------------------------------------------------ one sequence's verification

@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", ["chain", "tree"])
@pytest.mark.parametrize("drafts", [True, False])
@pytest.mark.parametrize("nodes,vocab", [(4, 32000), (8, 131072), (2, 2048), (12, 5003)])
def test_verify_one_sequence(kind, shape, drafts, nodes, vocab):
    """All rows of one sequence, over seeds in which drafts are accepted and rejected."""
    accepted = rejected = sure = 0
    for seed in range(8):
        case = verify_rows([nodes], vocab, kind, shape, drafts, seed, temps=(0.5 if seed % 2 else 1.0,))
        n_acc, path, nxt, status, _ = base.verify(case)
        want, last, margin = spec_ref.verify(
            base.f64(case["logits"]), case["tokens"][0], None if shape == "chain" else case["parents"][0],
            None if not drafts else case["draft"].cpu().numpy(), case["temp"][0],
            np.float32(case["u"][0]).astype(np.float64), np.float32(case["noise"][0]).astype(np.float64))
        assert status == 0
        if margin > base.MARGIN:
            sure += 1
            assert n_acc == [len(want)] and nxt == [last] and path == want + [-1] * (nodes - len(want)), seed
            accepted += len(want)
            rejected += len(want) < nodes - 1
    assert sure >= 7 and rejected > 0 and accepted > 0


@pytest.mark.parametrize("group,rows", [(2, 2), (8, 61)])
@pytest.mark.parametrize("length", [(1 << 31) - 1, (1 << 31) - 255])
def test_lengths_whose_tiles_would_pass_31_bits(group, rows, length):
    """In a table that has room for them: refused, the other sequences as ever. (As numbers of blocks and tiles
    they would be negative.)"""
    s = base.Sequences(moe.MOE_KV_Q8, 128, 1, group, 1024, [400, 20, 300], [rows] * 3, 45, "tree")
    ws = s.workspace()
    table = torch.zeros((3, 1 << 21), dtype=torch.int32, device="cuda")
    table[:, :s.table.shape[1]] = s.table
    s.kv_len[1] = length
    out = torch.full_like(s.q, 5.0)
    moe.tree_attention(s.cache, s.q, out, s.q_start, s.kv_len, table, s.mask, s.scale, ws)
    assert moe.read_status(ws) == moe.MOE_WS_INDEX
    s.check(out, {0, 2})  # (in other runs than beside a third sequence: other last bits)
    assert (out[rows:2 * rows] == 0).all()

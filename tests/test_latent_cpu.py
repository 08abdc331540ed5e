"""Rotary positions, latent attention and the care of pages without a GPU: tables, sizes, and
refusals made on the host before any device call."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import moe_decode_quantized_gb300 as moe
from moe_decode_quantized_gb300 import _lib

ADDR = 1 << 20  # stands for a device address: a refused call does not touch it
BF = torch.bfloat16


def _refused(rc, code, text):
    assert rc == code, (rc, _lib.moe().moe_last_error())
    assert text in _lib.moe().moe_last_error().decode(), _lib.moe().moe_last_error()


def test_rope_table_scalings():
    """Against the formulas; long positions keep their angle to 2^-30 of a turn."""
    dim, base, factor, original = 64, 500000.0, 8.0, 8192.0
    f = [base ** (-2 * i / dim) for i in range(dim // 2)]
    r = [original * x / (2 * math.pi) for x in f]
    keep = [min(max((x - 1) / 31, 0.0), 1.0) for x in r]
    want = {moe.MOE_ROPE_PLAIN: f, moe.MOE_ROPE_LINEAR: [x / factor for x in f],
            moe.MOE_ROPE_BASE: [(base * factor ** (dim / (dim - 2))) ** (-2 * i / dim) for i in range(dim // 2)],
            moe.MOE_ROPE_PARTS: [x * (k + (1 - k) / factor) for x, k in zip(f, keep)]}
    for scaling, w in want.items():
        t, magnitude = moe.rope_table(dim, base, scaling, factor, original)
        got = t.astype(np.float64) / 2.0 ** 64 * 2 * math.pi
        # a frequency's turn is rounded to a whole number of 2^-64: by 2^-65 of 2 pi radians at most, which of the smallest
        # here (3.8e-7) is 5e-13; the rest are roundings of 64-bit floats
        assert np.allclose(got, w, rtol=1e-13, atol=2 * math.pi * 2.0 ** -65)
        assert abs(magnitude - (0.1 * math.log(factor) + 1 if scaling == moe.MOE_ROPE_PARTS else 1.0)) < 1e-6


def test_rope_table_turns_exactly():
    """Pair 0 turns by one radian a position: 2^64 / 2 pi, to the last of the double's bits; the product with a position
    wraps as whole turns do."""
    t, _ = moe.rope_table(4)
    assert abs(int(t[0]) - 2935890503282001226) < 2 ** 11  # 2^64 / 2 pi (a double has 53 bits)
    p = 2 ** 31 - 1
    angle = (p * int(t[0]) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi
    assert abs(math.sin(angle) - math.sin(p)) < 1e-6


@pytest.mark.parametrize("kw,code,text", [
    (dict(dim=3), -1, "dim"), (dict(dim=0), -1, "dim"), (dict(dim=1026), -2, "dim"), (dict(scaling=4), -1, "scaling"),
    (dict(base=0.5), -1, "base"), (dict(base=float("nan")), -1, "base"),
    (dict(scaling=moe.MOE_ROPE_LINEAR, factor=0.5), -1, "factor"), (dict(dim=2, scaling=moe.MOE_ROPE_BASE, factor=2.0), -1, "dim 2"),
    (dict(scaling=moe.MOE_ROPE_PARTS, factor=2.0, slow=4.0, fast=4.0), -1, "slow"),
    (dict(scaling=moe.MOE_ROPE_PARTS, factor=2.0, original=0.0), -1, "original")])
def test_rope_table_refusals(kw, code, text):
    a = dict(dim=64)
    a.update(kw)
    with pytest.raises(moe.MoeError, match=text) as e:
        moe.rope_table(**a)
    assert e.value.code == code


def _rope(**kw):
    a = dict(x=ADDR, xt=1024, xh=128, out=ADDR + 4096, ot=1024, oh=128, kind=moe.MOE_BF16, tokens=4, heads=8, dim=128, offset=0,
             rope=128, layout=0, pos=ADDR, table=ADDR, magnitude=1.0, back=0)
    a.update(kw)
    return _lib.moe().moe_rope(a["x"], a["xt"], a["xh"], a["out"], a["ot"], a["oh"], a["kind"], a["tokens"], a["heads"], a["dim"],
                               a["offset"], a["rope"], a["layout"], a["pos"], a["table"], a["magnitude"], a["back"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(kind=2), -1, "type"), (dict(layout=2), -1, "layout"), (dict(tokens=-1), -1, "tokens"), (dict(heads=-1), -1, "heads"),
    (dict(rope=127), -1, "rope_dim"), (dict(rope=130), -1, "rope_dim"), (dict(rope=64, offset=66), -1, "offset"),
    (dict(offset=-2, rope=64), -1, "offset"), (dict(dim=1026, rope=64), -2, "head_dim"), (dict(heads=65537), -2, "heads"),
    (dict(magnitude=float("inf")), -1, "magnitude"), (dict(x=None), -1, "NULL"), (dict(table=None), -1, "NULL"),
    (dict(x=ADDR + 1), -1, "aligned"), (dict(kind=moe.MOE_F32, out=ADDR + 2), -1, "aligned"), (dict(table=ADDR + 4), -1, "aligned"),
    (dict(out=ADDR, ot=2048), -1, "in place")])
def test_rope_refusals(kw, code, text):
    _refused(_rope(**kw), code, text)


def test_rope_of_nothing():
    assert _rope(tokens=0, x=None) == 0 and _rope(heads=0, x=None) == 0


def _cache(**kw):
    c = _lib.MoeLatentCache(ADDR, 4, 512, 64, 64)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("latent,rope,page", [(512, 64, 64), (128, 8, 16), (256, 40, 1024)])
def test_latent_page_bytes(latent, rope, page):
    c = moe.LatentCache(None, latent, rope, page)
    assert moe.latent_page_bytes(c) == page * (latent + rope) * 2 and c.n_pages == 0
    c.pages = torch.empty((3, page, latent + rope), dtype=BF)
    assert c.n_pages == 3 and c.ref()._obj.n_pages == 3
    c.pages = torch.empty(3, dtype=BF)
    with pytest.raises(ValueError, match="not a multiple"):
        c.ref()


@pytest.mark.parametrize("field,value,code,text", [
    ("latent_dim", 192, -2, "latent_dim"), ("latent_dim", 0, -1, "latent_dim"), ("rope_dim", 0, -1, "rope_dim"),
    ("rope_dim", 72, -2, "rope_dim"), ("rope_dim", 12, -2, "rope_dim"), ("page_size", 24, -2, "page_size"),
    ("page_size", 2048, -2, "page_size"), ("pages", None, -1, "pages"), ("pages", ADDR + 8, -1, "16-byte"),
    ("n_pages", 0, -1, "n_pages"), ("n_pages", 1 << 26, -1, "n_pages")])
def test_latent_cache_refusals(field, value, code, text):
    L, c = _lib.moe(), _cache(**{field: value})
    _refused(L.moe_latent_append(C.byref(c), ADDR, 576, ADDR, 576, ADDR, 4, None, None, 0, 1.0, None, None), code, text)
    _refused(L.moe_latent_read(C.byref(c), ADDR, 4, ADDR, 512, ADDR, 64, None, None), code, text)
    _refused(_attend(c), code, text)


def test_latent_row_refusals():
    L, c = _lib.moe(), _cache()
    append = lambda *a: L.moe_latent_append(C.byref(c), *a)  # noqa: E731
    _refused(append(None, 576, ADDR, 576, ADDR, 4, None, None, 0, 1.0, None, None), -1, "NULL")
    _refused(append(ADDR, 576, ADDR, 576, None, 4, None, None, 0, 1.0, None, None), -1, "NULL")
    _refused(append(ADDR, 576, ADDR, 576, ADDR, -1, None, None, 0, 1.0, None, None), -1, "n_tokens")
    _refused(append(ADDR, 576, ADDR, 576, ADDR, 4, ADDR, None, 0, 1.0, None, None), -1, "together")
    _refused(append(ADDR, 576, ADDR, 576, ADDR, 4, ADDR, ADDR, 2, 1.0, None, None), -1, "layout")
    _refused(append(ADDR, 576, ADDR, 576, ADDR, 4, ADDR, ADDR, 0, float("nan"), None, None), -1, "magnitude")
    _refused(append(ADDR + 1, 576, ADDR, 576, ADDR, 4, None, None, 0, 1.0, None, None), -1, "aligned")
    assert append(None, 576, None, 576, None, 0, None, None, 0, 1.0, None, None) == 0
    read = lambda *a: L.moe_latent_read(C.byref(c), *a)  # noqa: E731
    _refused(read(ADDR, 4, ADDR, 511, ADDR, 64, None, None), -1, "stride")
    _refused(read(ADDR, 4, ADDR, 512, None, 64, None, None), -1, "NULL")
    assert read(None, 0, None, 512, None, 64, None, None) == 0


def _attend(c, **kw):
    a = dict(q=ADDR, qr=ADDR, out=ADDR, heads=16, q_start=ADDR, kv_len=ADDR, table=ADDR, stride=8, pages=8, mask=None, batch=1,
             tokens=1, scale=1.0, ws=ADDR, size=1 << 40)
    a.update(kw)
    return _lib.moe().moe_latent_attention(C.byref(c), a["q"], 8192, 512, a["qr"], 1024, 64, a["out"], 8192, 512, a["heads"],
                                           a["q_start"], a["kv_len"], a["table"], a["stride"], a["pages"], a["mask"], a["batch"],
                                           a["tokens"], a["scale"], a["ws"], a["size"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(heads=0), -1, "heads"), (dict(heads=129), -2, "heads"), (dict(batch=1025), -2, "batch"), (dict(tokens=65), -2, "n_tokens"),
    (dict(batch=-1), -1, "batch"), (dict(q=None), -1, "NULL"), (dict(qr=None), -1, "NULL"), (dict(ws=None), -1, "NULL"),
    (dict(ws=ADDR + 16), -1, "256"), (dict(size=8), -1, "workspace"), (dict(q=ADDR + 1), -1, "aligned"),
    (dict(mask=ADDR + 4), -1, "aligned"), (dict(pages=0), -1, "table_pages"), (dict(batch=2, stride=4), -1, "table_stride"),
    (dict(scale=float("nan")), -1, "scale"), (dict(scale=float("inf")), -1, "scale")])
def test_latent_attention_refusals(kw, code, text):
    _refused(_attend(_cache(), **kw), code, text)


def test_latent_attention_of_nothing():
    assert _attend(_cache(), batch=0, tokens=0, q=None, q_start=None) == 0
    assert _attend(_cache(), batch=3, tokens=0) == 0


def _prompt(**kw):
    a = dict(q=ADDR, k=ADDR, ks=4096, kr=ADDR, v=ADDR, out=ADDR, heads=16, nope=128, rope=64, q_start=ADDR, kv_start=ADDR, batch=2,
             n=8, t=8, scale=1.0, status=None)
    a.update(kw)
    return _lib.moe().moe_latent_prompt_attention(a["q"], 3200, 200, a["k"], a["ks"], 256, a["kr"], 64, a["v"], 4096, 256, a["out"],
                                                  2048, 128, a["heads"], a["nope"], a["rope"], a["q_start"], a["kv_start"],
                                                  a["batch"], a["n"], a["t"], 1, a["scale"], a["status"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(heads=0), -1, "heads"), (dict(heads=1025), -2, "heads"), (dict(nope=96), -2, "nope_dim"), (dict(rope=72), -2, "rope_dim"),
    (dict(rope=0), -1, "rope_dim"), (dict(batch=-1), -1, "batch"), (dict(batch=1025), -2, "batch"), (dict(t=-1), -1, "kv_tokens"),
    (dict(q=None), -1, "NULL"), (dict(k=None), -1, "NULL"), (dict(kv_start=None), -1, "NULL"), (dict(q=ADDR + 1), -1, "aligned"),
    (dict(v=ADDR + 8), -1, "16-byte"), (dict(ks=4100), -1, "multiples of 8"), (dict(status=ADDR + 2), -1, "aligned"),
    (dict(scale=float("nan")), -1, "scale")])
def test_prompt_refusals(kw, code, text):
    _refused(_prompt(**kw), code, text)


def test_prompt_of_nothing():
    assert _prompt(batch=0, q=None) == 0 and _prompt(n=0, q=None) == 0


def _pool(**kw):
    p = _lib.MoePagePool(ADDR, 100, 64)
    for k, v in kw.items():
        setattr(p, k, v)
    return C.byref(p)


def _calls(pool, table=ADDR, stride=8, pages=8, rows=4, arg=ADDR, n=2, cap=50, status=None):
    L = _lib.moe()
    return [L.moe_pages_grow(pool, table, stride, pages, rows, arg, status, None),
            L.moe_pages_fork(pool, table, stride, pages, rows, arg, arg, arg, n, arg, status, None),
            L.moe_pages_free(pool, table, stride, pages, rows, arg, n, status, None),
            L.moe_pages_compact(pool, table, stride, pages, rows, arg, arg, arg, cap, arg, status, None)]


@pytest.mark.parametrize("pool,kw,code", [
    (dict(refs=None), {}, -1), (dict(n_pages=0), {}, -1), (dict(n_pages=(1 << 24) + 1), {}, -2), (dict(page_size=0), {}, -1),
    ({}, dict(rows=-1), -1), ({}, dict(rows=1025), -2), ({}, dict(pages=0), -1), ({}, dict(stride=7), -1), ({}, dict(table=None), -1),
    ({}, dict(table=ADDR + 2), -1), ({}, dict(arg=None), -1), ({}, dict(arg=ADDR + 1), -1), ({}, dict(status=ADDR + 1), -1)])
def test_pages_refusals(pool, kw, code):
    assert _calls(_pool(**pool), **kw) == [code] * 4


def test_pages_counts_refused():
    assert _calls(_pool(), n=-1, rows=0, table=None)[1:3] == [-1, -1]
    assert _calls(_pool(), n=1025, rows=0, table=None)[1] == -2
    assert _calls(_pool(), cap=49, rows=0)[3] == -1
    assert _calls(_pool(), n=0, rows=0, table=None, arg=None)[:3] == [0, 0, 0]
    assert _lib.moe().moe_pages_grow(None, ADDR, 8, 8, 4, ADDR, None, None) == -1


def test_pages_copy_refusals():
    L = _lib.moe()

    def copy(pages=ADDR, stride=1 << 20, layers=2, n_pages=4, per=4096, copies=ADDR, n=2):
        return L.moe_pages_copy(pages, stride, layers, n_pages, per, copies, n, None, None, None)

    for kw in (dict(n=-1), dict(layers=-1), dict(n_pages=0), dict(per=0), dict(pages=None), dict(copies=None), dict(pages=ADDR + 8),
               dict(per=24), dict(stride=8), dict(stride=-16), dict(copies=ADDR + 2),
               dict(stride=4 * 4096 - 16), dict(stride=4096), dict(stride=0)):  # layers that overlap
        assert copy(**kw) == -1, kw
    assert copy(per=(1 << 32) + 16) == -2
    assert copy(n=0, pages=None) == 0 and copy(layers=0, pages=None) == 0


def test_the_binding_checks_what_it_is_given():
    z = lambda *s, t=BF: torch.zeros(s, dtype=t)  # noqa: E731
    i = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    table = z(32, t=torch.int64)
    for call, text in [
            (lambda: moe.rope(z(3, 2, 64, t=torch.float16), z(3, 2, 64, t=torch.float16), i(3), table), "x must be"),
            (lambda: moe.rope(z(3, 2, 64), z(3, 2, 63), i(3), table), "x and out"),
            (lambda: moe.rope(z(3, 2, 64), z(3, 2, 64, t=torch.float32), i(3), table), "out must be"),
            (lambda: moe.rope(z(3, 2, 64), z(3, 64, 2).transpose(1, 2), i(3), table), "contiguous"),
            (lambda: moe.rope(z(3, 2, 64), z(3, 2, 64), i(2), table), "positions holds"),
            (lambda: moe.rope(z(3, 2, 64), z(3, 2, 64), i(3), table.int()), "table must be"),
            (lambda: moe.rope(z(3, 2, 64), z(1, 2, 64).expand(3, 2, 64), i(3), table), "share memory"),
            (lambda: moe.rope(z(3, 2, 64), z(3, 2, 64), i(3), table), "on the GPU")]:
        with pytest.raises(ValueError, match=text):
            call() if "GPU" not in text else moe.rope(z(3, 2, 64), z(3, 2, 64), i(3), table, stream=0)
    c = moe.LatentCache(z(2, 16, 160), 128, 32, 16)
    for call, text in [
            (lambda: moe.latent_append(c, z(3, 128), z(2, 32), i(3), stream=0), "same number"),
            (lambda: moe.latent_append(c, z(3, 127), z(3, 32), i(3), stream=0), "c must be"),
            (lambda: moe.latent_append(c, z(3, 128), z(3, 32), i(2), stream=0), "slots holds"),
            (lambda: moe.latent_append(c, z(3, 128), z(3, 32), i(3), i(3), table, stream=0), "table must be int64 of 16"),
            (lambda: moe.latent_append(c, z(3, 128), z(3, 32), i(3), stream=0), "pages must be on the GPU"),
            (lambda: moe.latent_read(c, i(3), z(2, 128), z(3, 32), stream=0), "c_out must be"),
            (lambda: moe.latent_read(c, i(3), z(3, 128), z(1, 32).expand(3, 32), stream=0), "share memory"),
            (lambda: moe.latent_read(c, i(3), z(3, 128), z(3, 32), stream=0), "on the GPU")]:
        with pytest.raises(ValueError, match=text):
            call()
    q, qr, ws = z(3, 4, 128), z(3, 4, 32), z(512, t=torch.uint8)

    def attend(**kw):
        a = dict(q=q, q_rope=qr, out=q.clone(), q_start=i(2), kv_len=i(1), table=i(1, 2), mask=None, scale=1.0, ws=ws, stream=0)
        a.update(kw)
        moe.latent_attention(c, **a)

    for kw, text in [(dict(out=z(3, 4, 127)), "its shape"), (dict(q_rope=qr[:2]), "same number"), (dict(q_rope=z(3, 3, 32)), "q_rope must"),
                     (dict(mask=i(3)), "mask must be"), (dict(q_start=i(1)), "q_start holds"), (dict(table=i(2)), "table must be"),
                     (dict(ws=z(512, 2, t=torch.uint8)[:, 0]), "ws must be contiguous"), (dict(), "on the GPU")]:
        with pytest.raises(ValueError, match=text):
            attend(**kw)

    def prompt(**kw):
        a = dict(q=z(3, 4, 96), k=z(5, 4, 64), k_rope=z(5, 32), v=z(5, 4, 64), out=z(3, 4, 64), q_start=i(2), kv_start=i(2),
                 causal=True, scale=1.0, stream=0)
        a.update(kw)
        moe.latent_prompt_attention(**a)

    for kw, text in [(dict(q=z(3, 4, 95)), "q must be"), (dict(v=z(5, 4, 63)), "v k's shape"), (dict(k_rope=z(4, 32)), "same number"),
                     (dict(out=z(2, 4, 64)), "q's number"), (dict(kv_start=i(1)), "kv_start holds"), (dict(), "on the GPU")]:
        with pytest.raises(ValueError, match=text):
            prompt(**kw)
    pool, t = moe.PagePool(i(100), 16), torch.full((4, 8), -1, dtype=torch.int32)
    for call, text in [
            (lambda: moe.pages_grow(moe.PagePool(i(100).long(), 16), t, i(4), stream=0), "refs must be"),
            (lambda: moe.pages_grow(pool, t, i(3), stream=0), "lengths holds"),
            (lambda: moe.pages_grow(pool, t[0], i(4), stream=0), "table must be"),
            (lambda: moe.pages_grow(pool, t[:1].expand(4, 8), i(4), stream=0), "share memory"),
            (lambda: moe.pages_grow(pool, t, i(4), stream=0), "on the GPU"),
            (lambda: moe.pages_fork(pool, t, i(4), i(2), i(1), i(2, 2), stream=0), "target holds"),
            (lambda: moe.pages_fork(pool, t, i(4), i(2), i(2), i(3), stream=0), "copies holds"),
            (lambda: moe.pages_free(pool, t, i(2).long(), stream=0), "rows must be"),
            (lambda: moe.pages_compact(pool, t, i(99), t, i(50, 2), i(1), stream=0), "refs_out holds"),
            (lambda: moe.pages_compact(pool, t, i(100), t[:3], i(50, 2), i(1), stream=0), "table_out must have"),
            (lambda: moe.pages_copy(z(2, 4), i(2, 2), stream=0), "pages must be"),
            (lambda: moe.pages_copy(z(2, 4, 32)[:, :, ::2], i(2, 2), stream=0), "contiguous"),
            (lambda: moe.pages_copy(z(2, 4, 32), i(2, 2), stream=0), "on the GPU")]:
        with pytest.raises(ValueError, match=text):
            call()


def test_a_pool_looks_at_its_counts_at_each_call():
    """Other tensors at the address and of the size that were taken before: refused as they would be at first."""
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    counts, table = i(200), torch.full((4, 8), -1, dtype=torch.int32)
    pool = moe.PagePool(counts[:100], 16)
    for refs, text in [(counts[:100], "on the GPU"), (counts[::2], "refs must be contiguous"), (counts[:100], "on the GPU"),
                       (counts[:100].view(torch.float32), "refs must be int32"),
                       (counts.view(torch.int16)[:100], "refs must be int32"), (counts[:99], "on the GPU")]:
        pool.refs = refs
        for call in (lambda: moe.pages_grow(pool, table, i(4), stream=0), lambda: moe.pages_free(pool, table, i(2), stream=0)):
            with pytest.raises(ValueError, match=text):
                call()


def test_grow_refuses_tables_whose_entries_pass_31_bits():
    """Their sum over the rows is counted in 32 bits: a thousand rows of 2^21 entries asked for at once had got none."""
    L = _lib.moe()
    grow = lambda rows, pages: L.moe_pages_grow(_pool(), ADDR, 1 << 24, pages, rows, None, None, None)  # noqa: E731
    _refused(grow(1024, 1 << 21), -2, "2^31")
    _refused(grow(128, 1 << 24), -2, "2^31")
    _refused(grow(1024, (1 << 21) - 1), -1, "lengths")  # (the next check)


def test_lists_of_copies_that_pass_31_bits_are_refused():
    """A list's numbers are counted in 31 bits: of more than 2^30 pairs, those past them had been read and written before it."""
    L = _lib.moe()
    for n in (2 ** 30 + 1, 2 ** 31 - 1):
        _refused(L.moe_pages_copy(ADDR, 1 << 20, 2, 4, 4096, ADDR, n, None, None, None), -2, "2^30")
        _refused(L.moe_pages_compact(_pool(), ADDR, 8, 8, 4, ADDR, ADDR, ADDR, n, ADDR, None, None), -2, "2^30")
    _refused(L.moe_pages_copy(None, 1 << 20, 2, 4, 4096, ADDR, 2 ** 30, None, None, None), -1, "NULL")  # (the next check)

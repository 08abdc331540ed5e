"""The speculative-decoding entry points without a GPU: sizes, and refusals made on the
host before any device call."""
import ctypes as C

import numpy as np
import pytest
import torch

import moe_decode_quantized_gb300 as moe
from moe_decode_quantized_gb300 import _lib

import spec_ref

ADDR = 1 << 20  # stands for a device address: a refused call does not touch it


def _cache(**kw):
    c = _lib.MoeKvCache(ADDR, 4, 128, 8, 64, moe.MOE_KV_Q8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _refused(rc, code, text):
    assert rc == code, (rc, _lib.moe().moe_last_error())
    assert text in _lib.moe().moe_last_error().decode()


@pytest.mark.parametrize("fmt", [moe.MOE_KV_Q8, moe.MOE_KV_Q4])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_page_bytes(fmt, dim):
    pages = torch.empty(0, dtype=torch.uint8)
    c = moe.KvCache(pages, dim, 3, 48, fmt)
    assert moe.kv_page_bytes(c) == 3 * 3 * spec_ref.block_bytes(fmt, dim)
    assert spec_ref.block_bytes(fmt, dim) % 128 == 0
    big = moe.KvCache(torch.empty(5 * moe.kv_page_bytes(c), dtype=torch.uint8), dim, 3, 48, fmt)
    assert big.n_pages == 5
    with pytest.raises(ValueError, match="not a multiple"):
        moe.KvCache(torch.empty(moe.kv_page_bytes(c) + 1, dtype=torch.uint8), dim, 3, 48, fmt)


def test_pages_set_later_are_counted():
    c = moe.KvCache(None, 64, 2, 16)
    per = moe.kv_page_bytes(c)
    assert c.n_pages == 0
    for n in (5, 2):
        c.pages = torch.empty(n * per, dtype=torch.uint8)
        assert c.n_pages == n and c.ref()._obj.n_pages == n
    c.pages = torch.empty(per + 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="not a multiple"):
        c.ref()


@pytest.mark.parametrize("field,value,code,text", [
    ("head_dim", 96, -2, "head_dim"), ("head_dim", 0, -1, "head_dim"), ("n_kv_heads", 0, -1, "n_kv_heads"),
    ("n_kv_heads", 257, -2, "n_kv_heads"), ("page_size", 24, -2, "page_size"), ("page_size", 2048, -2, "page_size"),
    ("format", 2, -1, "format"), ("pages", None, -1, "pages"), ("pages", ADDR + 8, -1, "16-byte"),
    ("n_pages", 0, -1, "n_pages"), ("n_pages", 1 << 26, -1, "n_pages")])
def test_cache_refusals(field, value, code, text):
    L, c = _lib.moe(), _cache(**{field: value})
    _refused(L.moe_kv_append(C.byref(c), ADDR, 1024, 128, ADDR, 1024, 128, ADDR, 4, None, None), code, text)
    _refused(L.moe_kv_read(C.byref(c), ADDR, 4, ADDR, ADDR, moe.MOE_BF16, None, None), code, text)
    _refused(L.moe_tree_attention(C.byref(c), ADDR, 4096, 128, ADDR, 4096, 128, 32, ADDR, ADDR, ADDR, 8, 8, None, 1, 1,
                                  1.0, ADDR, 1 << 30, None), code, text)


def test_kv_argument_refusals():
    L, c = _lib.moe(), _cache()
    _refused(L.moe_kv_append(None, ADDR, 1, 1, ADDR, 1, 1, ADDR, 4, None, None), -1, "NULL")
    _refused(L.moe_kv_append(C.byref(c), None, 1, 1, ADDR, 1, 1, ADDR, 4, None, None), -1, "NULL")
    _refused(L.moe_kv_append(C.byref(c), ADDR, 1, 1, ADDR, 1, 1, None, 4, None, None), -1, "NULL")
    _refused(L.moe_kv_append(C.byref(c), ADDR + 1, 1, 1, ADDR, 1, 1, ADDR, 4, None, None), -1, "aligned")
    _refused(L.moe_kv_append(C.byref(c), ADDR, 1, 1, ADDR, 1, 1, ADDR, -1, None, None), -1, "n_tokens")
    _refused(L.moe_kv_read(C.byref(c), ADDR, 4, ADDR + 8, ADDR, moe.MOE_BF16, None, None), -1, "16-byte")
    _refused(L.moe_kv_read(C.byref(c), ADDR, 4, ADDR, ADDR, 7, None, None), -1, "out_type")
    assert L.moe_kv_append(C.byref(c), None, 1, 1, None, 1, 1, None, 0, None, None) == 0
    assert L.moe_kv_read(C.byref(c), None, 0, None, None, moe.MOE_F32, None, None) == 0


def _attend(c, **kw):
    a = dict(q=ADDR, out=ADDR, heads=32, q_start=ADDR, kv_len=ADDR, table=ADDR, stride=8, pages=8, mask=None, batch=1,
             tokens=1, scale=1.0, ws=ADDR, size=1 << 32)
    a.update(kw)
    return _lib.moe().moe_tree_attention(C.byref(c), a["q"], 4096, 128, a["out"], 4096, 128, a["heads"], a["q_start"],
                                         a["kv_len"], a["table"], a["stride"], a["pages"], a["mask"], a["batch"],
                                         a["tokens"], a["scale"], a["ws"], a["size"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(heads=12), -1, "multiple"), (dict(heads=0), -1, "multiple"), (dict(heads=8 * 65), -2, "n_q_heads"),
    (dict(batch=1025), -2, "batch"), (dict(tokens=65), -2, "n_tokens"), (dict(batch=-1), -1, "batch"),
    (dict(q=None), -1, "NULL"), (dict(ws=None), -1, "NULL"), (dict(ws=ADDR + 16), -1, "256"), (dict(size=8), -1, "workspace"),
    (dict(q=ADDR + 1), -1, "aligned"), (dict(mask=ADDR + 4), -1, "aligned"), (dict(pages=0), -1, "table_pages"),
    (dict(batch=2, stride=4), -1, "table_stride"), (dict(scale=float("nan")), -1, "scale"),
    (dict(scale=float("inf")), -1, "scale")])
def test_attention_refusals(kw, code, text):
    _refused(_attend(_cache(), **kw), code, text)


def test_attention_of_nothing():
    assert _attend(_cache(), batch=0, tokens=0, q=None, q_start=None) == 0
    assert _attend(_cache(), batch=3, tokens=0) == 0


def _verify(**kw):
    a = dict(logits=ADDR, kind=moe.MOE_BF16, stride=100, q_start=ADDR, tokens=ADDR, parents=None, draft=None, dstride=0,
             temp=None, u=ADDR, noise=ADDR, nstride=100, batch=2, rows=4, vocab=100, n=ADDR, path=ADDR, nxt=ADDR,
             ws=ADDR, size=1 << 32)
    a.update(kw)
    return _lib.moe().moe_spec_verify(a["logits"], a["kind"], a["stride"], a["q_start"], a["tokens"], a["parents"],
                                      a["draft"], a["dstride"], a["temp"], a["u"], a["noise"], a["nstride"], a["batch"],
                                      a["rows"], a["vocab"], a["n"], a["path"], a["nxt"], a["ws"], a["size"], None)


@pytest.mark.parametrize("kw,code,text", [
    (dict(kind=2), -1, "logits_type"), (dict(vocab=0), -1, "vocab"), (dict(vocab=(1 << 24) + 1), -2, "vocab"),
    (dict(batch=-1), -1, "bad"), (dict(batch=65536), -2, "batch"), (dict(logits=None), -1, "NULL"),
    (dict(path=None), -1, "NULL"), (dict(u=None), -1, "together"), (dict(noise=None), -1, "together"),
    (dict(logits=ADDR + 1), -1, "aligned"), (dict(kind=moe.MOE_F32, logits=ADDR + 2), -1, "aligned"),
    (dict(ws=ADDR + 64), -1, "256"), (dict(stride=99), -1, "stride"), (dict(draft=ADDR, dstride=99), -1, "stride"),
    (dict(nstride=99), -1, "stride"), (dict(size=0), -1, "workspace")])
def test_verify_refusals(kw, code, text):
    _refused(_verify(**kw), code, text)


def test_binding_checks_types_and_sizes():
    c = moe.KvCache(torch.zeros(moe.kv_page_bytes(moe.KvCache(None, 64, 2, 16)), dtype=torch.uint8), 64, 2, 16)
    k = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    s = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="slots"):
        moe.kv_append(c, k, k, s.long(), stream=0)
    with pytest.raises(ValueError, match="slots holds"):
        moe.kv_append(c, k, k, s[:2], stream=0)
    with pytest.raises(ValueError, match="k must be"):
        moe.kv_append(c, k.float(), k, s, stream=0)
    with pytest.raises(ValueError, match="v must be"):
        moe.kv_append(c, k, k[:, :1], s, stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        moe.kv_append(c, k.transpose(1, 2).contiguous().transpose(1, 2), k, s, stream=0)
    with pytest.raises(ValueError, match="same number"):
        moe.kv_append(c, k[:2], k, s, stream=0)
    with pytest.raises(ValueError, match="k_out holds"):
        moe.kv_read(c, s, k[:2], k, stream=0)
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="q_start holds"):
        moe.tree_attention(c, q, q, i, i, i[:, None], None, 1.0, ws, stream=0)
    with pytest.raises(ValueError, match="mask"):
        moe.tree_attention(c, q, q, s, i, i[:, None], s, 1.0, ws, stream=0)
    l = torch.zeros((3, 7), dtype=torch.float32)
    with pytest.raises(ValueError, match="noise must be"):
        moe.spec_verify(l, i, s, None, None, None, l[:, 0].contiguous(), l[:, :6], i[:1], s, i[:1], ws, stream=0)


def test_reference_quantiser_bound():
    """|x - value| <= d / 2 over many magnitudes, the ends included (what the rounding of the scale is for)."""
    rng = np.random.default_rng(5)
    x = spec_ref.bf16(rng.standard_normal((64, 256)) * 10.0 ** rng.uniform(-7, 4.5, (64, 1)))
    for fmt in (spec_ref.Q8, spec_ref.Q4):
        _, d, m, values = spec_ref.quantise(x, fmt)
        # a Q4 minimum rounded down can be below the smallest value, but no code is clipped
        err = np.abs(np.clip(x, -60000, 60000) - values).reshape(64, 8, 32).max(-1)
        assert (err <= d.astype(np.float64) / 2 * (1 + 1e-12)).all()
        assert (np.abs(values) < 65504).all()

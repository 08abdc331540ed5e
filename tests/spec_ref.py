"""Plain 64-bit implementations of the speculative-decoding operators (include/moe.h:
moe_kv_append, moe_kv_read, moe_tree_attention, moe_spec_verify), from their
definitions, in numpy. They share no code with the package."""
import math

import numpy as np

Q8, Q4 = 0, 1
LIMIT = 60000.0


def bf16(x):
    """float array rounded to bf16 (nearest even), as float64 (finite values)."""
    b = np.asarray(x, np.float32).view(np.uint32)
    return (((b + 0x7FFF + ((b >> 16) & 1)) >> 16) << 16).astype(np.uint32).view(np.float32).astype(np.float64)


def f16_towards(x, up):
    h = np.asarray(x, np.float64).astype(np.float16)
    step = np.nextafter(h, np.float16(np.inf if up else -np.inf))
    off = h.astype(np.float64) < x if up else h.astype(np.float64) > x
    return np.where(off, step, h)


def quantise(x, fmt):
    """rows [..., D] -> codes uint8 [..., D], d f16 [..., D / 32], m f16 or None, values float64 [..., D]."""
    g = np.clip(np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=LIMIT, neginf=-LIMIT), -LIMIT, LIMIT)
    shape = g.shape
    g = g.reshape(shape[:-1] + (shape[-1] // 32, 32))
    if fmt == Q8:
        d = f16_towards(np.abs(g).max(-1) / 127.0, True)
        f = d.astype(np.float64)[..., None]
        c = np.clip(np.rint(g / np.where(f > 0, f, 1.0)) * (f > 0), -127, 127)
        return (c + 128).astype(np.uint8).reshape(shape), d, None, (c * f).reshape(shape)
    m = f16_towards(g.min(-1), False)
    fm = m.astype(np.float64)[..., None]
    d = f16_towards((g - fm).max(-1) / 15.0, True)
    f = d.astype(np.float64)[..., None]
    c = np.clip(np.rint((g - fm) / np.where(f > 0, f, 1.0)) * (f > 0), 0, 15)
    return c.astype(np.uint8).reshape(shape), d, m, (c * f + fm).reshape(shape)


def row_bytes(fmt, dim):
    return dim if fmt == Q8 else dim // 2


def block_bytes(fmt, dim):
    return 2 * (16 * row_bytes(fmt, dim) + 16 * (dim // 32) * (2 if fmt == Q8 else 4))


def store_row(pool, fmt, heads, page_size, slot, head, value, codes, d, m):
    """Writes one quantised row (codes [D]) into a pool of bytes, by the documented places."""
    dim, rb, groups = codes.size, row_bytes(fmt, codes.size), codes.size // 32
    page, token = divmod(slot, page_size)
    base = ((page * heads + head) * (page_size // 16) + token // 16) * block_bytes(fmt, dim)
    base += block_bytes(fmt, dim) // 2 if value else 0
    t = token % 16
    if fmt == Q8:
        row = codes
    else:
        row = np.zeros(rb, np.uint8)
        for c in range(dim):
            bit = (c % 8) // 2 * 4 + (c % 2) * 16
            row[c // 8 * 4 + bit // 8] |= codes[c] << (bit % 8)
    for i in range(rb):
        if value:
            lane, x = i // (rb // 8) * 4 + t % 8 // 2, (t // 8 * 2 + t % 2) * (rb // 8) + i % (rb // 8)
        else:
            lane, x = t % 8 * 4 + i // (rb // 4), t // 8 * (rb // 4) + i % (rb // 4)
        pool[base + x // 16 * 512 + lane * 16 + x % 16] = row[i]
    words = pool[base + 16 * rb:base + 16 * rb + 16 * groups * (2 if fmt == Q8 else 4)].view(np.float16)
    for g in range(groups):
        if fmt == Q8:
            words[g * 16 + t if value else t * groups + g] = d[g]
        else:
            words[g * 16 + t if value else (t * groups + g) * 2] = d[g]
            words[(groups + g) * 16 + t if value else (t * groups + g) * 2 + 1] = m[g]


def attention(q, k, v, n, group, scale, masks):
    """One sequence: q [n, Hq, D], k, v [len, H, D] float64, masks: n ints or None ->
    out [n, Hq, D] and the bound of an evaluation in f16 operands (see below)."""
    length = k.shape[0]
    out, bound = np.zeros_like(q), np.zeros_like(q)
    for i in range(n):
        m = (2 << i) - 1 if masks is None else masks[i]
        seen = [j for j in range(length) if j < length - n or m >> (j - (length - n)) & 1]
        if not seen:
            continue
        for h in range(q.shape[1]):
            ks, vs = k[seen, h // group], v[seen, h // group]
            s = scale * (ks @ q[i, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h] = p @ vs
            # K and V rounded to f16 (2^-11 of each value at most): a score moves by at most e, a weight by a
            # factor of at most exp(2 e); the weights rounded to f16 and V's rounding add 2^-11 each; f32 sums and
            # exponentials 2^-14 in all; then one rounding to bf16
            e = 2.0 ** -11 * abs(scale) * (np.abs(ks) @ np.abs(q[i, h])).max()
            bound[i, h] = (math.expm1(2 * e) + 2.0 ** -10 + 2.0 ** -14) * (p @ np.abs(vs))
    return out, bound + 2.0 ** -8 * (np.abs(out) + bound) + 1e-7


def verify(logits, tokens, parents, draft, temp, u, noise):
    """One sequence: logits [n, V] -> (accepted nodes, next token, the smallest relative margin of a decision)."""
    n, vocab = logits.shape
    margin = [1.0]

    def probs(j):
        l = np.where(np.isnan(logits[j]) | (logits[j] == np.inf), -np.inf, logits[j]).astype(np.float64)
        if not np.isfinite(l).any():
            return np.zeros(vocab)
        if not temp > 0 or noise is None:
            return (np.arange(vocab) == l.argmax()).astype(np.float64)
        with np.errstate(over="ignore"):
            p = np.exp((l - l.max()) / temp)
        return p / p.sum()

    def closer(a, b):
        big = max(abs(a), abs(b))
        if big > 0:
            margin[0] = min(margin[0], abs(a - b) / big)

    cur, path = 0, []
    r, z = probs(0), 1.0
    for j in range(1, n):
        if (parents[j] if parents is not None else j - 1) != cur or not 0 <= tokens[j] < vocab:
            continue
        x = tokens[j]
        q = draft[j].astype(np.float64) if draft is not None else (np.arange(vocab) == x).astype(np.float64)
        lhs = (u[j] if u is not None else 0.5) * z * q[x]
        closer(lhs, r[x])
        if lhs < r[x]:
            cur, r, z = j, probs(j), 1.0
            path.append(j)
        else:
            r = np.maximum(r - z * q, 0.0)
            z = r.sum()
    p = probs(cur)
    if not p.any():
        return path, -1, margin[0]
    if not z > 0:
        r = p
    elif z < 1e-5:  # a residual made of rounding errors alone
        margin[0] = 0.0
    s = r / (noise if noise is not None and temp > 0 else np.ones(vocab))
    nxt = int(s.argmax())
    if vocab > 1 and noise is not None and temp > 0:
        top = np.partition(s, -2)[-2:]
        closer(top[0], top[1])
    return path, nxt, margin[0]

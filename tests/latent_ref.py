"""Plain 64-bit implementations of rotary positions, latent attention and the care of pages
(include/moe.h: moe_rope*, moe_latent_*, moe_pages_*), from their definitions. They share no
code with the package."""
import math

import torch

HALF, INTER = 0, 1
BF16 = 2.0 ** -8   # half a step of bf16, relative to the value
F32 = 2.0 ** -24


def turned(x, positions, table, layout, magnitude=1.0, transposed=False):
    """x float64 [tokens, heads, dims] with all dimensions turned; positions and table: lists of ints (the table's
    parts of a turn times 2^64), the angles by whole-number arithmetic."""
    pairs = x.shape[-1] // 2
    turns = torch.tensor([[(p * f % 2 ** 64) / 2.0 ** 64 for f in table] for p in positions], dtype=torch.float64)
    turns = turns.reshape(len(positions), 1, pairs)
    cos, sin = torch.cos(2 * math.pi * turns) * magnitude, torch.sin(2 * math.pi * turns) * magnitude
    sin = -sin if transposed else sin
    y = x.clone()
    a, b = (slice(0, pairs), slice(pairs, 2 * pairs)) if layout == HALF else (slice(0, None, 2), slice(1, None, 2))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def turned_bound(x, layout, magnitude, bf16):
    """How far moe_rope's result may be off: the angle in f32 (half of 2 pi 2^-24 at most, with the turn's 2^-33), sine
    and cosine to two units of 2^-24, the magnitude and two operations at 2^-24 each: 5e-7 of |m| (|a| + |b|); bf16: one
    rounding more."""
    pairs = x.shape[-1] // 2
    m = x.abs()
    both = m[..., :pairs] + m[..., pairs:] if layout == HALF else m[..., 0::2] + m[..., 1::2]
    both = torch.cat([both, both], -1) if layout == HALF else both.repeat_interleave(2, -1)
    bound = 5e-7 * abs(magnitude) * both
    return bound * (1 + BF16) + BF16 * abs(magnitude) * both if bf16 else bound


def attention(q, k, v, sees, scale):
    """q [n, heads, dims], k [t, heads or 1, dims], v [t, heads or 1, vdims] float64, sees bool [n, t] ->
    out [n, heads, vdims] and the bound of an evaluation with f32 sums and weights rounded to bf16 (see below).
    Tokens that a row does not see may hold anything."""
    n, heads, dims = q.shape
    out = torch.zeros((n, heads, v.shape[2]), dtype=torch.float64)
    bound = torch.zeros_like(out)
    for i in range(n):
        seen = sees[i].nonzero()[:, 0]
        if seen.numel() == 0:
            continue
        for h in range(heads):
            ks, vs = k[seen, h % k.shape[1]], v[seen, h % v.shape[1]]
            s = scale * (ks @ q[i, h])
            p = torch.exp(s - s.max())
            p /= p.sum()
            o = p @ vs
            out[i, h] = o
            # a score is a sum of `dims` f32 additions, each off by 2^-23 of what it has (cut off, not rounded, at worst):
            # by e, and a weight by a factor of exp(2 e); exponentials and their f32 arguments 2^-14 in all; the weights
            # are rounded to bf16 and add up to one as rounded, so that each moves the sum by 2^-8 of its token's distance
            # from it; sums of f32 2^-14; then one rounding to bf16
            e = dims * 2.0 ** -23 * abs(scale) * float((ks.abs() @ q[i, h].abs()).max())
            far = p @ (vs - o).abs()
            bound[i, h] = 1.01 * BF16 * far + (math.expm1(2 * e) + 2.0 ** -13) * (p @ vs.abs())
    return out, bound * (1 + BF16) + BF16 * out.abs() + 1e-30


class Pages:
    """The pool and table as plain lists."""

    def __init__(self, n_pages, page, rows, table_pages):
        self.refs, self.page = [0] * n_pages, page
        self.table = [[-1] * table_pages for _ in range(rows)]

    def lowest(self):
        return next((p for p, r in enumerate(self.refs) if r == 0), -1)

    def grow(self, lengths):
        short = False
        for row, n in zip(self.table, lengths):
            for j in range(-(-n // self.page)):
                if row[j] < 0:
                    p = self.lowest()
                    if p < 0:
                        short = True
                        continue
                    row[j] = p
                    self.refs[p] = 1
        return short

    def fork(self, lengths, pairs):
        copies, part = [], []
        for s, t in pairs:
            whole, src = lengths[s] // self.page, self.table[s]
            self.table[t] = [src[j] if j < whole else -1 for j in range(len(src))]
            for p in self.table[t][:whole]:
                self.refs[p] += 1
            part.append(lengths[s] % self.page != 0)
        for (s, t), more in zip(pairs, part):
            p = self.lowest() if more else -1
            if p >= 0:
                whole = lengths[s] // self.page
                self.table[t][whole] = p
                self.refs[p] = 1
                copies.append((self.table[s][whole], p))
            else:
                copies.append((-1, -1))
        return copies

    def free(self, rows):
        for r in rows:
            for j, p in enumerate(self.table[r]):
                if p >= 0:
                    self.refs[p] -= 1
                    self.table[r][j] = -1

    def compact(self):
        held = sum(r > 0 for r in self.refs)
        src = [p for p, r in enumerate(self.refs) if r > 0 and p >= held]
        dst = [p for p, r in enumerate(self.refs) if r == 0 and p < held]
        to = dict(zip(src, dst))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return list(zip(src, dst))

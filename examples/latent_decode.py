"""Prompts and parallel samples of a model with latent attention around the MoE layer step.

A small random model (embedding, two layers of latent attention and MoE, output head) takes a
few prompts and decodes several samples of each:

    pages_grow               pages for the prompts' tokens
    rope, latent_append      positions on the queries; latent vectors into the cache
    latent_prompt_attention  the prompts, in expanded form
    pages_fork, pages_copy   samples that share their prompt's full pages
    per step: pages_grow, rope, latent_append, latent_attention (absorbed form), layer_step
    pages_free, pages_compact, pages_copy   samples that end make room

Run: python examples/latent_decode.py [--tokens 24] [--samples 3]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_decode_quantized_gb300 as moe  # noqa: E402
from moe_decode_quantized_gb300.workload import Workload  # noqa: E402

ROWS = 8  # sequences of a step (the layer step's tokens)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """Embedding, layers of (latent attention, MoE), head; random weights, bf16 products by torch."""

    def __init__(self, n_layers=2, vocab=256, heads=4, nope=64, rope=16, latent=128, pages=64, page_size=16, seed=0):
        self.cfg = moe.Config(dim=256, inter=256, n_routed=16, topk=2, max_tokens=ROWS)
        self.n_layers, self.heads, self.nope, self.rope, self.latent = n_layers, heads, nope, rope, latent
        self.work = Workload(self.cfg, n_layers=n_layers, seed=seed, shared=True)
        g, dim = torch.Generator(device="cuda").manual_seed(seed), self.cfg.dim

        def rand(*shape, scale):
            return (torch.randn(shape, device="cuda", generator=g) * scale).bfloat16()

        self.embed, self.head = rand(vocab, dim, scale=1.0), rand(vocab, dim, scale=dim ** -0.5)
        layers = range(n_layers)
        self.wq = [rand(heads * (nope + rope), dim, scale=2 * dim ** -0.5) for _ in layers]
        self.wc = [rand(latent + rope, dim, scale=dim ** -0.5) for _ in layers]     # latent vector, turning part of the key
        self.uk = [rand(heads, nope, latent, scale=latent ** -0.5) for _ in layers]  # up-projections of keys and values
        self.uv = [rand(heads, nope, latent, scale=latent ** -0.5) for _ in layers]
        self.proj = [rand(dim, heads * nope, scale=0.5 * (heads * nope) ** -0.5) for _ in layers]
        table, self.magnitude = moe.rope_table(rope, scaling=moe.MOE_ROPE_PARTS, factor=4.0, original=64.0)
        self.turns = torch.from_numpy(table.view(np.int64)).cuda()
        self.scale = (nope + rope) ** -0.5
        # one pool and table serve the caches of all layers
        self.pages = torch.zeros((n_layers, pages, page_size, latent + rope), dtype=torch.bfloat16, device="cuda")
        self.caches = [moe.LatentCache(self.pages[layer], latent, rope, page_size) for layer in layers]
        self.pool = moe.PagePool(torch.zeros(pages, dtype=torch.int32, device="cuda"), page_size)
        self.table = torch.full((ROWS, pages // 2), -1, dtype=torch.int32, device="cuda")
        self.ws = torch.empty(moe.latent_attention_workspace_bytes(self.caches[0], heads, ROWS, ROWS), dtype=torch.uint8,
                              device="cuda")
        moe.workspace_init(self.ws)
        self.header = torch.zeros(moe.header_words(self.cfg, ROWS), dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def slots(self, rows, places):
        """Slots of places of the table's rows (int64 tensors)."""
        size = self.pool.page_size
        return (self.table[rows, places // size] * size + places % size).int()

    def project(self, layer, x, positions, slots):
        """Queries [tokens, heads, nope + rope], turned; latent vectors and keys' parts into the cache, and as written."""
        q = (x @ self.wq[layer].t()).view(-1, self.heads, self.nope + self.rope)
        moe.rope(q, q, positions, self.turns, offset=self.nope, layout=moe.MOE_ROPE_INTERLEAVED, magnitude=self.magnitude)
        c = x @ self.wc[layer].t()
        moe.latent_append(self.caches[layer], c[:, :self.latent], c[:, self.latent:], slots, positions, self.turns,
                          moe.MOE_ROPE_INTERLEAVED, self.magnitude, self.status)
        return q

    def experts(self, layer, residual):
        """The MoE layer of any number of rows, ROWS at a time."""
        for part in residual.split(ROWS):
            x = self.norm(part)
            moe.layer_step(self.cfg, self.work.layer(layer), self.work.arena, x, part, torch.empty_like(x), self.header,
                           part.shape[0], self.work.ws)

    def prompts(self, tokens):
        """Prompts (lists of tokens) into the table's first rows -> logits of each one's last token."""
        lens = [len(t) for t in tokens]
        starts = np.cumsum([0] + lens).tolist()
        moe.pages_grow(self.pool, self.table, i32(lens + [0] * (ROWS - len(lens))), self.status)
        rows = torch.tensor([b for b, n in enumerate(lens) for _ in range(n)], device="cuda")
        places = torch.tensor([j for n in lens for j in range(n)], device="cuda")
        slots, start = self.slots(rows, places), i32(starts)
        residual = self.embed[torch.tensor(sum(tokens, []), device="cuda")].float()
        for layer in range(self.n_layers):
            q = self.project(layer, self.norm(residual), places.int(), slots)
            c = torch.empty((places.numel(), self.latent), dtype=torch.bfloat16, device="cuda")
            kr = torch.empty((places.numel(), self.rope), dtype=torch.bfloat16, device="cuda")
            moe.latent_read(self.caches[layer], slots, c, kr, self.status)
            k, v = (torch.einsum("tl,hdl->thd", c, w) for w in (self.uk[layer], self.uv[layer]))
            out = torch.empty_like(k)
            moe.latent_prompt_attention(q, k, kr, v, out, start, start, True, self.scale, self.status)
            residual += (out.flatten(1) @ self.proj[layer].t()).float()
            self.experts(layer, residual)
        return (self.norm(residual[start[1:].long() - 1]) @ self.head.t()).float() * 4.0

    def step(self, rows, lens, tokens):
        """One token for each of the table's rows `rows` that hold `lens` tokens (lists) -> logits."""
        new = [0] * ROWS
        for r, n in zip(rows, lens):
            new[r] = n + 1
        moe.pages_grow(self.pool, self.table, i32(new), self.status)
        at, places = torch.tensor(rows, device="cuda"), torch.tensor(lens, device="cuda")
        slots, table = self.slots(at, places), self.table[at].contiguous()
        start, kv_len = torch.arange(len(rows) + 1, dtype=torch.int32, device="cuda"), (places + 1).int()
        residual = self.embed[torch.tensor(tokens, device="cuda")].float()
        for layer in range(self.n_layers):
            q = self.project(layer, self.norm(residual), places.int(), slots)
            folded = torch.einsum("nhd,hdl->nhl", q[..., :self.nope], self.uk[layer])
            out = torch.empty_like(folded)
            moe.latent_attention(self.caches[layer], folded, q[..., self.nope:], out, start, kv_len, table, None, self.scale,
                                 self.ws)
            values = torch.einsum("nhl,hdl->nhd", out, self.uv[layer])
            residual += (values.flatten(1) @ self.proj[layer].t()).float()
            self.experts(layer, residual)
        return (self.norm(residual) @ self.head.t()).float() * 4.0

    def fork(self, pairs, lens):
        """Rows of the table as forks of others: (source, target) pairs; lens: tokens of all rows."""
        copies = torch.empty((len(pairs), 2), dtype=torch.int32, device="cuda")
        moe.pages_fork(self.pool, self.table, i32(lens), i32([s for s, _ in pairs]), i32([t for _, t in pairs]), copies,
                       self.status)
        moe.pages_copy(self.pages, copies, status=self.status)

    def compact(self):
        """The pages held to the pool's front."""
        pages = self.pages.shape[1]
        copies, count = torch.empty((pages // 2, 2), dtype=torch.int32, device="cuda"), i32([0])
        moe.pages_compact(self.pool, self.table, self.pool.refs, self.table, copies, count, self.status)
        moe.pages_copy(self.pages, copies, count, self.status)


def generate(model, prompts, samples, count, seed=1, ends=(2, 5)):
    """`samples` continuations of `count` tokens of each prompt -> (lists of tokens, one a sample). After `ends[0]` steps the
    prompts' own rows are given up, after `ends[1]` the pool is compacted."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = model.prompts(prompts)
    n = len(prompts)
    rows = list(range(n, n + n * samples))
    source = [i // samples for i in range(n * samples)]
    lens = [len(p) for p in prompts]
    model.fork(list(zip(source, rows)), lens + [0] * (ROWS - n))
    held, logits = [lens[s] for s in source], logits[torch.tensor(source, device="cuda")]
    out = [[] for _ in rows]
    for step in range(count):
        noise = torch.empty_like(logits).exponential_(generator=g)
        tokens = (torch.softmax(logits, -1) / noise).argmax(-1).tolist()
        for o, t in zip(out, tokens):
            o.append(t)
        if step == ends[0]:
            moe.pages_free(model.pool, model.table, i32(list(range(n))), model.status)
        if step == ends[1]:
            model.compact()
        if step + 1 < count:
            logits = model.step(rows, held, tokens)
            held = [h + 1 for h in held]
    assert moe.read_status(model.ws) == 0 and moe.read_status(model.work.ws) == 0 and model.status.item() == 0
    return out


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=24)
    ap.add_argument("--samples", type=int, default=3, choices=[1, 2, 3])
    a = ap.parse_args()
    model = Model()
    out = generate(model, [[3, 1, 4, 1, 5, 9, 2, 6] * 5, [2, 7, 1, 8]], a.samples, a.tokens)
    for o in out:
        print(o)
    print(f"pages held: {int((model.pool.refs > 0).sum())} of {model.pool.refs.numel()}")


if __name__ == "__main__":
    main()

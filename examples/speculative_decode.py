"""Speculative decoding with a tree of drafted tokens around the MoE layer step.

A small random model (embedding, two layers of attention and MoE, output head)
decodes one sequence. Each round takes the last token and up to seven drafted
ones (a tree: the likeliest followers, and theirs) through the layers at once:

    kv_append        the rows' keys and values into the quantised cache
    tree_attention   every row over the context and its own ancestors
    layer_step       the MoE layer of all rows (m = 8)
    spec_verify      which drafted nodes the target accepts, and the next token
    kv_append        the accepted rows to the places that follow the context

Run: python examples/speculative_decode.py [--tokens 64] [--temperature 0.7]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_decode_quantized_gb300 as moe  # noqa: E402
from moe_decode_quantized_gb300.workload import Workload  # noqa: E402

# rows of a round: the last token, three followers, two followers of each of the first two
PARENTS = [-1, 0, 0, 0, 1, 1, 2, 2]
ROWS = len(PARENTS)


def ancestor_masks(parents):
    masks = []
    for j, p in enumerate(parents):
        masks.append((masks[p] if j else 0) | 1 << j)
    return masks


class Model:
    """Embedding, layers of (attention, MoE), head; random weights, bf16 products by torch."""

    def __init__(self, n_layers=2, vocab=512, heads=4, kv_heads=2, head_dim=64, seed=0, pages=64, page_size=16,
                 kv_format=moe.MOE_KV_Q8):
        self.cfg = moe.Config(dim=256, inter=256, n_routed=16, topk=2, max_tokens=ROWS)
        self.n_layers, self.vocab, self.heads, self.kv_heads, self.head_dim = n_layers, vocab, heads, kv_heads, head_dim
        self.page_size = page_size
        self.work = Workload(self.cfg, n_layers=n_layers, seed=seed, shared=True)
        g = torch.Generator(device="cuda").manual_seed(seed)
        dim, width = self.cfg.dim, (heads + 2 * kv_heads) * head_dim

        def rand(*shape, scale):
            return (torch.randn(shape, device="cuda", generator=g) * scale).bfloat16()

        self.embed = rand(vocab, dim, scale=1.0)
        self.head = rand(vocab, dim, scale=dim ** -0.5)
        self.follow = rand(dim, dim, scale=dim ** -0.5)  # what makes a token's followers: kept large, so that drafts agree
        self.qkv = [rand(width, dim, scale=dim ** -0.5) for _ in range(n_layers)]
        self.proj = [rand(dim, heads * head_dim, scale=0.3 * (heads * head_dim) ** -0.5) for _ in range(n_layers)]
        self.caches = []
        for _ in range(n_layers):
            c = moe.KvCache(None, head_dim, kv_heads, page_size, kv_format)
            c = moe.KvCache(torch.zeros(pages * moe.kv_page_bytes(c), dtype=torch.uint8, device="cuda"), head_dim,
                            kv_heads, page_size, kv_format)
            self.caches.append(c)
        self.table = torch.randperm(pages, device="cuda", generator=g).int()[None]  # the sequence's pages, in any order
        self.attn_ws = torch.empty(moe.tree_attention_workspace_bytes(self.caches[0], heads, 1, ROWS), dtype=torch.uint8,
                                   device="cuda")
        self.spec_ws = torch.empty(moe.spec_verify_workspace_bytes(1, ROWS), dtype=torch.uint8, device="cuda")
        for ws in (self.attn_ws, self.spec_ws):
            moe.workspace_init(ws)
        self.header = torch.zeros(moe.header_words(self.cfg, ROWS), dtype=torch.int32, device="cuda")
        self.kv = [None] * n_layers  # the last round's key and value rows

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def slots(self, places):
        """Slots of places (int32 tensor) of the sequence."""
        return self.table[0][places.long() // self.page_size] * self.page_size + places % self.page_size

    def start(self, tokens):
        """Residual of tokens [m]: each token's embedding and what tends to follow it."""
        e = self.embed[tokens.long()]
        return e.float() * 0.2 + (e @ self.follow.t()).float()

    def rows(self, tokens, context, masks):
        """Logits [m, vocab] of m rows behind `context` tokens; masks: int64 [m] or None (a chain)."""
        m = tokens.numel()
        residual = self.start(tokens)
        places = context + torch.arange(m, dtype=torch.int32, device="cuda")
        slots = self.slots(places).int()
        q_start = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        kv_len = torch.tensor([context + m], dtype=torch.int32, device="cuda")
        for layer in range(self.n_layers):
            qkv = (self.norm(residual) @ self.qkv[layer].t()).view(m, -1, self.head_dim)
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
            self.kv[layer] = (k, v)
            moe.kv_append(self.caches[layer], k, v, slots)
            out = torch.empty((m, self.heads, self.head_dim), dtype=torch.bfloat16, device="cuda")
            moe.tree_attention(self.caches[layer], q, out, q_start, kv_len, self.table, masks, self.head_dim ** -0.5,
                               self.attn_ws)
            residual += (out.view(m, -1) @ self.proj[layer].t()).float()
            x = self.norm(residual)
            moe.layer_step(self.cfg, self.work.layer(layer), self.work.arena, x, residual, torch.empty_like(x),
                           self.header, m, self.work.ws)
        return (self.norm(residual) @ self.head.t()).float() * 4.0

    def keep(self, context, path):
        """The accepted rows (int list) to the places after the last token's."""
        if path != list(range(1, len(path) + 1)):  # else they are there
            rows = torch.tensor(path, device="cuda")
            slots = self.slots(context + 1 + torch.arange(len(path), dtype=torch.int32, device="cuda")).int()
            for cache, (k, v) in zip(self.caches, self.kv):
                moe.kv_append(cache, k[rows], v[rows], slots)

    def draft(self, token):
        """Tokens of a round from the embedding alone (a model without layers)."""
        def likely(t, n):
            return (self.norm(self.start(t)) @ self.head.t()).float().topk(n, -1).indices.int()

        first = likely(token.view(1), 3)[0]
        second = likely(first[:2], 2).flatten()
        return torch.cat([token.view(1), first, second])


def generate(model, prompt, count, temperature=0.0, seed=1):
    """-> (tokens, rounds): at least `count` tokens after the prompt."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    parents = torch.tensor(PARENTS, dtype=torch.int32, device="cuda")
    masks = torch.tensor(ancestor_masks(PARENTS), dtype=torch.int64, device="cuda")
    q_start = torch.tensor([0, ROWS], dtype=torch.int32, device="cuda")
    temp = torch.full((1,), float(temperature), device="cuda")
    n_acc, nxt = (torch.empty(1, dtype=torch.int32, device="cuda") for _ in range(2))
    path = torch.empty(ROWS, dtype=torch.int32, device="cuda")
    for i in range(0, len(prompt) - 1, ROWS):  # the prompt but its last token, in chains of up to ROWS
        model.rows(torch.tensor(prompt[:-1][i:i + ROWS], dtype=torch.int32, device="cuda"), i, None)
    context, last, out, rounds = len(prompt) - 1, prompt[-1], [], 0
    while len(out) < count:
        tokens = model.draft(torch.tensor([last], dtype=torch.int32, device="cuda"))
        logits = model.rows(tokens, context, masks)
        u = torch.rand(ROWS, device="cuda", generator=g)
        noise = torch.empty((1, model.vocab), device="cuda").exponential_(generator=g)
        moe.spec_verify(logits, q_start, tokens, parents, None, temp, u, noise, n_acc, path, nxt, model.spec_ws)
        taken = path[:int(n_acc)].tolist()
        model.keep(context, taken)
        out += [int(tokens[j]) for j in taken] + [int(nxt)]
        context += 1 + len(taken)
        last = out[-1]
        rounds += 1
    assert moe.read_status(model.attn_ws) == 0 and moe.read_status(model.spec_ws) == 0
    assert moe.read_status(model.work.ws) == 0
    return out, rounds


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--temperature", type=float, default=0.7)
    a = ap.parse_args()
    model = Model()
    out, rounds = generate(model, [3, 1, 4, 1, 5], a.tokens, a.temperature)
    print(f"{len(out)} tokens in {rounds} rounds: {len(out) / rounds:.2f} a round")
    print(out)


if __name__ == "__main__":
    main()

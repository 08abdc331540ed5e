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

"""What the binding of the speculative-decoding calls checks before it hands addresses to the
library, without a GPU."""
import pytest
import torch

import moe_decode_quantized_gb300 as moe


def _cache(pages=3):
    c = moe.KvCache(None, 64, 2, 16)
    c.pages = torch.zeros(pages * moe.kv_page_bytes(c), dtype=torch.uint8)
    return c


def test_pages_that_get_other_memory_are_followed():
    """A pages tensor resized, or given another storage, in place: its address and count as of each call."""
    c = _cache()
    per = moe.kv_page_bytes(c)
    for change in (lambda t: t.resize_(500 * per), lambda t: t.set_(torch.zeros(7 * per, dtype=torch.uint8)),
                   lambda t: setattr(t, "data", torch.zeros(2 * per, dtype=torch.uint8))):
        c.ref()
        change(c.pages)
        assert c.ref()._obj.pages == c.pages.data_ptr() and c.ref()._obj.n_pages == c.pages.numel() // per
    c.pages.resize_(per + 1)
    with pytest.raises(ValueError, match="not a multiple"):
        c.ref()


def test_host_tensors_are_refused():
    """In calls that are right but for where their tensors are. (Without the refusal these would launch nothing here:
    there is no device.)"""
    c, i32 = _cache(), dict(dtype=torch.int32)
    k, s = torch.zeros((3, 2, 64), dtype=torch.bfloat16), torch.zeros(3, **i32)
    with pytest.raises(ValueError, match="pages must be on the GPU"):
        moe.kv_append(c, k, k, s, stream=0)
    with pytest.raises(ValueError, match="pages must be on the GPU"):
        moe.kv_read(c, s, k.clone(), k.clone(), stream=0)
    q, ws = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="on the GPU"):
        moe.tree_attention(c, q, q.clone(), torch.tensor([0, 3], **i32), s[:1], torch.zeros((1, 2), **i32), None, 1.0, ws,
                           stream=0)
    l = torch.zeros((3, 7))
    with pytest.raises(ValueError, match="logits must be on the GPU"):
        moe.spec_verify(l, torch.tensor([0, 3], **i32), s, None, None, None, l[:, 0].contiguous(), l[:1], s[:1].clone(),
                        s.clone(), s[:1].clone(), ws, stream=0)


def test_a_strided_workspace_is_refused():
    """Its bytes are fewer than those between its first and last: the kernels would write past it or into others'."""
    c, i32 = _cache(), dict(dtype=torch.int32)
    q, ws, s = torch.zeros((3, 4, 64), dtype=torch.bfloat16), torch.zeros((256, 2), dtype=torch.uint8)[:, 0], torch.zeros(3, **i32)
    with pytest.raises(ValueError, match="ws must be contiguous"):
        moe.tree_attention(c, q, q.clone(), torch.tensor([0, 3], **i32), s[:1], torch.zeros((1, 2), **i32), None, 1.0, ws,
                           stream=0)
    l = torch.zeros((3, 7))
    with pytest.raises(ValueError, match="ws must be contiguous"):
        moe.spec_verify(l, torch.tensor([0, 3], **i32), s, None, None, None, l[:, 0].contiguous(), l[:1], s[:1].clone(),
                        s.clone(), s[:1].clone(), ws, stream=0)

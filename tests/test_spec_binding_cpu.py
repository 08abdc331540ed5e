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

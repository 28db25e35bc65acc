"""The extension module of the serving calls: what it refuses before it looks
at any memory (host tensors without elements, nothing is launched)."""

import pytest
import torch

import learned_token_pruning_score_b200 as tg

BIG = 2 ** 32  # what 32 bits would cut to nothing


def test_sizes_beyond_32_bits_are_refused():
    """A size is refused, not cut: 2^32 + 16 columns are not 16."""
    e = lambda *s: torch.empty(*s, dtype=torch.int8)  # noqa: E731
    one = torch.empty(0)
    with pytest.raises(ValueError, match="columns 4294967312 is above"):
        tg.tg_quantize_rows(torch.empty(0, BIG + 16))
    with pytest.raises(ValueError, match="k 4294967312 is above"):
        tg.tg_linear_quantized(e(0, BIG + 16), one, e(0, BIG + 16), one)
    with pytest.raises(ValueError, match="n 4294967328 is above"):
        tg.tg_linear_quantized(e(4, 0), one, e(BIG + 32, 0), one)
    kv = torch.empty(0, 16, 2, 64)
    for k, table in ((kv, torch.empty(0, BIG + 1, dtype=torch.int32)),
                     (kv, torch.empty(BIG + 1, 0, dtype=torch.int32)),
                     (torch.empty(0, 16, BIG + 2, 64), torch.empty(1, 1, dtype=torch.int32)),
                     (torch.empty(0, BIG + 16, 2, 64), torch.empty(1, 1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="below 2\\^31"):
            tg.PagedKV(k, k, table)


def test_a_cache_keeps_to_its_tensors():
    """A table that has grown is another cache: the calls would go on with the
    old one's memory. The handle that they get keeps that memory."""
    k, table = torch.zeros(4, 16, 2, 64), torch.zeros(2, 2, dtype=torch.int32)
    v, bias = torch.zeros_like(k), torch.zeros(4, 16)
    held = [t._use_count() for t in (k, v, table, bias)]
    c = tg.PagedKV(k, v, table, bias)
    for name in ("k", "v", "table", "bias", "capacity", "page_size", "batch", "c"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))
    assert c.table is table and c.capacity == 32 and c.bias is bias
    handle = c._h
    del c
    assert [t._use_count() for t in (k, v, table, bias)] == [n + 1 for n in held]
    del handle
    assert [t._use_count() for t in (k, v, table, bias)] == held

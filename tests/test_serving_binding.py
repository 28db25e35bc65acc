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


def test_the_module_is_rebuilt_for_another_torch(monkeypatch, tmp_path):
    """What the module's binary interface comes from is part of the check that
    finds it up to date."""
    from learned_token_pruning_score_b200 import _build

    runs = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    monkeypatch.setattr(_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(_build, "_newer", lambda *a: False)
    monkeypatch.setattr(_build.subprocess, "run", lambda cmd, **kw: runs.append(cmd) or Done())
    _build.build_binding()
    assert len(runs) == 1  # no stamp
    _build.build_binding()
    assert len(runs) == 1  # up to date
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    _build.build_binding()
    _build.build_binding()
    assert len(runs) == 2
    monkeypatch.setattr(_build, "CXX_FLAGS", [*_build.CXX_FLAGS, "-g"])
    _build.build_binding()
    _build.build_binding(force=True)
    assert len(runs) == 4

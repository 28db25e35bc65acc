"""Refusals of the calls that serve from a paged cache and of the 8-bit
projections: host-side validation, before anything is launched (no GPU)."""

import ctypes

import pytest
import torch

import learned_token_pruning_score_b200 as tg

P = ctypes.c_void_p(4096)       # never dereferenced
ODD = ctypes.c_void_p(4096 + 4)


def _cache(**kw):
    f = dict(k=4096, v=8192, bias=None, table=4096, n_pages=4, k_page_stride=64 * 8 * 128,
             v_page_stride=64 * 8 * 128, bias_page_stride=64, table_stride=4, page_size=64,
             n_heads_kv=8, head_dim=128, dtype=tg.TG_BF16)
    f.update(kw)
    return tg.TgPagedKv(*[f[n] for n, _ in tg.TgPagedKv._fields_])


def _append(c, q=P, qs=4096, k=P, ks=4096, v=P, vs=4096, rows=5, cu=P, ln=P, batch=2, hq=16,
            qn=None, eps=1e-6, base=1e6, q_out=P):
    return tg._paged_append(ctypes.byref(c) if c is not None else None, q, qs, k, ks, v, vs, rows,
                            cu, ln, batch, hq, None, None, qn, None, eps, base, q_out, None)


def _attn(c, q=P, qs=2048, rows=5, cu=P, ln=P, batch=2, hq=16, max_kv=256, out=P, lse=None,
          ws=P, ws_bytes=1 << 40):
    return tg._paged_attn(ctypes.byref(c) if c is not None else None, q, qs, rows, cu, ln, batch,
                          hq, max_kv, None, None, out, lse, ws, ws_bytes, None)


BAD_CACHES = [
    (dict(dtype=5), tg.TG_ERR_UNSUPPORTED),
    (dict(head_dim=96), tg.TG_ERR_UNSUPPORTED),
    (dict(page_size=48), tg.TG_ERR_UNSUPPORTED),
    (dict(page_size=8), tg.TG_ERR_UNSUPPORTED),
    (dict(page_size=512), tg.TG_ERR_UNSUPPORTED),
    (dict(k=None), tg.TG_ERR_INVALID_ARG),
    (dict(v=8192 + 2), tg.TG_ERR_INVALID_ARG),
    (dict(table=None), tg.TG_ERR_INVALID_ARG),
    (dict(n_pages=0), tg.TG_ERR_INVALID_ARG),
    (dict(table_stride=0), tg.TG_ERR_INVALID_ARG),
    (dict(n_heads_kv=0), tg.TG_ERR_INVALID_ARG),
    (dict(k_page_stride=64 * 8 * 128 - 8), tg.TG_ERR_INVALID_ARG),
    (dict(v_page_stride=64 * 8 * 128 + 4), tg.TG_ERR_INVALID_ARG),
    (dict(bias=4096, bias_page_stride=63), tg.TG_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("bad,want", BAD_CACHES)
def test_bad_caches_are_refused(bad, want):
    assert _append(_cache(**bad)) == want
    assert _attn(_cache(**bad)) == want


def test_append_refusals():
    ok = _cache()
    assert _append(None) == tg.TG_ERR_INVALID_ARG
    for kw in (dict(k=None), dict(v=None), dict(k=ODD), dict(ks=1020), dict(vs=1016),
               dict(cu=None), dict(ln=None), dict(batch=-1), dict(rows=-1), dict(rows=1 << 31),
               dict(q=ODD), dict(qs=2040), dict(qs=2052), dict(q_out=None), dict(hq=0),
               dict(q=None), dict(q=None, hq=0), dict(base=-1.0), dict(base=float("inf")),
               dict(base=float("nan")), dict(qn=P, eps=-1.0)):
        assert _append(ok, **kw) == tg.TG_ERR_INVALID_ARG, kw
    # in place only where the rows are already apart as q_out's
    assert _append(ok, q=P, q_out=P, qs=4096) == tg.TG_ERR_INVALID_ARG
    # nothing to do: fine, whatever the pointers
    assert _append(ok, k=None, v=None, q=None, q_out=None, hq=0, rows=0) == tg.TG_OK
    assert _append(ok, batch=0, q=None, q_out=None, hq=0) == tg.TG_OK


def test_attn_refusals():
    ok = _cache()
    assert _attn(None) == tg.TG_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(out=None), dict(q=ODD), dict(out=ODD), dict(qs=2040),
               dict(qs=2052), dict(hq=12), dict(hq=0), dict(cu=None), dict(ln=None),
               dict(rows=-1), dict(batch=-1), dict(max_kv=0), dict(max_kv=257)):
        assert _attn(ok, **kw) == tg.TG_ERR_INVALID_ARG, kw
    assert _attn(ok, q=None, out=None, rows=0) == tg.TG_OK
    assert _attn(ok, batch=0) == tg.TG_OK
    need = tg.tg_workspace_size(tg.TG_OP_PAGED_ATTN, n=2, k=5, n_heads_q=16, n_heads_kv=8,
                                head_dim=128)
    if need:
        assert _attn(ok, ws_bytes=need - 1) == tg.TG_ERR_WORKSPACE
        assert _attn(ok, ws=None) == tg.TG_ERR_WORKSPACE


def test_quantize_refusals():
    f = tg._quantize
    assert f(P, 64, 5, 64, 7, P, P, None) == tg.TG_ERR_UNSUPPORTED
    assert f(P, 72, 5, 72, tg.TG_BF16, P, P, None) == tg.TG_ERR_UNSUPPORTED  # cols % 16
    for a in ((None, 64, 5, 64, tg.TG_BF16, P, P), (P, 64, 5, 64, tg.TG_BF16, None, P),
              (P, 64, 5, 64, tg.TG_BF16, P, None), (P, 48, 5, 64, tg.TG_BF16, P, P),
              (P, 68, 5, 64, tg.TG_BF16, P, P), (ODD, 64, 5, 64, tg.TG_BF16, P, P),
              (P, 64, 5, 64, tg.TG_BF16, ODD, P), (P, 64, -1, 64, tg.TG_BF16, P, P),
              (P, 64, 5, 0, tg.TG_BF16, P, P)):
        assert f(*a, None) == tg.TG_ERR_INVALID_ARG, a
    assert f(None, 64, 0, 64, tg.TG_F32, None, None, None) == tg.TG_OK


def test_linear_quantized_refusals():
    f = tg._linear_q
    assert f(P, P, P, P, None, 5, 64, 64, 9, P, None) == tg.TG_ERR_UNSUPPORTED
    for n, k in ((48, 64), (64, 72), (64, 131072)):
        assert f(P, P, P, P, None, 5, n, k, tg.TG_BF16, P, None) == tg.TG_ERR_UNSUPPORTED
    for a in ((None, P, P, P, None, 5), (P, None, P, P, None, 5), (P, P, None, P, None, 5),
              (P, P, P, None, None, 5), (ODD, P, P, P, None, 5), (P, P, ODD, P, None, 5),
              (P, P, P, P, ODD, 5), (P, P, P, P, None, -1), (P, P, P, P, None, 1 << 31)):
        assert f(*a, 64, 64, tg.TG_BF16, P, None) == tg.TG_ERR_INVALID_ARG, a
    assert f(P, P, P, P, None, 5, 64, 64, tg.TG_BF16, None, None) == tg.TG_ERR_INVALID_ARG
    assert f(None, None, P, P, None, 0, 64, 64, tg.TG_BF16, None, None) == tg.TG_OK


def test_python_shapes_are_checked():
    """The binding refuses tensors whose shape, type or layout does not fit
    (host tensors: nothing is launched)."""
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    table = torch.zeros(2, 2, dtype=torch.int32)
    c = tg.PagedKV(k, k.clone(), table)
    assert c.capacity == 32 and c.batch == 2
    for args in ((k, k[:3], table), (k, k, table.long()), (k, k, table[0]),
                 (k, k, table, torch.zeros(4, 15)), (k.transpose(1, 2), k.transpose(1, 2), table),
                 (k.half(), k.half(), table)):
        with pytest.raises(ValueError):
            tg.PagedKV(*args)
    # pages of one layer of a pool that holds several
    pool = torch.zeros(4, 3, 16, 2, 64)
    assert tg.PagedKV(pool[:, 1], pool[:, 2], table).c.k_page_stride == 3 * 16 * 2 * 64
    cu, ln = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    for bad in (lambda: tg.tg_paged_append(c, x.float(), x, cu, ln),
                lambda: tg.tg_paged_append(c, x, x[:4], cu, ln),
                lambda: tg.tg_paged_append(c, x, x, cu, ln, q_out=x),
                lambda: tg.tg_paged_attn(c, x[..., ::2], cu, ln),
                lambda: tg.tg_paged_attn(c, x, cu, ln, out=x[:4])):
        with pytest.raises(ValueError):
            bad()
    xq, wq = torch.zeros(3, 64, dtype=torch.int8), torch.zeros(32, 64, dtype=torch.int8)
    s3, s32 = torch.zeros(3), torch.zeros(32)
    for bad in (lambda: tg.tg_linear_quantized(xq, s3, wq[:, :48], s32),
                lambda: tg.tg_linear_quantized(xq.float(), s3, wq, s32),
                lambda: tg.tg_linear_quantized(xq, s3, wq, s32, residual=torch.zeros(3, 32)),
                lambda: tg.tg_quantize_rows(torch.zeros(4, 64).t())):
        with pytest.raises(ValueError):
            bad()


def test_host_tensors_are_refused():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    c = tg.PagedKV(k, k.clone(), torch.zeros(2, 2, dtype=torch.int32))
    cu, ln = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    xq, wq = torch.zeros(3, 64, dtype=torch.int8), torch.zeros(32, 64, dtype=torch.int8)
    for bad in (lambda: tg.tg_paged_append(c, x, x, cu, ln), lambda: tg.tg_paged_attn(c, x, cu, ln),
                lambda: tg.tg_quantize_rows(torch.zeros(4, 64)),
                lambda: tg.tg_linear_quantized(xq, torch.zeros(3), wq, torch.zeros(32))):
        with pytest.raises(ValueError):
            bad()

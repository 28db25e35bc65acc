"""GPU test of what a trace says of the serving calls: their algorithmic work."""

import pytest
import torch

from tests.test_gpu_paged import BF, F32, Setup

pytestmark = pytest.mark.gpu

tg = pytest.importorskip("learned_token_pruning_score_b200")


def test_trace_of_the_serving_calls():
    st = Setup([(1, 300), (1, 299)], 8, 4, 128, 32, BF, seed=60).fill()
    q, (gain, tau) = st.queries(), st.gates()
    x = torch.randn(2, 16, 128, device="cuda").to(BF)
    a = torch.randn(40, 256, device="cuda").to(BF)
    wq, ws = tg.tg_quantize_rows(torch.randn(64, 256, device="cuda"))
    res = torch.randn(40, 64, device="cuda")
    tg.tg_trace_start()
    tg.tg_paged_append(st.cache, x[:, 8:12], x[:, 12:], st.cu, st.kv_len, q=x[:, :8])
    tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, max_kv=301)
    tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, max_kv=320)
    xq, xs = tg.tg_quantize_rows(a)
    tg.tg_linear_quantized(xq, xs, wq, ws)
    tg.tg_linear_quantized(xq, xs, wq, ws, residual=res, dtype=F32)
    got = [(r["kernel"], r["rows"], r["flops"], r["bytes"]) for r in tg.tg_trace_stop()]
    io = 2 * 2 * 8 * 128 * 2  # q in, out out
    kv = 2 * 4 * 128 * 2      # a key and a value of every head
    assert got == [
        ("paged_append", 2, 0.0, 2.0 * 2 * 16 * 128 * 2),
        ("paged_attn", 2, 4.0 * 128 * 8 * 2 * 301, io + 2.0 * 301 * (kv + 4)),
        ("paged_attn", 2, 4.0 * 128 * 8 * 2 * 320, io + 2.0 * 320 * kv),
        ("quantize", 40, 0.0, 40.0 * (256 * 3 + 4)),
        ("gemm_int", 40, 2.0 * 40 * 64 * 256, 40.0 * 260 + 64 * 260 + 40 * 64 * 2),
        ("gemm_int", 40, 2.0 * 40 * 64 * 256, 40.0 * 260 + 64 * 260 + 40 * 64 * 4 * 2),
    ]

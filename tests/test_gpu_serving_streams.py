"""GPU tests of `stream=` in the serving calls: what a call allocates belongs to
the stream that it runs on. Work that waits on the current stream (a bounded
spin) must neither reach results that a call on another stream writes meanwhile
nor lose results that it was still to read."""

import pytest
import torch

from tests.test_gpu_paged import BF, Setup

pytestmark = pytest.mark.gpu

tg = pytest.importorskip("learned_token_pruning_score_b200")

SPIN = 20_000_000  # about 10 ms


@pytest.fixture(autouse=True)
def _no_device_errors():
    tg.tg_device_error(clear=True)
    yield
    assert tg.tg_device_error() == 0


def calls():
    """name -> a call with stream=, whose results it returns as a tuple."""
    g = torch.Generator(device="cuda").manual_seed(70)
    x = torch.randn(256, 4096, generator=g, device="cuda").to(BF)
    xq, xs = tg.tg_quantize_rows(x)
    wq, ws = tg.tg_quantize_rows(torch.randn(1024, 4096, generator=g, device="cuda"))
    st = Setup([(1, 5000), (1, 3000)], 16, 8, 128, 64, BF, seed=71).fill()
    q = st.queries()
    row = torch.randn(2, 32, 128, generator=g, device="cuda").to(BF)
    return {
        "quantize": lambda s: tg.tg_quantize_rows(x, stream=s),
        "linear": lambda s: (tg.tg_linear_quantized(xq, xs, wq, ws, stream=s),),
        "attn": lambda s: (tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, stream=s),),
        "append": lambda s: (tg.tg_paged_append(st.cache, row[:, 16:24], row[:, 24:], st.cu,
                                                st.kv_len, q=row[:, :16], stream=s),),
    }


@pytest.mark.parametrize("name", ["quantize", "linear", "attn", "append"])
def test_freed_memory_of_the_current_stream_is_not_used(name):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    need = tg.tg_workspace_size(tg.TG_OP_PAGED_ATTN, n=2, k=2, n_heads_q=16, n_heads_kv=8,
                                head_dim=128)
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        old = [torch.empty_like(t) for t in want] + [torch.empty(need, dtype=torch.uint8, device="cuda")]
        torch.cuda._sleep(SPIN)
        for t in old:
            t.fill_(99)
        del old, t
        got = call(side)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", ["quantize", "linear", "attn", "append"])
def test_results_stay_until_the_current_stream_has_read_them(name):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    side.synchronize()
    torch.cuda._sleep(SPIN)
    copies = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(side):
        for _ in range(3):
            new = [torch.full(s, 99, dtype=d, device="cuda") for s, d in shapes]
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b)
    assert new

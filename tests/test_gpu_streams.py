"""GPU tests of `stream=` in the calls that allocate from Python: what a call
allocates (results, workspace) belongs to the stream that it runs on."""

import pytest
import torch

pytestmark = pytest.mark.gpu

tg = pytest.importorskip("learned_token_pruning_score_b200")

SPIN = 20_000_000  # about 10 ms
BF = torch.bfloat16


def calls():
    """name -> a call with stream=, whose results it returns as a tuple."""
    g = torch.Generator(device="cuda").manual_seed(80)
    x = torch.randn(512, 1024, generator=g, device="cuda").to(BF)
    w = torch.randn(1024, 1024, generator=g, device="cuda").to(BF)
    scores = torch.randn(4096, generator=g, device="cuda")
    qkv = [torch.randn(512, h, 128, generator=g, device="cuda").to(BF) for h in (8, 2, 2)]
    pos = torch.arange(512, dtype=torch.int32, device="cuda")
    return {
        "linear": lambda s: (tg.tg_linear(x, w, stream=s),),
        "positional": lambda s: (tg.tg_linear(x, w, None, None, s),),
        "select": lambda s: (tg.tg_topk_select(scores, None, 1000, stream=s),),
        "attn": lambda s: (tg.tg_gated_attn_prefill(*qkv, pos, stream=s),),
        "forward": lambda s: tg.tg_gated_attn_forward(*qkv, pos, stream=s),
    }


NAMES = ["linear", "positional", "select", "attn", "forward"]
HANDLES = {"stream": lambda s: s, "handle": lambda s: s.cuda_stream}


@pytest.mark.parametrize("kind", list(HANDLES))
@pytest.mark.parametrize("name", NAMES)
def test_freed_memory_of_the_current_stream_is_not_used(name, kind):
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        old = [torch.empty_like(t) for t in want] + [
            torch.empty(n, dtype=torch.uint8, device="cuda") for n in (1 << 16, 1 << 22)]
        torch.cuda._sleep(SPIN)
        for t in old:
            t.fill_(99)
        del old, t
        got = call(HANDLES[kind](side))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("name", NAMES)
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


def test_the_default_stream_by_its_handle():
    call = calls()["linear"]
    want = call(None)[0].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = call(0)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)

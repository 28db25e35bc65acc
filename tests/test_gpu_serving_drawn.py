"""GPU parity of the serving calls at sizes drawn from the whole range of
perf/operators.py (a fixed seed; cases of up to 128 MB and 20 GFLOP), against
its values in 64 bits.

Tolerances, with u = eps / 2 of the type (bf16 2^-8, fp32 2^-24):
  append   those of test_gpu_paged.py, the size of a rotated pair taken from
           the result (|lo| + |hi| <= sqrt(2) of its length, which the rotation
           keeps); v exact
  attn     those of test_gpu_paged.py, from the same inputs
  quant    the integers exact, the scale one rounding
  linear   four fp32 roundings of the product, one of the sum with the
           residual, one to the type
"""

import math
import random
from types import SimpleNamespace

import pytest
import torch

import perf.operators as P
from tests.test_gpu_paged import U, attn_reference

pytestmark = pytest.mark.gpu

tg = pytest.importorskip("learned_token_pruning_score_b200")

PER_OPERATOR = 10


def drawn():
    rng, left, out = random.Random(20), dict(append=0, attn=0, quant=0, linear=0), []
    while min(left.values()) < PER_OPERATOR:
        c = P.draw(rng)
        w = P.work(c)
        if left[c["op"]] < PER_OPERATOR and w["bytes"] <= 1 << 27 and w["flops"] <= 2e10:
            left[c["op"]] += 1
            out.append(dict(c, name=f"{c['op']}-{left[c['op']]}"))
    return out


@pytest.mark.parametrize("case", drawn(), ids=lambda c: c["name"])
def test_drawn_sizes(case, monkeypatch):
    monkeypatch.setattr(P, "own", True)
    tg.tg_device_error(clear=True)
    st = P.prepare(case, 5)
    got, want = P.run(st), P.exact(case, 5)
    u = U[torch.bfloat16 if case["dtype"] == "bf16" else torch.float32]
    if case["op"] == "quant":
        assert torch.equal(got["xq"], want["xq"])
        check(got["scale"], want["scale"], 2.0 ** -24 * want["scale"])
    elif case["op"] == "linear":
        res = 0.0 if st["residual"] is None else st["residual"].double()
        check(got, want, 4 * 2.0 ** -24 * (want - res).abs() + (2.0 ** -24 + u) * want.abs())
    elif case["op"] == "append":
        assert set(got) == set(want) and torch.equal(got["v_pages"].double(), want["v_pages"])
        rel = 2.0 ** -21 + ((case["dh"] + 8) * 2.0 ** -24 if case["norm"] else 0.0)
        for name in ("q", "k_pages"):
            y = want[name]
            pair = torch.hypot(*y.chunk(2, -1)).repeat(*[1] * (y.dim() - 1), 2)
            check(got[name], y, u * y.abs() + math.sqrt(2.0) * rel * pair)
        if "bias" in want:
            check(got["bias"], want["bias"], 2.0 ** -21 * want["bias"].abs() + 2.0 ** -24)
    else:
        q = st["q"]
        like = SimpleNamespace(
            rows=q.shape[0], hq=case["hq"], hkv=case["hkv"], dh=case["dh"], dtype=q.dtype,
            lens=st["lens"], cu_host=st["cu_host"], k=st["k_pages"], v=st["v_pages"],
            bias=st["bias"], where=lambda b, lo, hi: P._slots(st["table"], b, lo, hi, case["page"]))
        _, _, tol, _ = attn_reference(like, q, st["gain"], st["tau"])
        check(got, want, tol)
    assert tg.tg_device_error() == 0


def check(got, want, tol):
    over = (got.double() - want).abs() - 1.01 * tol
    assert (over <= 0).all(), float(over.max())

"""GPU tests of the paged attention where logits are far from zero: gate biases
of -1e9 and beyond that still leave their keys in place (only a logit below
-1e30 removes one), in every variant.

Tolerances are those derived in test_gpu_paged.py. Next to an ordinary key, a
key whose bias is -1e9 has a weight of exactly 0 in 64 bits, too: such rows are
held to the result without these keys. A row that has no other key gets a mean
of their values: the logits differ by less than a unit in the last place of
their fp32 sums (64 at 1e9), so that the weights may be any; the output is held
to the range of the values, with one rounding of the weights, of their sum and
of the output (each 2^-8 in bf16), and lse to its tolerance.
"""

import math

import pytest
import torch

from tests.test_gpu_paged import Setup, attn_reference, gen
from tests.test_gpu_serving import VARIANTS

pytestmark = pytest.mark.gpu

tg = pytest.importorskip("learned_token_pruning_score_b200")


@pytest.fixture(autouse=True)
def _no_device_errors():
    tg.tg_device_error(clear=True)
    yield
    assert tg.tg_device_error() == 0


@pytest.fixture(params=list(VARIANTS))
def variant(request):
    lens, hq, hkv, dh, page, dt = VARIANTS[request.param]
    return Setup(lens, hq, hkv, dh, page, dt, seed=60).fill()


def gates(st):
    """Gains that are not small, so that each head has its keys far away."""
    g = gen(61)
    return (0.2 + 1.8 * torch.rand(st.hq, generator=g, device="cuda"),
            0.5 + torch.rand(st.hq, generator=g, device="cuda"))


FAR = {  # which of a request's `total` keys j are far
    "first 200": lambda j, total: j < 200,
    "all": lambda j, total: j >= 0,
    "odd tiles": lambda j, total: j // 128 % 2 == 1,
    "even tiles": lambda j, total: j // 128 % 2 == 0,
    "first half": lambda j, total: j < total // 2,
    "all but the last": lambda j, total: j < total - 1,
}


@pytest.mark.parametrize("where", list(FAR))
def test_far_biases(variant, where):
    st = variant
    q, (gain, tau) = st.queries(), gates(st)
    real = st.bias.clone()
    far = torch.zeros_like(st.bias, dtype=torch.bool)
    seen = torch.zeros(2, st.rows, st.hkv, st.dh, device="cuda")  # lowest and highest values
    for b, (n, p) in enumerate(st.lens):
        pg, r = st.where(b, 0, n + p)
        far[pg, r] = FAR[where](torch.arange(n + p, device="cuda"), n + p)
        vb = st.v[pg, r].float()
        at = slice(st.cu_host[b], st.cu_host[b] + n)
        seen[0, at] = vb.cummin(0).values[p:]
        seen[1, at] = vb.cummax(0).values[p:]
    low, high = (x.repeat_interleave(st.hq // st.hkv, 1) for x in seen)
    slack = 2.0 ** -6 * torch.maximum(low.abs(), high.abs())
    st.bias[far] = -math.inf
    near, near_lse, tol, tol_l = attn_reference(st, q, gain, tau)
    none = torch.isneginf(near_lse)  # rows (by head) that see far keys alone
    for size in (1e9, 1e10, 1e12, 1e15, 1e25):
        st.bias.copy_(real)
        st.bias[far] = -size
        _, want_lse, _, far_tol = attn_reference(st, q, gain, tau)
        lse = torch.full((st.hq, st.rows), 7.0, device="cuda")
        out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, lse=lse)
        assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all(), size
        rows = ~none.t()
        over = (out.double() - near).abs() - tol
        assert (over <= 0)[rows].all(), (size, float(over[rows].max()))
        inside = (out.float() >= low - slack) & (out.float() <= high + slack)
        assert inside[~rows].all(), size
        over = (lse.double() - want_lse).abs() - torch.where(none, far_tol, tol_l)
        assert (over <= 0).all(), (size, float(over.max()))

"""GPU tests of the paged attention's log-sum-exp: its accuracy, and NaN
logits, which show in it."""

import math

import pytest
import torch

from tests.test_gpu_paged import BF, Setup, attn_reference
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


@pytest.mark.parametrize("key", [0, 3, 6, 7, 13, 30])
def test_nan_logits_reach_lse(variant, key):
    """A NaN in one key, at each kind of place among 32: its rows' outputs and
    lse are NaN, and no other row's."""
    st = variant
    q, (gain, tau) = st.queries(), st.gates()
    n, p = st.lens[1]
    st.k[st.table[1, key // st.page].long(), key % st.page, 0, 1] = math.nan
    lse = torch.full((st.hq, st.rows), 7.0, device="cuda")
    out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, lse=lse)
    sees = torch.zeros(st.rows, st.hq, dtype=torch.bool, device="cuda")
    sees[st.cu_host[1] + max(0, key - p):st.cu_host[2], :st.hq // st.hkv] = True
    assert torch.equal(torch.isnan(out.float()).all(-1), sees)
    assert torch.equal(torch.isnan(lse.t()), sees)
    assert torch.isfinite(out.float())[~sees].all()


@pytest.mark.parametrize("key", [1, 6, 15])
def test_infinite_logits_show(variant, key):
    """A gate bias of +infinity: the softmax is inf - inf, NaN for the rows
    that see the key, in every head with a gain."""
    st = variant
    q, (gain, tau) = st.queries(), st.gates()
    gain += 0.1
    n, p = st.lens[1]
    st.bias[st.table[1, key // st.page].long(), key % st.page] = math.inf
    lse = torch.full((st.hq, st.rows), 7.0, device="cuda")
    out = tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, lse=lse)
    sees = torch.zeros(st.rows, st.hq, dtype=torch.bool, device="cuda")
    sees[st.cu_host[1] + max(0, key - p):st.cu_host[2]] = True
    assert torch.equal(torch.isnan(out.float()).all(-1), sees)
    assert torch.equal(~torch.isfinite(lse.t()), sees)
    assert torch.isfinite(out.float())[~sees].all()


@pytest.mark.parametrize("shape", [([(300, 517)], 4, 2, 128), ([(100, 60), (9, 30)], 8, 2, 64)],
                         ids=["256-row tiles", "128-row tiles"])
@pytest.mark.parametrize("key", range(16))
def test_exponentials_of_the_chunk_kernel(shape, key):
    """Rows that see one key alone: lse is its logit, and shows the exponential
    of each place of a key. The tolerance is that of test_gpu_paged.py with the
    exponential within 4e-6 (2.9e-6 and four fp32 roundings) instead of 1.5e-4."""
    lens, hq, hkv, dh = shape
    st = Setup(lens, hq, hkv, dh, 64, BF, seed=62).fill()
    for b, (n, p) in enumerate(lens):
        pg, r = st.where(b, 0, n + p)
        st.bias[pg, r] = -math.inf
        st.bias[pg[key], r[key]] = 0.0
    q, (gain, tau) = st.queries(), st.gates()
    gain += 0.1
    lse = torch.full((st.hq, st.rows), 7.0, device="cuda")
    tg.tg_paged_attn(st.cache, q, st.cu, st.kv_len, gain=gain, tau=tau, lse=lse)
    _, want, _, tol = attn_reference(st, q, gain, tau)
    on = ~torch.isneginf(want)
    assert torch.equal(torch.isneginf(lse), ~on)
    over = (lse.double() - want).abs() - (tol - 1.5e-4 + 4e-6)
    assert (over[on] <= 0).all(), float(over[on].max())
